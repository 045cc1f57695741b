"""Rotation, prompt attention, tree attention and commit on the GPU against plain float64 forms."""
import itertools
import math

import numpy as np
import pytest
import torch

import _quant as Q
import _rows as R
from _rows import i32
from long_context_serving_gb300 import bsattn as B

pytestmark = pytest.mark.gpu


def _sync_status(c):
    torch.cuda.synchronize()
    return int(c.status.item())


# ---------------------------------------------------------------------------------------
# Rotation
# ---------------------------------------------------------------------------------------
def _rope_reference(x, w, pos, freq, rot, inter, m, eps):
    """x float64 [rows][heads][d]."""
    x = x.copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    angle = pos[:, None].astype(np.float64) * freq
    c, s = m * np.cos(angle)[:, None], m * np.sin(angle)[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * c - b * s, b * c + a * s
    size = np.zeros_like(x) + np.abs(x)
    h = m * np.hypot(a, b)
    if inter:
        x[..., 0:rot:2], x[..., 1:rot:2] = ya, yb
        size[..., 0:rot:2], size[..., 1:rot:2] = h, h
    else:
        x[..., :rot // 2], x[..., rot // 2:rot] = ya, yb
        size[..., :rot // 2], size[..., rot // 2:rot] = h, h
    return x, size


def _rope_tol(size, want, norm, d, dtype):
    """An angle is off by 2^-24 of a turn, its cosine and sine by two steps more, the two products
    and their sum by a half step each; a norm by half steps of a sum of d squares (halved by the root)
    and four operations. Then one rounding to the output type."""
    u = 2.0 ** -24
    rel = 2 * math.pi * u + 8 * u + ((d / 2 + 4) * u if norm else 0)
    return rel * size + (R.HALF_BF16 if dtype == torch.bfloat16 else u) * (np.abs(want) + rel * size) + 1e-38


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (128, 64, False), (64, 64, False),
                                         (64, 32, True), (64, 16, False), (128, 16, True), (128, 112, False)])
@pytest.mark.parametrize("act,code", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("norms", [(True, True), (False, False), (True, False)])
def test_rope_against_the_formula(d, rot, inter, act, code, norms):
    rng = np.random.default_rng(d + rot)
    Hq, Hkv, rows = 6, 2, 21
    at = R.CODE[act]
    x = torch.as_tensor(rng.standard_normal((rows, (Hq + 2 * Hkv) * d + 16)).astype(np.float32)).to(at)
    pos = np.concatenate([[0, 1, 2, (1 << 24) - 1, 1000003, 131071], rng.integers(0, 200000, rows - 6)])
    freq = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    w = [(1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if n else None for n in norms]
    xd = x.cuda()
    dims = B.Dims(batch=1, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, page_size=16, max_pages_per_unit=1,
                  max_blocks_per_unit=1, max_sel_per_unit=1, max_subs_per_unit=1, max_gather_pages_per_unit=1, n_pages=1,
                  kv_dtype=R.KIND[code], q_dtype=R.KIND[act])
    fd = torch.as_tensor(freq).cuda()
    wd = [None if v is None else torch.as_tensor(v).cuda() for v in w]
    rope = B.Rope(inv_freq=fd.data_ptr(), rot_dim=rot, interleaved=int(inter), magnitude=1.25,
                  q_weight=0 if wd[0] is None else wd[0].data_ptr(), k_weight=0 if wd[1] is None else wd[1].data_ptr(),
                  eps=1e-5)
    q_out = torch.full((rows, Hq, d), float("nan"), dtype=at, device="cuda")
    k_out = torch.full((rows, Hkv, d), float("nan"), dtype=at, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pd = i32(pos)
    B.rope_append(dims, rope, xd, xd[:, Hq * d:], None, xd.stride(0), rows, pd, None, None, None, q_out, k_out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    x64 = x.double().numpy()
    for got, lo, heads, wn in ((q_out, 0, Hq, w[0]), (k_out, Hq, Hkv, w[1])):
        src = x64[:, lo * d:(lo + heads) * d].reshape(rows, heads, d)
        want, size = _rope_reference(src, wn, pos, freq, rot, inter, float(np.float32(1.25)), float(np.float32(1e-5)))
        tol = _rope_tol(size, want, wn is not None, d, at)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("rows", [1, 7, 700])
@pytest.mark.parametrize("code", ["bf16", "fp32"])
def test_rope_writes_the_cache(rows, code):
    """K and V land in the slots that positions and tables name, padding rows and other slots stay; the
    keys are those of the call without a cache, V the row's own."""
    rng = np.random.default_rng(rows)
    Bn, Hq, Hkv, d = 3, 4, 2, 64
    seq = rng.integers(0, Bn, rows)
    pos = np.zeros(rows, np.int64)
    for b in range(Bn):                       # distinct positions of each sequence
        n = int((seq == b).sum())
        pos[seq == b] = rng.permutation(3 * n + 5)[:n]
    seq[rng.random(rows) < 0.2] = -2
    c = R.Cache(Bn, Hkv, Hq // Hkv, d, [16 * -(-(int(pos.max()) + 1) // 16)] * Bn, code, seed=rows)
    before_k, before_v = c.k.clone(), c.v.clone()
    x = torch.as_tensor(rng.standard_normal((rows, (Hq + 2 * Hkv) * d)).astype(np.float32)).bfloat16().cuda()
    freq = torch.as_tensor(10000.0 ** (-2.0 * np.arange(d // 2) / d)).cuda()
    rope = B.Rope(inv_freq=freq.data_ptr(), rot_dim=d, interleaved=0, magnitude=1.0, q_weight=0, k_weight=0, eps=0.0)
    q_out = torch.full((rows, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((rows, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (x, x[:, Hq * d:], x[:, (Hq + Hkv) * d:], x.stride(0), rows, i32(pos), i32(seq))
    B.rope_append(c.dims, rope, *args, c.pools(), c.table, q_out, k_out, c.status)
    assert _sync_status(c) == 0
    k_alone = torch.zeros_like(k_out)
    q_alone = torch.zeros_like(q_out)
    B.rope_append(c.dims, rope, *args, None, None, q_alone, k_alone, c.status)
    assert _sync_status(c) == 0
    live = torch.as_tensor(seq >= 0).cuda()
    assert torch.equal(q_out[live], q_alone[live]) and torch.equal(k_out[live], k_alone[live])
    assert (q_out[~live] == 7.0).all() and (k_out[~live] == 7.0).all()
    v = x[:, (Hq + Hkv) * d:].view(rows, Hkv, d)
    for r in range(rows):
        if seq[r] < 0:
            continue
        for h in range(Hkv):
            ph = c.table_np[seq[r] * Hkv + h, pos[r] // 16]
            if code == "bf16":
                assert torch.equal(c.k[ph, pos[r] % 16], k_out[r, h])
            else:
                assert torch.equal(c.k[ph, pos[r] % 16].bfloat16(), k_out[r, h])
            assert torch.equal(c.v[ph, pos[r] % 16], v[r, h].to(c.v.dtype))
            before_k[ph, pos[r] % 16] = c.k[ph, pos[r] % 16]
            before_v[ph, pos[r] % 16] = c.v[ph, pos[r] % 16]
    bits = lambda t: t.view(torch.int16 if code == "bf16" else torch.int32)  # noqa: E731 (unwritten slots hold NaN)
    assert torch.equal(bits(before_k), bits(c.k)) and torch.equal(bits(before_v), bits(c.v))


def test_rope_rows_that_do_not_fit_are_skipped():
    Hq, Hkv, d, rows = 2, 1, 64, 5
    c = R.Cache(1, Hkv, 2, d, [32], "bf16")
    x = torch.ones((rows, 4 * d), dtype=torch.bfloat16, device="cuda")
    freq = torch.zeros(d // 2, dtype=torch.float64, device="cuda")
    rope = B.Rope(inv_freq=freq.data_ptr(), rot_dim=d, interleaved=0, magnitude=1.0, q_weight=0, k_weight=0, eps=0.0)
    for pos, seq, table, code in (([0, -1, 2, 3, 4], [0] * 5, None, B.BS_ERR_INVALID_ARG),
                                  ([0, 1 << 24, 2, 3, 4], [0] * 5, None, B.BS_ERR_INVALID_ARG),
                                  ([0, 1, 2, 3, 4], [0, 1, 0, 0, 0], None, B.BS_ERR_DEVICE_BOUNDS),
                                  ([0, 32, 2, 3, 4], [0] * 5, None, B.BS_ERR_CAPACITY),
                                  ([0, 17, 2, 3, 4], [0] * 5, 99, B.BS_ERR_DEVICE_BOUNDS)):
        q_out = torch.full((rows, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        c.k.fill_(7.0)
        t = c.table.clone()
        if table is not None:
            t[0, 1] = table
        c.status.zero_()
        B.rope_append(c.dims, rope, x, x, x, x.stride(0), rows, i32(pos), i32(seq), c.pools(), t, q_out, None, c.status)
        assert _sync_status(c) == code
        assert (q_out[[0, 2, 3, 4]] == 1.0).all()
        assert (q_out[1] == (1.0 if table is not None else 7.0)).all()
        ph = int(t[0, 0])
        assert (c.k[ph, [0, 2, 3, 4]] == 1.0).all() and (c.k[ph, 1] == 7.0).all()


# ---------------------------------------------------------------------------------------
# Prompt attention
# ---------------------------------------------------------------------------------------
class Prefill:
    def __init__(self, c, new, cls=1, sink=0, local=1, seed=1, pad=3, stride_pad=0, gap=0):
        rng = np.random.default_rng(seed)
        self.c, self.new = c, np.asarray(new, np.int64)
        U, H = c.B * c.Hkv, c.Hkv * c.G
        full = lambda x: np.broadcast_to(np.asarray(x), (U,)).astype(np.int64)  # noqa: E731
        self.cls, self.sink, self.local = full(cls), full(sink), full(local)
        # (rows of no sequence before, between and behind)
        self.row0 = pad + np.cumsum(self.new + gap) - self.new - gap
        self.rows = int(self.row0[-1] + self.new[-1]) + pad
        self.q_np = R.bf16(rng.standard_normal((self.rows, H, c.d)) * 1.5)
        q = torch.full((self.rows, H * c.d + stride_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        q[:, :H * c.d] = torch.as_tensor(self.q_np.reshape(self.rows, -1)).cuda().bfloat16()
        self.q = q
        self.old = i32(c.lens - self.new)
        self.begin = i32(self.row0)
        self.cfg_t = [i32(x) for x in (self.cls, self.sink, self.local)]
        self.cfg = B.HeadCfg(cls=self.cfg_t[0].data_ptr(), sink_tokens=self.cfg_t[1].data_ptr(),
                             local_tokens=self.cfg_t[2].data_ptr())
        self.max_new = max(1, int(self.new.max()))
        self.out = torch.full((self.rows, H, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.rows, H), 7.0, dtype=torch.float32, device="cuda")
        size = B.prefill_workspace_size(c.dims, self.rows, self.max_new)
        self.ws = torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device="cuda")   # (NaN: nothing of it may be read unwritten)

    def run(self, lse=True, stream=None):
        B.prefill_attn(self.c.dims, self.q, self.q.stride(0), self.rows, self.c.kv(), self.cfg, self.old, self.begin,
                       self.max_new, self.out, self.lse if lse else None, self.ws, self.c.status, stream)

    def check(self, rows=None, skip_units=(), lse=True):
        c = self.c
        out, z = self.out.double().cpu().numpy(), self.lse.cpu().numpy()
        untouched = np.ones(self.rows, bool)
        for b in range(c.B):
            o, n, r0 = int(c.lens[b] - self.new[b]), int(self.new[b]), int(self.row0[b])
            untouched[r0:r0 + n] = False
            pick = range(n) if rows is None or n <= rows else sorted(
                set(np.linspace(0, n - 1, rows).astype(int).tolist()))
            for h in range(c.Hkv):
                u = b * c.Hkv + h
                if u in skip_units:
                    continue
                for i in pick:
                    s = R.prefill_seen(o + i, len(c.K[u]), self.cls[u] == B.BS_STREAMING, self.sink[u], self.local[u])
                    for g in range(c.G):
                        hq = h * c.G + g
                        want = R.attend_row(self.q_np[r0 + i, hq].astype(np.float64), c.K[u][s], c.V[u][s])
                        R.check_row(out[r0 + i, hq], z[r0 + i, hq] if lse else None, want, (b, h, i, g))
        assert (out[untouched] == 7.0).all() and (z[untouched] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new,lens", [(4, [1], [1]), (4, [17], [17]), (1, [130], [130]), (8, [33, 1, 0, 16], [40, 1, 5, 16]),
                                        (7, [50], [180]), (3, [1, 2, 1], [300, 129, 16]), (4, [70, 5], [71, 260]),
                                        (5, [0], [3])])
def test_prefill_dense(kind, d, G, new, lens):
    c = R.Cache(len(new), 2, G, d, lens, kind, seed=sum(lens))
    p = Prefill(c, new, gap=1)
    p.run()
    assert _sync_status(c) == 0
    p.check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sink,local", [(0, 1), (1, 1), (0, 16), (4, 17), (16, 100), (37, 128), (128, 1000), (5000, 1),
                                        (0, 2 ** 31 - 1), (2 ** 31 - 1, 1), (1, 150)])
@pytest.mark.parametrize("new,lens", [([40, 1], [333, 290]), ([300], [300])])
def test_prefill_windows(kind, sink, local, new, lens):
    c = R.Cache(len(new), 2, 4, 64, lens, kind, seed=local % 1000 + sink % 1000)
    cls = [0, 1] * len(new)                       # a streaming and a retrieval head in each sequence
    p = Prefill(c, new, cls=cls, sink=sink, local=local)
    p.run()
    assert _sync_status(c) == 0
    p.check()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 128), ("int8", 64)])
def test_prefill_many_tiles(kind, d):
    """Blocks of two row tiles, key tiles past the ring's length, and rows that end inside a tile."""
    c = R.Cache(2, 2, 4, d, [1500, 700], kind)
    p = Prefill(c, [1100, 333], cls=[1, 0, 2, 1], sink=20, local=260)
    p.run()
    assert _sync_status(c) == 0
    p.check(rows=60)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("new,max_pages", [([1, 1], 600), ([3, 40], 600)])
def test_prefill_splits(kind, new, max_pages):
    """Few rows over long caches are split; the merge takes every piece, and only those that exist."""
    c = R.Cache(2, 1, 4, 128, [5000, 1111], kind, max_pages=max_pages)
    p = Prefill(c, new)
    assert B.prefill_workspace_size(c.dims, p.rows, p.max_new) > 0
    p.run()
    assert _sync_status(c) == 0
    p.check()
    first = p.out.clone()
    p.ws.fill_(0xFF)
    p.run()
    assert _sync_status(c) == 0
    assert torch.equal(first, p.out)              # bitwise the same again


@pytest.mark.parametrize("units", [1, 200])
def test_prefill_more_units_than_a_wave(units):
    c = R.Cache(units, 1, 2, 64, [40 + (7 * i) % 600 for i in range(units)], "bf16", max_pages=512)
    p = Prefill(c, [1 + i % 3 for i in range(units)])
    p.run()
    assert _sync_status(c) == 0
    p.check()


def test_prefill_many_sequences():
    """Blocks are found among hundreds of sequences, most of them with few or no new tokens."""
    new = [(5 * i) % 4 if i % 97 else 90 + i // 97 for i in range(300)]
    c = R.Cache(300, 1, 4, 64, [n + (3 * i) % 50 for i, n in enumerate(new)], "bf16")
    p = Prefill(c, new)
    p.run()
    assert _sync_status(c) == 0
    p.check(rows=12)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_waits_that_run_out_are_reported(kind):
    """With a limit of a microsecond the waits for the first copies may run out: the call then says so,
    ends, and the next one is right."""
    c = R.Cache(2, 2, 4, 128, [3000, 900], kind, max_gather_pages_per_unit=192)
    p, t = Prefill(c, [300, 40]), Tree(c, [9, 33], g=32)
    limit = B.wait_limit_ns()
    try:
        B.set_wait_limit_ns(1000)
        for x in (p, t):
            x.run()
            assert _sync_status(c) in (0, B.BS_ERR_TIMEOUT)
            c.status.zero_()
    finally:
        B.set_wait_limit_ns(limit)
    for x in (p, t):
        x.out.fill_(7.0)
        x.lse.fill_(7.0)
        x.run()
    assert _sync_status(c) == 0
    p.check(rows=20)
    t.check()


def test_prefill_strides_and_no_lse():
    c = R.Cache(2, 2, 4, 128, [77, 20], "bf16")
    p = Prefill(c, [20, 20], stride_pad=8 * 128)
    p.run(lse=False)
    assert _sync_status(c) == 0
    assert (p.lse == 7.0).all()
    p.lse.copy_(p.lse)
    out = p.out.clone()
    p.run()
    assert _sync_status(c) == 0
    p.check()
    assert torch.equal(out, p.out)


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_prefill_unseen_keys_do_not_matter(what):
    """A key behind a row, or outside its window, is nothing to it, whatever it holds; the rows that
    see it get what the formula gives."""
    c = R.Cache(1, 2, 4, 128, [200], "bf16")
    p = Prefill(c, [150], cls=[1, 0], sink=4, local=20)
    x = float(what)
    for u in range(2):
        ph = c.table_np[u, 160 // 16]
        c.v[ph, 160 % 16, 5] = x
        c.K[u][160], c.V[u][160] = c.K[u][160], c.V[u][160].copy()
        c.V[u][160, 5] = x
        ph = c.table_np[u, 120 // 16]
        c.k[ph, 120 % 16, 9] = x
    p.run()
    assert _sync_status(c) == 0
    out = p.out.double().cpu().numpy()
    for u, h, i, g in itertools.product(range(2), [0], range(150), range(4)):
        pos = 50 + i
        s = R.prefill_seen(pos, 200, u == 1, 4, 20)
        row = out[p.row0[0] + i, u * 4 + g]
        if s[120]:
            continue                              # a NaN or infinite logit: see below
        if s[160]:
            assert not np.isfinite(row[5])
            keep = np.arange(128) != 5
        else:
            keep = np.ones(128, bool)
        V = np.where(np.isfinite(c.V[u]), c.V[u], 0.0)
        want = R.attend_row(p.q_np[p.row0[0] + i, u * 4 + g].astype(np.float64), c.K[u][s], V[s])
        R.check_row(row[keep], None, tuple(w[keep] if isinstance(w, np.ndarray) else w for w in want), (u, i, g))
    if what == "nan":                             # a NaN key makes every row that sees it NaN
        assert np.isnan(out[p.row0[0] + 70:p.row0[0] + 110, :4]).all()
        assert np.isfinite(out[p.row0[0]:p.row0[0] + 70]).all()


def test_prefill_large_values():
    """Values up to 2^90 and their sums stay finite, also where a later half of a tile passes the first
    by far more than weights are let grow."""
    c = R.Cache(1, 1, 2, 64, [400], "bf16")
    x = float(torch.tensor(1.2e27).bfloat16())
    c.v[:] = x
    p = Prefill(c, [300])
    p.run()
    assert _sync_status(c) == 0
    out = p.out[p.row0[0]:p.row0[0] + 300].double()
    assert ((out - x).abs() <= 2 * R.HALF_BF16 * x).all()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("at", [5, 70, 100, 130, 200, 258])
def test_prefill_logits_that_jump(kind, at):
    """One key whose logit stands hundreds above the others', in either half of the first tiles and in
    later ones: the reference follows it, and rows before it are as ever."""
    c = R.Cache(1, 1, 4, 64, [300], kind, seed=at)
    p = Prefill(c, [300])
    lp, slot = c.table_np[0, at // 16], at % 16
    q = p.q_np[p.row0[0]:p.row0[0] + 300].astype(np.float64)
    key = q[:, 0].mean(0)
    key = key / np.linalg.norm(key) * 4000.0
    if kind == "bf16":
        key = R.bf16(key)
        c.k[lp, slot] = torch.as_tensor(key).bfloat16().cuda()
        c.K[0][at] = key
    else:                                         # the page's scale serves all its keys
        code = Q.round_half_even(key / np.abs(key).max() * 127, "int8")
        s = np.float32(np.abs(key).max() / 127)
        f = np.float64(s) / np.float64(float(c.ks[lp]))
        n = min(16, 300 - at // 16 * 16)
        for t in range(n):
            c.K[0][at // 16 * 16 + t] = c.K[0][at // 16 * 16 + t] * f
        c.ks[lp] = float(s)
        c.k.view(torch.uint8)[lp, slot] = torch.as_tensor(code).cuda()
        c.K[0][at] = Q.decode(code, "int8") * np.float64(s)
    p.run()
    assert _sync_status(c) == 0
    p.check(rows=80)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prefill_cache_of_nan(kind):
    """A cache that holds nothing else gives NaN, and soon: no row is searched to its end."""
    c = R.Cache(1, 2, 4, 128, [6000], kind)
    c.v.view(torch.uint8).fill_(0x7F if kind == "e4m3" else 0xFF)
    p = Prefill(c, [3000])
    p.run()
    assert _sync_status(c) == 0
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    p.run()
    e1.record()
    assert _sync_status(c) == 0
    assert torch.isnan(p.out[p.row0[0]:p.row0[0] + 3000].float()).all()
    assert e0.elapsed_time(e1) < 1000


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("log2", [-126, -100, 20, 100])
def test_prefill_extreme_scales(kind, log2):
    """V scales at either end of their range, K scales that make up for the queries."""
    c = R.Cache(1, 1, 4, 64, [100], kind, k_std=1.0)
    f = 2.0 ** log2
    s = c.vs.double()
    c.vs.copy_((s / s[torch.isfinite(s)].max() * f).float())
    ratio = (c.vs.double().cpu().numpy() / s.cpu().numpy())
    for t in range(100):
        c.V[0][t] = c.V[0][t] * ratio[c.table_np[0, t // 16]]
    p = Prefill(c, [9])
    p.run()
    assert _sync_status(c) == 0
    if log2 == -126:
        # (results may be subnormal in bf16: half a step there is 2^-134)
        out = p.out.double().cpu().numpy()
        for i, g in itertools.product(range(9), range(4)):
            want = R.attend_row(p.q_np[p.row0[0] + i, g].astype(np.float64), c.K[0][:92 + i], c.V[0][:92 + i])
            err = np.abs(out[p.row0[0] + i, g] - want[0])
            assert (err <= 2.5 * R.HALF_BF16 * (np.abs(want[0]) + want[2]) + 2.0 ** -132).all()
    else:
        p.check()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_prefill_every_code(kind):
    """Each code as V of a single key is itself in the result, NaN codes too."""
    codes = np.arange(256, dtype=np.uint8)
    c = R.Cache(2, 1, 1, 128, [1, 1], kind)
    for b in range(2):
        raw = torch.as_tensor(codes[128 * b:128 * b + 128]).cuda()
        c.v.view(torch.uint8)[c.table_np[b, 0], 0] = raw
        c.vs[c.table_np[b, 0]] = 1.0
    p = Prefill(c, [1, 1])
    p.run()
    assert _sync_status(c) == 0
    want = Q.decode(codes, kind).reshape(2, 128)
    got = np.stack([p.out[p.row0[b], 0].double().cpu().numpy() for b in range(2)])
    if kind == "e4m3":
        nan = np.isnan(want)
        assert np.isnan(got[nan]).all()
        want, got = want[~nan], got[~nan]
    assert np.array_equal(got, want)              # one weight of 1: exact


def test_prefill_bad_sequences_and_units():
    lens = [40, 50, 60, 70]
    for field, value, code in (("old", [20, -1, 40, 50], B.BS_ERR_INVALID_ARG),
                               ("old", [20, 51, 40, 50], B.BS_ERR_INVALID_ARG),
                               ("begin", [3, -4, 53, 73], B.BS_ERR_DEVICE_BOUNDS),
                               ("begin", [3, 10 ** 6, 53, 73], B.BS_ERR_DEVICE_BOUNDS),
                               ("max_new", 29, B.BS_ERR_CAPACITY), ("cls", 3, B.BS_ERR_INVALID_ARG),
                               ("local", 0, B.BS_ERR_INVALID_ARG), ("sink", -1, B.BS_ERR_INVALID_ARG),
                               ("page", 10 ** 6, B.BS_ERR_DEVICE_BOUNDS)):
        c = R.Cache(4, 1, 4, 64, lens, "bf16")
        p = Prefill(c, [20, 30, 20, 20], cls=[0, 0, 1, 1], sink=3, local=30)
        if field == "page":
            c.table[1, 0] = value
        elif field in ("cls", "local", "sink"):
            p.cfg_t[("cls", "sink", "local").index(field)][1] = value
        elif field == "max_new":
            p.max_new = value
        else:
            getattr(p, field).copy_(i32(value))
        p.run()
        assert _sync_status(c) == code, field
        if field == "page":
            continue
        out = p.out.double().cpu().numpy()
        assert (out[p.row0[1]:p.row0[1] + 30] == 7.0).all(), field
        p.new[1], keep = 0, p.new[1]
        p.check(skip_units=(1,))
        p.new[1] = keep


# ---------------------------------------------------------------------------------------
# Trees
# ---------------------------------------------------------------------------------------
class Tree:
    def __init__(self, c, n, g=16, sel="all", seed=2, masks=None, pad=2, max_draft=None):
        rng = np.random.default_rng(seed)
        self.c, self.n = c, np.asarray(n, np.int64)
        U, H = c.B * c.Hkv, c.Hkv * c.G
        self.g = np.broadcast_to(np.asarray(g), (U,)).astype(np.int64)
        self.sel = []
        for u in range(U):
            T = int(c.lens[u // c.Hkv])
            nb = -(-T // int(self.g[u]))
            if sel == "all":
                self.sel.append(list(range(nb)))
            elif sel == "none":
                self.sel.append([])
            else:
                k = rng.integers(0, nb + 1)
                self.sel.append(sorted(rng.choice(nb, size=k, replace=False).tolist()))
        self.row0 = pad + np.cumsum(self.n) - self.n
        self.rows = int(self.n.sum()) + 2 * pad
        self.q_np = R.bf16(rng.standard_normal((self.rows, H, c.d)) * 1.5)
        self.kv_np = R.bf16(rng.standard_normal((self.rows, 2, c.Hkv, c.d)))
        self.mask = np.zeros(self.rows, np.uint64)
        for b in range(c.B):
            for i in range(int(self.n[b])):
                m = masks(i, rng) if masks else int(rng.integers(0, 1 << 62)) & ((1 << i) - 1) | 1 << i
                self.mask[self.row0[b] + i] = m
        self.q = torch.as_tensor(self.q_np.reshape(self.rows, -1)).cuda().bfloat16()
        kv = torch.as_tensor(self.kv_np.reshape(self.rows, -1)).cuda().bfloat16()
        kv[:pad] = float("nan")                   # rows of nobody's
        kv[self.rows - pad:] = float("nan")
        self.kv = kv
        self.lists = torch.full((U, c.dims.max_sel_per_unit), -1, dtype=torch.int32)
        for u, s in enumerate(self.sel):
            self.lists[u, :len(s)] = torch.as_tensor(s, dtype=torch.int32)
        self.lists = self.lists.cuda()
        self.cnt = i32([len(s) for s in self.sel])
        self.g_t, self.n_t, self.begin = i32(self.g), i32(self.n), i32(self.row0)
        self.mask_t = torch.as_tensor(self.mask.view(np.int64)).cuda()
        self.cfg = B.HeadCfg(block_tokens=self.g_t.data_ptr())
        self.max_draft = max_draft or max(1, int(self.n.max()))
        self.out = torch.full((self.rows, H, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.rows, H), 7.0, dtype=torch.float32, device="cuda")
        self.ws = torch.full((max(16, B.tree_workspace_size(c.dims, self.max_draft)),), 0xFF, dtype=torch.uint8, device="cuda")

    def drafts(self):
        return B.Drafts(k_new=self.kv.data_ptr(), v_new=self.kv[:, self.c.Hkv * self.c.d:].data_ptr(),
                        row_stride=self.kv.stride(0), n_rows=self.rows, row_begin=self.begin.data_ptr(),
                        n_draft=self.n_t.data_ptr(), visible=self.mask_t.data_ptr(), max_draft=self.max_draft)

    def run(self, lse=True, stream=None):
        c = self.c
        B.tree_decode_attn(c.dims, self.q, self.q.stride(0), c.kv(), self.cfg, self.lists, self.cnt, self.drafts(), self.out,
                           self.lse if lse else None, self.ws, c.status, stream)

    def check(self, skip_units=()):
        c = self.c
        out, z = self.out.double().cpu().numpy(), self.lse.cpu().numpy()
        mine = np.zeros(self.rows, bool)
        for b, h in itertools.product(range(c.B), range(c.Hkv)):
            u, n, r0 = b * c.Hkv + h, int(self.n[b]), int(self.row0[b])
            if u in skip_units:
                continue
            mine[r0:r0 + n] = True
            t = np.array([x for k in self.sel[u] for x in range(k * self.g[u], min((k + 1) * self.g[u], c.lens[b]))], int)
            for i in range(n):
                js = [j for j in range(n) if int(self.mask[r0 + i]) >> j & 1]
                new = self.kv_np[r0:r0 + n].astype(np.float64)
                K, V = np.concatenate([c.K[u][t], new[js, 0, h]]), np.concatenate([c.V[u][t], new[js, 1, h]])
                for g in range(c.G):
                    want = R.attend_row(self.q_np[r0 + i, h * c.G + g].astype(np.float64), K, V)
                    R.check_row(out[r0 + i, h * c.G + g], z[r0 + i, h * c.G + g], want, (b, h, i, g))
        if not skip_units:
            assert (out[~mine] == 7.0).all() and (z[~mine] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n,lens,g", [(4, [1], [1], 16), (4, [8], [333], 32), (7, [20, 0, 64], [100, 50, 17], 48),
                                        (8, [64], [400], 16), (1, [33, 5], [129, 128], 128), (2, [3, 64], [700, 15], [16, 64, 128, 32])])
def test_tree_random_selections(kind, d, G, n, lens, g):
    c = R.Cache(len(n), 2, G, d, lens, kind, seed=sum(lens), max_gather_pages_per_unit=64)
    for sel in ("some", "all"):
        t = Tree(c, n, g=g, sel=sel)
        t.run()
        assert _sync_status(c) == 0
        t.check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_tree_rows_that_see_nothing(kind):
    """Masks without a bit over no selection: zeros and -inf; with drafts' NaN out of sight."""
    c = R.Cache(2, 1, 4, 64, [50, 0], kind)
    t = Tree(c, [6, 9], sel="none", masks=lambda i, rng: 0 if i % 2 else 1 << i)
    t.kv[t.row0[0] + 1] = float("nan")            # a draft that nobody sees
    t.kv[t.row0[1] + 3] = float("inf")
    t.run()
    assert _sync_status(c) == 0
    t.check()
    rows = t.out[t.row0[0] + 1].float()
    assert (rows == 0).all() and torch.isneginf(t.lse[t.row0[0] + 1]).all()


def test_tree_bits_past_the_drafts_do_not_count():
    c = R.Cache(2, 2, 4, 64, [40, 90], "bf16")
    t = Tree(c, [5, 17], masks=lambda i, rng: (1 << 64) - 1)
    t.run()
    assert _sync_status(c) == 0
    want = t.mask.copy()
    for b in range(2):
        t.mask[t.row0[b]:t.row0[b] + t.n[b]] &= np.uint64((1 << int(t.n[b])) - 1)
    t.check()
    assert (want != t.mask).any()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_tree_splits(kind):
    c = R.Cache(1, 2, 4, 128, [9000], kind, max_gather_pages_per_unit=576)   # (whole blocks)
    t = Tree(c, [40], g=64)
    assert B.tree_workspace_size(c.dims, 40) > 0
    t.run()
    assert _sync_status(c) == 0
    t.check()


def test_tree_refusals_on_the_device():
    for field, value, code in (("n_t", [5, 9], B.BS_ERR_INVALID_ARG), ("n_t", [5, -1], B.BS_ERR_INVALID_ARG),
                               ("begin", [2, 100], B.BS_ERR_DEVICE_BOUNDS), ("g_t", [16, 24], B.BS_ERR_INVALID_ARG),
                               ("g_t", [16, 0], B.BS_ERR_INVALID_ARG), ("cnt", [4, -1], B.BS_ERR_INVALID_ARG),
                               ("cnt", [4, 500], B.BS_ERR_CAPACITY), ("lists", 99, B.BS_ERR_DEVICE_BOUNDS),
                               ("lists", -3, B.BS_ERR_DEVICE_BOUNDS)):
        c = R.Cache(2, 1, 4, 64, [60, 60], "bf16")
        t = Tree(c, [5, 8])
        if field == "lists":
            t.lists[1, 1] = value
        else:
            getattr(t, field).copy_(i32(value))
        t.run()
        assert _sync_status(c) == code, field
        if field == "lists":                      # the block is left out
            t.sel[1] = [0, 2, 3]
            t.check()
        else:
            assert (t.out[t.row0[1]:t.row0[1] + 8] == 7.0).all(), field
            t.check(skip_units=(1,))


@pytest.mark.parametrize("batch,n", [(33, 3), (70, 40)])
def test_tree_many_units(batch, n):
    """More units than share a wave's CTAs, and as many as just do."""
    lens = [(37 * i) % 700 for i in range(batch)]
    c = R.Cache(batch, 1, 8, 64, lens, "bf16", max_gather_pages_per_unit=300)
    t = Tree(c, [(i * 7) % (n + 1) for i in range(batch)], g=16, sel="some")
    t.run()
    assert _sync_status(c) == 0
    t.check()


# ---------------------------------------------------------------------------------------
# Commit
# ---------------------------------------------------------------------------------------
def _commit_inputs(c, n, acc, act, rng):
    rows = c.B * n + 1
    x = torch.as_tensor((rng.standard_normal((rows, 2 * c.Hkv * c.d)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32))
    path = np.full((c.B, max(1, max(acc))), 10 ** 6, np.int32)      # (past the accepted ones: not read)
    for b in range(c.B):
        path[b, :acc[b]] = np.sort(rng.choice(n, size=acc[b], replace=False))
    return x.to(R.CODE[act]).cuda(), path, 1 + np.arange(c.B) * n


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3", "int8"])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("d,n,acc,old", [(64, 8, [3, 0, 1], [5, 16, 31]), (128, 64, [64, 17, 2], [0, 15, 33])])
def test_commit_is_an_append_of_the_path(kind, act, d, n, acc, old):
    rng = np.random.default_rng(n)
    lens = np.array(old) + np.array(acc)
    c = R.Cache(3, 2, 4, d, lens, kind, q_dtype=R.KIND[act])
    x, path, row0 = _commit_inputs(c, n, acc, act, rng)
    kn, vn = x[:, :2 * d], x[:, 2 * d:]
    k0, v0 = c.k.clone(), c.v.clone()
    ks0, vs0 = (None if t is None else t.clone() for t in (c.ks, c.vs))
    B.tree_commit(c.dims, c.pools(), c.table, c.seq_lens, i32(old), i32(row0), i32(path), path.shape[1], kn, vn, x.stride(0),
                  x.shape[0], c.status)
    assert _sync_status(c) == 0
    flat = np.concatenate([row0[b] + path[b, :acc[b]] for b in range(3)])
    packed = x[torch.as_tensor(flat).cuda().long()]
    if kind in ("e4m3", "int8"):                  # the same bits as bs_quant_append of the path's rows
        got = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs)]
        c.k.view(torch.uint8).copy_(k0.view(torch.uint8))
        c.v.view(torch.uint8).copy_(v0.view(torch.uint8))
        c.ks.copy_(ks0)
        c.vs.copy_(vs0)
        B.quant_append(c.dims, c.pools(), c.table, c.seq_lens, i32(old), i32(np.cumsum(acc) - acc), packed[:, :2 * d],
                       packed[:, 2 * d:], packed.stride(0), len(flat), max(acc), c.status)
        assert _sync_status(c) == 0
        want = [c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs]
        for a, b in zip(got, want):
            assert torch.equal(torch.nan_to_num(a.float(), nan=-1.0), torch.nan_to_num(b.float(), nan=-1.0))
        return
    at = 0
    for b in range(3):
        for i in range(acc[b]):
            t = old[b] + i
            for h in range(2):
                ph = c.table_np[b * 2 + h, t // 16]
                k0[ph, t % 16] = packed[at, h * d:(h + 1) * d].to(k0.dtype)
                v0[ph, t % 16] = packed[at, (2 + h) * d:(3 + h) * d].to(v0.dtype)
            at += 1
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), nan=-9.0), torch.nan_to_num(b.float(), nan=-9.0))  # noqa: E731
    assert same(k0, c.k) and same(v0, c.v)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad,code", [("node", B.BS_ERR_DEVICE_BOUNDS), ("negative", B.BS_ERR_DEVICE_BOUNDS),
                                      ("row", B.BS_ERR_DEVICE_BOUNDS), ("long", B.BS_ERR_CAPACITY),
                                      ("begin", B.BS_ERR_INVALID_ARG), ("pages", B.BS_ERR_CAPACITY),
                                      ("page", B.BS_ERR_DEVICE_BOUNDS)])
def test_commit_skips_what_does_not_fit(kind, bad, code):
    c = R.Cache(2, 1, 4, 64, [20, 20], kind)
    x, path, row0 = _commit_inputs(c, 8, [4, 4], "bf16", np.random.default_rng(3))
    old = [16, 16]
    if bad == "node":
        path[1, 3] = 10 ** 8
    elif bad == "negative":
        path[1, 0] = -1
    elif bad == "row":
        row0[1] = -1
    elif bad == "long":
        c.seq_lens.copy_(i32([20, 25]))
    elif bad == "begin":
        old = [16, 21]
    elif bad == "pages":
        c.seq_lens.copy_(i32([20, 33]))
        old = [16, 31]
    elif bad == "page":
        c.table[1, 1] = -5
    before = c.k.clone()
    B.tree_commit(c.dims, c.pools(), c.table, c.seq_lens, i32(old), i32(row0), i32(path), 4, x[:, :64], x[:, 64:], x.stride(0),
                  x.shape[0], c.status)
    assert _sync_status(c) == code
    raw = lambda t: t.view(torch.uint8 if kind == "e4m3" else torch.int16)  # noqa: E731
    mine = c.table_np[0, 1]
    changed = (raw(before) != raw(c.k)).flatten(1).any(1).cpu()
    assert changed[mine] and changed.sum() == 1


# ---------------------------------------------------------------------------------------
# Streams, graphs, and a run of them together
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("kv8", [None, "e4m3"])
def test_layer_attends_prompts_and_drafts(kv8):
    """PagedLayer's own calls: a whole prompt against the float64 form over its logical K and V, then
    drafts over the layer's selection, then their commit."""
    from workloads import make_workload
    from long_context_serving_gb300.layer import PagedLayer

    wl = make_workload(2, seed=3, T=700)
    layer = PagedLayer(wl, kv8=kv8)
    layer.prefill()
    layer.append(0)
    layer.fused_step(0)                           # the selection that drafts attend
    T = int(wl.T_prefill[0])
    rng = np.random.default_rng(5)
    lo, hi = np.array([T - 90]), np.array([T])
    q = torch.as_tensor(R.bf16(rng.standard_normal((90, wl.Hq, wl.d)))).cuda().bfloat16()
    out, lse = layer.prefill_attend(q, lo, hi)
    if kv8 is None:                               # (8-bit values: the other tests')
        for i, u in itertools.product((0, 40, 89), (0, 5)):
            K, V = (x.astype(np.float64) for x in (wl.K64(u)[:T], wl.V64(u)[:T]))
            s = R.prefill_seen(T - 90 + i, T, wl.cls[u] == B.BS_STREAMING, int(wl.sink[u]), int(wl.local[u]))
            want = R.attend_row(q[i, u * wl.G].double().cpu().numpy(), K[s], V[s])
            R.check_row(out[i, u * wl.G].double().cpu().numpy(), float(lse[i, u * wl.G]), want, (i, u))
    n = 5
    kv = torch.as_tensor(R.bf16(rng.standard_normal((n, 2 * wl.Hkv * wl.d)))).cuda().bfloat16()
    visible = torch.tensor([(1 << (i + 1)) - 1 for i in range(n)], dtype=torch.int64, device="cuda")   # a chain
    lens = np.array([T + 1])
    d_out, d_lse = layer.draft_attend(q[:n].contiguous(), kv[:, :wl.Hkv * wl.d], kv[:, wl.Hkv * wl.d:], [n], visible, lens)
    assert layer.read_status() == 0 and torch.isfinite(d_out.float()).all() and torch.isfinite(d_lse).all()
    if T + 3 <= wl.page_table.shape[1] * 16:
        layer.commit_drafts(kv[:, :wl.Hkv * wl.d], kv[:, wl.Hkv * wl.d:], [n], np.array([[0, 1]]), lens)
        assert layer.read_status() == 0
        ph = int(layer.page_table[0, (T + 1) // 16])
        if kv8 is None:
            assert torch.equal(layer.k_pool[ph, (T + 1) % 16], kv[0, :wl.d])


def test_other_streams_and_graphs():
    """On a stream of the caller's, and captured once and replayed over new inputs; two captured graphs
    with a workspace each replay side by side."""
    c = R.Cache(1, 2, 4, 128, [3000], "bf16", max_gather_pages_per_unit=192)
    p, t = Prefill(c, [5]), Tree(c, [7], g=32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.run(stream=s)
    t.run(stream=s)
    s.synchronize()
    assert int(c.status.item()) == 0
    p.check()
    t.check()
    graphs = []
    for x in (p, t):
        x.out.fill_(7.0)
        x.lse.fill_(7.0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for rep in range(2):
        for x in (p, t):
            x.q_np = R.bf16(np.random.default_rng(50 + rep).standard_normal(x.q_np.shape))
            x.q.copy_(torch.as_tensor(x.q_np.reshape(x.rows, -1)).cuda())
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        p.check()
        t.check()


def test_batch_does_not_change_a_sequence():
    """With the same bounds, a sequence's rows are bitwise the same whatever the others hold."""
    outs = []
    for other in (10, 500):
        c = R.Cache(2, 2, 4, 64, [300, 500], "bf16", seed=5)
        p = Prefill(c, [30, 30])
        c.seq_lens.copy_(i32([300, other]))
        p.old.copy_(i32([270, other - 10]))
        p.run()
        assert _sync_status(c) == 0
        outs.append(p.out[p.row0[0]:p.row0[0] + 30].clone())
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_prompt_then_drafts_then_their_commit(kind):
    """As a serving loop uses them: a prompt is rotated into the cache and attended; a selection is
    made; drafts are rotated, attended outside the cache, the accepted ones committed. The branch that
    was accepted then stands in the cache as if it had come token by token: attended as new tokens of
    dense heads it gives what the tree gave over a full selection."""
    rng = np.random.default_rng(11)
    Bn, Hq, Hkv, d, prompt, n = 2, 8, 2, 128, [75, 130], 6
    total = [x + 4 for x in prompt]
    act, dev = torch.bfloat16, "cuda"
    c = R.Cache(Bn, Hkv, Hq // Hkv, d, total, kind)
    for b in range(Bn):                           # the values that an append would have left: none yet
        for h in range(Hkv):
            c.K[b * Hkv + h] = c.V[b * Hkv + h] = None
    freq = torch.as_tensor(10000.0 ** (-2.0 * np.arange(d // 2) / d), device=dev)
    wq = torch.as_tensor(1 + 0.1 * rng.standard_normal(d), dtype=torch.float32, device=dev)
    rope = B.Rope(inv_freq=freq.data_ptr(), rot_dim=d, interleaved=0, magnitude=1.0, q_weight=wq.data_ptr(),
                  k_weight=wq.data_ptr(), eps=1e-6)
    one = lambda m, x: torch.as_tensor(np.asarray(x), dtype=m, device=dev)  # noqa: E731

    def rows(k):
        return torch.as_tensor(rng.standard_normal((k, (Hq + 2 * Hkv) * d)).astype(np.float32)).to(act).to(dev)

    def rotate(x, pos, seq, cache):
        q = torch.empty((x.shape[0], Hq, d), dtype=act, device=dev)
        k = torch.empty((x.shape[0], Hkv, d), dtype=act, device=dev)
        B.rope_append(c.dims, rope, x, x[:, Hq * d:], x[:, (Hq + Hkv) * d:], x.stride(0), x.shape[0], i32(pos), i32(seq),
                      c.pools() if cache else None, c.table if cache else None, q, k, c.status)
        return q, k

    def attend(q, lens, new, row0):
        c.seq_lens.copy_(i32(lens))
        out = torch.zeros((q.shape[0], Hq, d), dtype=act, device=dev)
        lse = torch.zeros((q.shape[0], Hq), device=dev)
        size = B.prefill_workspace_size(c.dims, q.shape[0], int(max(new)))
        ws = torch.zeros(max(16, size), dtype=torch.uint8, device=dev)
        B.prefill_attn(c.dims, q, Hq * d, q.shape[0], c.kv(), cfg, i32(np.array(lens) - new), i32(row0), int(max(new)), out, lse,
                       ws, c.status)
        return out, lse

    U = Bn * Hkv
    cls, sink, local, g = i32(np.full(U, 1)), i32(np.zeros(U)), i32(np.ones(U)), i32(np.full(U, 16))
    cfg = B.HeadCfg(cls=cls.data_ptr(), sink_tokens=sink.data_ptr(), local_tokens=local.data_ptr(), block_tokens=g.data_ptr())
    # the prompt
    x = rows(sum(prompt))
    pos = np.concatenate([np.arange(k) for k in prompt])
    seq = np.repeat(np.arange(Bn), prompt)
    row0 = np.cumsum(prompt) - prompt
    q, k = rotate(x, pos, seq, kind == "bf16")
    if kind != "bf16":
        B.quant_append(c.dims, c.pools(), c.table, i32(prompt), i32([0] * Bn), i32(row0), k.view(-1, Hkv * d),
                       x[:, (Hq + Hkv) * d:].contiguous(), Hkv * d, sum(prompt), max(prompt), c.status)
    out, _ = attend(q, prompt, np.array(prompt), row0)
    assert _sync_status(c) == 0 and torch.isfinite(out.float()).all()
    # drafts: node 0, its children 1 and 2, 1's child 3, 3's child 4, 2's child 5
    parent, depth = [-1, 0, 0, 1, 3, 2], [0, 1, 1, 2, 3, 2]
    see = []
    for i in range(n):
        see.append(1 << i | (see[parent[i]] if parent[i] >= 0 else 0))
    y = rows(Bn * n)
    dpos = np.concatenate([p + np.array(depth) for p in prompt])
    dq, dk = rotate(y, dpos, np.repeat(np.arange(Bn), n), False)
    dkv = torch.cat([dk.view(Bn * n, -1), y[:, (Hq + Hkv) * d:]], 1).contiguous()
    sel = torch.arange(c.dims.max_sel_per_unit, dtype=torch.int32, device=dev).repeat(U, 1).contiguous()
    cnt = i32(np.repeat([-(-p // 16) for p in prompt], Hkv))
    c.seq_lens.copy_(i32(prompt))
    vis, n_t, begin = one(torch.int64, see * Bn), i32([n] * Bn), i32([0, n])
    drafts = B.Drafts(k_new=dkv.data_ptr(), v_new=dkv[:, Hkv * d:].data_ptr(), row_stride=dkv.stride(0), n_rows=Bn * n,
                      row_begin=begin.data_ptr(), n_draft=n_t.data_ptr(), visible=vis.data_ptr(), max_draft=n)
    t_out = torch.zeros((Bn * n, Hq, d), dtype=act, device=dev)
    t_lse = torch.zeros((Bn * n, Hq), device=dev)
    ws = torch.zeros(max(16, B.tree_workspace_size(c.dims, n)), dtype=torch.uint8, device=dev)
    B.tree_decode_attn(c.dims, dq, Hq * d, c.kv(), cfg, sel, cnt, drafts, t_out, t_lse, ws, c.status)
    # the branch 0, 1, 3, 4 is accepted
    path = np.array([[0, 1, 3, 4]] * Bn)
    after = i32(total)
    B.tree_commit(c.dims, c.pools(), c.table, after, i32(prompt), begin, i32(path), 4, dkv, dkv[:, Hkv * d:], dkv.stride(0),
                  Bn * n, c.status)
    pick = torch.as_tensor(np.concatenate([b * n + path[b] for b in range(Bn)]), device=dev)
    out, lse = attend(dq[pick].contiguous(), total, np.array([4, 4]), [0, 4])
    assert _sync_status(c) == 0
    # Two results of bf16 weights and one rounding each; an 8-bit cache has rounded the drafts too
    # (E4M3: half a step is 2^-4 of a value, on the few new keys among many).
    a, b = out.double(), t_out[pick].double()
    tol = 4 * R.HALF_BF16 * 2 if kind == "bf16" else 0.25
    assert (a - b).abs().max() <= tol * max(1.0, float(b.abs().max()))
    if kind == "bf16":
        assert (lse - t_lse[pick]).abs().max() <= 1e-3
