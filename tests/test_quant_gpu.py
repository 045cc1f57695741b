"""8-bit caches on the GPU, through the C ABI: the quantising append code by code against
the plain form, attention and sub-block means against float64 over the dequantised values,
the fused decode step, and both under a captured graph.

Attention bound, derived: codes are exact in fp16; q enters within 2^-22 of itself; a dot
product of D terms accumulated in fp32 (each add within 2^-23, the tensor core truncating)
and its scaling are within (D 2^-23 + 2^-21) A of x, A = max_t sum_i |q_i K_ti| / sqrt(d), so
every weight is within that relative error, numerator and denominator each: 2 (...) A Vmax on
the output; the sums over N pages add N 2^-23 and P's rounding, exp2 and the merges 2^-19.
"""
import numpy as np
import pytest
import torch

import _quant as Q
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build
from long_context_serving_gb300.layer import PagedLayer
from oracle import bsattn_oracle as O
from workloads import make_workload

pytestmark = pytest.mark.gpu
KINDS = {"e4m3": (B.BS_E4M3, torch.float8_e4m3fn), "int8": (B.BS_INT8, torch.int8)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build()
    B.lib()


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


class Cache:
    """A random 8-bit cache: B sequences of the given lengths, pages of a shuffled pool. Slots
    past a sequence's end hold NaN codes (E4M3) and pages of nobody a NaN scale."""

    def __init__(self, lens, Hkv, d, kind, rng, G=1, q32=False, extra=3, cap=0, odd_scales=False):
        self.kind, self.d, self.Hkv, self.B, self.G = kind, d, Hkv, len(lens), G
        self.lens = np.asarray(lens, np.int64)
        U = self.B * Hkv
        self.T = np.repeat(self.lens, Hkv)
        pages = -(-np.maximum(self.T, cap) // 16)
        self.P = max(1, int(pages.max()))
        self.n_pages = int(pages.sum()) + extra
        perm = rng.permutation(self.n_pages)
        self.table = np.full((U, self.P), -1, np.int64)
        at = 0
        for u in range(U):
            self.table[u, :pages[u]] = perm[at:at + pages[u]]
            at += pages[u]
        self.pools = {}
        for s in "kv":
            n_base = min(self.n_pages, 300)           # (large pools repeat pages, under scales of their own)
            x = rng.normal(size=(n_base, 16, d)).astype(np.float32)
            sc = np.exp(rng.normal(size=self.n_pages)).astype(np.float32)
            if not odd_scales and kind == "e4m3":
                sc = np.exp2(np.rint(np.log2(sc))).astype(np.float32)
            top = 448.0 if kind == "e4m3" else 127.0
            codes = Q.round_half_even(x / np.abs(x).max((1, 2), keepdims=True) * top, kind)
            if n_base < self.n_pages:
                codes = codes[rng.integers(0, n_base, self.n_pages)]
            self.pools[s] = [codes, (sc * np.float32(4 / top)).astype(np.float32)]
        if kind == "e4m3":
            owned = np.zeros(self.n_pages, bool)
            for u in range(U):
                n = -(-self.T[u] // 16)
                owned[self.table[u, :n]] = True
                if self.T[u] % 16:
                    for s in "kv":
                        self.pools[s][0][self.table[u, n - 1], self.T[u] % 16:] = 0x7F
            for s in "kv":
                self.pools[s][1][~owned] = np.nan
        code, dt = KINDS[kind]
        self.k, self.v = (torch.as_tensor(self.pools[s][0], device="cuda") for s in "kv")
        self.ks, self.vs = (torch.as_tensor(self.pools[s][1], device="cuda") for s in "kv")
        self.t_table, self.t_lens = i32(self.table), i32(self.lens)
        self.q32 = q32
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = B.Dims(batch=self.B, n_q_heads=G * Hkv, n_kv_heads=Hkv, head_dim=d, page_size=16,
                           max_pages_per_unit=self.P, max_blocks_per_unit=1, max_sel_per_unit=1, max_subs_per_unit=1,
                           max_gather_pages_per_unit=1, n_pages=self.n_pages, kv_dtype=code,
                           q_dtype=B.BS_FP32 if q32 else B.BS_BF16)
        self.kv = B.KV(k_pool=self.k.data_ptr(), v_pool=self.v.data_ptr(), page_table=self.t_table.data_ptr(),
                       seq_lens=self.t_lens.data_ptr(), k_scale=self.ks.data_ptr(), v_scale=self.vs.data_ptr())
        self.pool_ptrs = B.Pools(k_pool=self.k.data_ptr(), v_pool=self.v.data_ptr(), k_scale=self.ks.data_ptr(),
                                 v_scale=self.vs.data_ptr())

    def unit(self, u):
        """K and V of unit u in float64."""
        return tuple(Q.dequant_unit(u8(p), s.cpu().numpy(), self.table[u], int(self.T[u]), self.kind)
                     for p, s in ((self.k, self.ks), (self.v, self.vs)))


# ----------------------------------------------------------------------------------
# Append
# ----------------------------------------------------------------------------------
def append_and_compare(rng, kind, d, q32, Hkv, old, new, pad=0, values=None, odd_scales=False):
    old, new = np.asarray(old), np.asarray(new)
    c = Cache(old, Hkv, d, kind, rng, q32=q32, cap=int((old + new).max()), odd_scales=odd_scales)
    n = int(new.sum())
    stride = 2 * Hkv * d + pad
    x = rng.normal(size=(n + 2, stride)).astype(np.float32) * np.exp(2 * rng.normal(size=(n + 2, 1))).astype(np.float32)
    if values is not None:
        values(x)
    t = torch.as_tensor(x, device="cuda")
    if not q32:
        t = t.bfloat16()
    x = t.float().cpu().numpy()
    row0 = np.cumsum(new) - new + 1                       # the first row is nobody's
    order = rng.permutation(len(new))                     # sequences' rows in any order
    row0 = np.empty(len(new), np.int64)
    at = 1
    for b in order:
        row0[b], at = at, at + new[b]
    kn, vn = t[:, :Hkv * d], t[:, Hkv * d:2 * Hkv * d]
    B.quant_append(c.dims, c.pool_ptrs, c.t_table, i32(old + new), i32(old), i32(row0), kn, vn, stride, n + 2,
                   max(int(new.max()), 1), c.status)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    for s, pool, scale, off in (("k", c.k, c.ks, 0), ("v", c.v, c.vs, Hkv * d)):
        codes, sc = c.pools[s][0].copy(), c.pools[s][1].copy()
        for b in range(len(new)):
            for h in range(Hkv):
                rows = x[row0[b]:row0[b] + new[b], off + h * d:off + (h + 1) * d]
                t0 = int(old[b])
                while len(rows):
                    ph, kept = c.table[b * Hkv + h, t0 // 16], t0 % 16
                    take = min(len(rows), 16 - kept)
                    codes[ph], sc[ph] = Q.append_page(codes[ph], sc[ph], kept, rows[:take], kind)
                    rows, t0 = rows[take:], t0 + take
        got = u8(pool)
        assert np.array_equal(scale.cpu().numpy(), sc, equal_nan=True), s
        if kind == "int8":
            assert np.array_equal(got, codes), s
        else:
            assert Q.same_codes(got, codes, kind), s


APPENDS = {"one-token": ([0, 1, 15, 16, 17, 31], [1, 1, 1, 1, 1, 1]),
           "nothing-for-some": ([0, 7, 32], [0, 3, 0]),
           "prompts": ([0, 0, 5, 16], [1, 33, 200, 16]),
           "across-pages": ([3, 14, 0], [50, 2, 47])}


@pytest.mark.parametrize("q32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("name", sorted(APPENDS))
def test_append_codes_equal_the_plain_form(name, kind, d, q32):
    old, new = APPENDS[name]
    append_and_compare(np.random.default_rng(len(name) + d), kind, d, q32, 3, old, new)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_row_stride_and_foreign_scales(kind):
    """Rows wider than K and V, and pages filled elsewhere with scales that are no powers of two."""
    append_and_compare(np.random.default_rng(5), kind, 128, False, 2, [5, 9, 30], [4, 40, 1], pad=72, odd_scales=True)


def special(x):
    x[1] = 0                                                     # a token of zeros
    x[2, ::7] = np.inf
    x[3, ::5] = -np.inf
    x[4, ::3] = np.nan
    x[5] = 2.0 ** -130                                           # subnormal as fp32, zero as bf16 or not
    x[6] = 3e38
    x[7:30] = 0
    x[30:31, 0] = 1e-30


@pytest.mark.parametrize("q32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_special_values(kind, q32):
    for old, new in (([0, 0], [1, 31]), ([4, 9], [20, 30]), ([0] * 8, [1] * 8)):
        append_and_compare(np.random.default_rng(6), kind, 64, q32, 1, old, new, values=special)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_token_by_token_rounds_pages_again(kind):
    """Forty single-token appends of growing values: each step equals the plain form."""
    rng = np.random.default_rng(8)
    c = Cache([0], 2, 64, kind, rng, cap=48)
    codes, sc = {s: c.pools[s][0].copy() for s in "kv"}, {s: c.pools[s][1].copy() for s in "kv"}
    for t in range(40):
        x = torch.as_tensor(rng.normal(size=(1, 256)) * 1.3 ** t, device="cuda").bfloat16()
        B.quant_append(c.dims, c.pool_ptrs, c.t_table, i32([t + 1]), i32([t]), i32([0]), x[:, :128], x[:, 128:], 256, 1,
                       1, c.status)
        xs = x.float().cpu().numpy()
        for s, pool, scale, off in (("k", c.k, c.ks, 0), ("v", c.v, c.vs, 128)):
            for h in range(2):
                ph = c.table[h, t // 16]
                codes[s][ph], sc[s][ph] = Q.append_page(codes[s][ph], sc[s][ph], t % 16,
                                                        xs[:, off + 64 * h:off + 64 * (h + 1)], kind)
            assert Q.same_codes(u8(pool), codes[s], kind) and np.array_equal(scale.cpu().numpy(), sc[s], equal_nan=True), (t, s)
    assert int(c.status) == 0


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_after_a_page_of_zeros(kind):
    """A page whose scale is 0 takes real values: its zeros stay zeros."""
    rng = np.random.default_rng(10)
    c = Cache([0], 1, 128, kind, rng, cap=16)
    codes, sc = {s: c.pools[s][0].copy() for s in "kv"}, {s: c.pools[s][1].copy() for s in "kv"}
    for t, x in enumerate((torch.zeros((1, 256)), torch.zeros((1, 256)), torch.randn((1, 256)), torch.zeros((1, 256)))):
        x = x.cuda().bfloat16()
        B.quant_append(c.dims, c.pool_ptrs, c.t_table, i32([t + 1]), i32([t]), i32([0]), x[:, :128], x[:, 128:], 256, 1,
                       1, c.status)
        xs, ph = x.float().cpu().numpy(), c.table[0, 0]
        for s, pool, scale, off in (("k", c.k, c.ks, 0), ("v", c.v, c.vs, 128)):
            codes[s][ph], sc[s][ph] = Q.append_page(codes[s][ph], sc[s][ph], t, xs[:, off:off + 128], kind)
            assert Q.same_codes(u8(pool), codes[s], kind) and np.array_equal(scale.cpu().numpy(), sc[s], equal_nan=True)
    assert int(c.status) == 0 and sc["k"][c.table[0, 0]] > 0


def test_append_takes_more_tokens_than_the_grid_was_sized_for():
    """max_new_tokens sizes the grid only."""
    rng = np.random.default_rng(12)
    c = Cache([5, 0], 2, 64, "int8", rng, cap=400)
    x = torch.as_tensor(rng.normal(size=(700, 256)), device="cuda").bfloat16()
    both = []
    for max_new in (350, 1):
        k, v, ks, vs = c.k.clone(), c.v.clone(), c.ks.clone(), c.vs.clone()
        pools = B.Pools(k_pool=k.data_ptr(), v_pool=v.data_ptr(), k_scale=ks.data_ptr(), v_scale=vs.data_ptr())
        B.quant_append(c.dims, pools, c.t_table, i32([355, 350]), i32([5, 0]), i32([0, 350]), x[:, :128], x[:, 128:], 256,
                       700, max_new, c.status)
        both.append((k, v, ks, vs))
    assert int(c.status) == 0 and all(torch.equal(a, b) for a, b in zip(*both)) and not torch.equal(both[0][0], c.k)


def test_append_skips_what_does_not_fit():
    """Each sequence's own fault is reported and the others are written."""
    rng = np.random.default_rng(9)
    for old, new, row0, rows, code in (([0, 4], [-3, 2], [0, 0], 2, B.BS_ERR_INVALID_ARG),      # lens below begin
                                       ([0, 4], [400, 2], [0, 0], 400, B.BS_ERR_CAPACITY),      # beyond the row
                                       ([0, 4], [3, 2], [-1, 0], 8, B.BS_ERR_DEVICE_BOUNDS),    # rows before the first
                                       ([0, 4], [3, 2], [6, 0], 8, B.BS_ERR_DEVICE_BOUNDS)):    # rows past the last
        c = Cache([16, 16], 1, 64, "int8", rng)
        x = torch.as_tensor(rng.normal(size=(max(rows, 8), 64)).astype(np.float32), device="cuda").bfloat16()
        B.quant_append(c.dims, c.pool_ptrs, c.t_table, i32(np.add(old, new)), i32(old), i32(row0), x, x, 64, rows, 400,
                       c.status)
        torch.cuda.synchronize()
        assert int(c.status) == code
        got = u8(c.k)
        want = c.pools["k"][0].copy()
        ph = c.table[1, 0]
        want[ph], _ = Q.append_page(want[ph], c.pools["k"][1][ph], 4, x[:2].float().cpu().numpy(), "int8")
        assert np.array_equal(got, want)
    for bad in (-1, 10 ** 6):                                                                    # a page outside the pool
        c = Cache([16, 16], 1, 64, "int8", rng)
        c.t_table[0, 0] = bad
        x = torch.ones((2, 64), device="cuda", dtype=torch.bfloat16)
        B.quant_append(c.dims, c.pool_ptrs, c.t_table, i32([1, 5]), i32([0, 4]), i32([0, 1]), x, x, 64, 2, 1, c.status)
        torch.cuda.synchronize()
        assert int(c.status) == B.BS_ERR_DEVICE_BOUNDS
        assert np.array_equal(np.delete(u8(c.k), c.table[1, 0], 0), np.delete(c.pools["k"][0], c.table[1, 0], 0))
        assert not np.array_equal(u8(c.k)[c.table[1, 0]], c.pools["k"][0][c.table[1, 0]])


# ----------------------------------------------------------------------------------
# Attention
# ----------------------------------------------------------------------------------
def bound(q, K, V, pages, d):
    """(out, lse) bounds of one head group; see the module's text."""
    A = float((np.abs(q) @ np.abs(K).T).max()) / np.sqrt(d) if len(K) else 0.0
    x = (d * 2.0 ** -23 + 2.0 ** -21) * A
    vmax = float(np.abs(V).max()) if len(V) else 0.0
    return (2 * x + pages * 2.0 ** -23 + 2.0 ** -19) * vmax, x + pages * 2.0 ** -23 + 2.0 ** -19 + A * 2.0 ** -22


def attend_and_compare(rng, kind, d, G, Hkv, lens, g, frac, q32=False, bias=False, noalloc=False, odd_scales=False,
                       q_scale=1.0, check_units=12, gather_cap=None, stream=None):
    c = Cache(lens, Hkv, d, kind, rng, G=G, q32=q32, odd_scales=odd_scales)
    U = c.B * Hkv
    gs = np.array([g[u % len(g)] for u in range(U)])
    n_blk = -(-c.T // gs)
    sels = []
    for u in range(U):
        nb = int(n_blk[u])
        pick = rng.permutation(nb - 1)[:int(frac * nb)] if nb > 1 else []
        sels.append(np.sort(np.concatenate([pick, [nb - 1]])).astype(np.int64) if nb else np.zeros(0, np.int64))
    S = max(1, max(len(s) for s in sels))
    sel = np.full((U, S), -1)
    for u in range(U):
        sel[u, :len(sels[u])] = sels[u]
    dims = c.dims
    dims.max_sel_per_unit, dims.max_blocks_per_unit = S, max(1, int(n_blk.max()))
    dims.max_gather_pages_per_unit = gather_cap or max(1, max(len(s) * gs[u] // 16 for u, s in enumerate(sels)))
    q = torch.as_tensor(rng.normal(size=(c.B, G * Hkv, d)).astype(np.float32) * np.float32(q_scale), device="cuda")
    q = q if q32 else q.bfloat16()
    e = None
    if bias:
        eb = rng.normal(size=(U, dims.max_blocks_per_unit)).astype(np.float32)
        eb[rng.random(eb.shape) < 0.2] = -np.inf
        if U > 1:
            eb[U // 2] = -np.inf                       # a unit with nothing left
        # dropped blocks hold NaN: nothing of them may count
        if kind == "e4m3":
            for u in range(U):
                for blk in np.flatnonzero(np.isneginf(eb[u, :n_blk[u]])):
                    ph = c.table[u, blk * gs[u] // 16:min((blk + 1) * gs[u] // 16, -(-c.T[u] // 16))]
                    c.k[torch.as_tensor(ph, device="cuda")] = 0x7F
                    c.vs[torch.as_tensor(ph, device="cuda")] = float("nan")
        e = torch.as_tensor(eb, device="cuda")
    cfg_g = i32(gs)
    cfg = B.HeadCfg(block_tokens=cfg_g.data_ptr())
    out = torch.full((c.B, G * Hkv, d), float("nan"), device="cuda")
    lse = torch.full((c.B, G * Hkv), float("nan"), device="cuda")
    ws = torch.zeros(B.workspace_size(dims) // 4, device="cuda")
    t_sel, t_cnt = i32(sel), i32([len(s) for s in sels])
    args = (dims, q, c.kv, cfg, t_sel, t_cnt, out, lse)
    torch.cuda.synchronize()
    B.sparse_decode_attn(*args, ws, c.status, stream, evict_bias=e)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    first, first_lse = out.clone(), lse.clone()
    if noalloc:
        out.zero_(), lse.zero_()
        B.sparse_decode_attn_noalloc(*args, c.status, evict_bias=e)
    else:
        B.sparse_decode_attn(*args, ws, c.status, stream, evict_bias=e)       # the workspace is ready again
    torch.cuda.synchronize()
    assert int(c.status) == 0 and torch.equal(out, first) and torch.equal(lse, first_lse)
    o, l = first.cpu().double().numpy(), first_lse.cpu().double().numpy()
    qf = q.double().cpu().numpy()
    units = range(U) if U <= check_units else sorted(set(rng.integers(0, U, check_units).tolist()) | {0, U // 2, U - 1})
    for u in units:
        b, h = divmod(u, Hkv)
        if len(sels[u]) == 0:
            continue
        t = O.selected_tokens(sels[u], int(gs[u]), int(c.T[u]))
        K, V = c.unit(u)
        if e is not None:
            t = t[~np.isneginf(eb[u, t // gs[u]])]
        K, V = K[t], V[t]
        x = qf[b, h * G:(h + 1) * G] @ K.T / np.sqrt(d)
        if e is not None:
            x = x + eb[u, t // gs[u]]
        to, tl = bound(qf[b, h * G:(h + 1) * G], K, V, len(sels[u]) * gs[u] / 16, d)
        if len(t) == 0:
            assert (o[b, h * G:(h + 1) * G] == 0).all() and np.isneginf(l[b, h * G:(h + 1) * G]).all()
            continue
        m = x.max(1, keepdims=True)
        p = np.exp(x - m)
        want, want_l = p @ V / p.sum(1, keepdims=True), m[:, 0] + np.log(p.sum(1))
        assert np.abs(o[b, h * G:(h + 1) * G] - want).max() <= to, (u, to)
        assert np.abs(l[b, h * G:(h + 1) * G] - want_l).max() <= tl, (u, tl)
        rel = np.linalg.norm(o[b, h * G:(h + 1) * G] - want) / np.linalg.norm(want)
        assert rel <= 1e-5, (u, rel)
    return o


PLANS = {  # name: (Hkv, lens, g, frac)
    "one-token": (1, [1], [64], 0.0),
    "tiny-ragged": (2, [1, 15, 16, 17, 33], [16, 32], 0.5),
    "cluster": (4, [3000, 2111], [32, 64], 0.3),
    "cluster-many-units": (8, [700 + 5 * i for i in range(40)], [64], 0.3),
    "workspace": (5, [9000 + 700 * i for i in range(5)], [16, 64, 128], 0.6),
    "workspace-long": (2, [20000, 17], [64], 0.95),
    "long-rows": (1, [12003], [16], 0.95),                            # more blocks than a CTA stages
    "many-pages-a-warp": (8, [2100 + 37 * i for i in range(40)], [64], 0.95),
    "most-pages-a-warp": (1, [130001], [64], 0.98),
}


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("plan", sorted(PLANS))
def test_attention_every_plan(plan, d, kind):
    Hkv, lens, g, frac = PLANS[plan]
    attend_and_compare(np.random.default_rng(11), kind, d, 4, Hkv, lens, g, frac)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("q32", [False, True], ids=["bf16", "fp32"])
def test_attention_group_sizes(G, q32):
    attend_and_compare(np.random.default_rng(G), "e4m3" if G % 2 else "int8", 128 if G < 5 else 64, G, 3, [517, 90], [48],
                       0.5, q32=q32)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("plan", ["tiny-ragged", "cluster", "workspace", "many-pages-a-warp"])
def test_attention_block_logits(plan, kind):
    """Random block logits; dropped blocks (-inf) hold NaN codes and scales; a unit drops whole."""
    Hkv, lens, g, frac = PLANS[plan]
    attend_and_compare(np.random.default_rng(13), kind, 128, 4, Hkv, lens, g, frac, bias=True)


@pytest.mark.parametrize("plan", ["cluster", "workspace-long"])
def test_attention_without_a_workspace_is_bitwise_equal(plan):
    Hkv, lens, g, frac = PLANS[plan]
    attend_and_compare(np.random.default_rng(14), "e4m3", 128, 7, Hkv, lens, g, frac, noalloc=True)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 1e25])
def test_attention_query_magnitudes(kind, q_scale):
    """Queries far from 1, as fp32: the row's power of two keeps them in fp16's range. (At 1e25
    one token takes all the weight: bounds as derived no longer mean anything, so the check
    there is that token's value.)"""
    rng = np.random.default_rng(15)
    if q_scale < 1e20:
        attend_and_compare(rng, kind, 128, 4, 2, [300, 41], [32], 0.9, q32=True, q_scale=q_scale)
        return
    c = Cache([40], 1, 128, kind, rng, q32=True)
    q = torch.as_tensor(rng.normal(size=(1, 1, 128)).astype(np.float32) * np.float32(q_scale), device="cuda")
    c.dims.max_sel_per_unit = c.dims.max_blocks_per_unit = 3
    c.dims.max_gather_pages_per_unit = 3
    out, lse = torch.zeros((1, 1, 128), device="cuda"), torch.zeros((1, 1), device="cuda")
    g, sel, cnt = i32([16]), i32([[0, 1, 2]]), i32([3])
    B.sparse_decode_attn(c.dims, q, c.kv, B.HeadCfg(block_tokens=g.data_ptr()), sel, cnt, out, lse,
                         torch.zeros(B.workspace_size(c.dims) // 4, device="cuda"), c.status)
    torch.cuda.synchronize()
    K, V = c.unit(0)
    top = int(np.argmax(q[0].double().cpu().numpy() @ K.T))
    assert int(c.status) == 0
    assert np.allclose(out[0, 0].cpu().numpy(), V[top], rtol=2.0 ** -20, atol=1e-6)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 60])
def test_attention_scales_far_from_one(scale):
    """V scales that fp16 could not hold: the output scales with them to the last bit."""
    rng = np.random.default_rng(16)
    c = Cache([100], 2, 64, "int8", rng, G=2)
    d = c.dims
    d.max_sel_per_unit = d.max_blocks_per_unit = 4
    d.max_gather_pages_per_unit = 8
    q = torch.as_tensor(rng.normal(size=(1, 4, 64)).astype(np.float32), device="cuda").bfloat16()
    g, sel, cnt = i32([32, 32]), i32([[0, 1, 2, 3]] * 2), i32([4, 4])
    ws = torch.zeros(B.workspace_size(d) // 4, device="cuda")
    outs = []
    for f in (1.0, scale):
        vs = c.vs * f
        kv = B.KV.from_buffer_copy(c.kv)
        kv.v_scale = vs.data_ptr()
        out, lse = torch.zeros((1, 4, 64), device="cuda"), torch.zeros((1, 4), device="cuda")
        B.sparse_decode_attn(d, q, kv, B.HeadCfg(block_tokens=g.data_ptr()), sel, cnt, out, lse, ws, c.status)
        torch.cuda.synchronize()
        outs.append(out)
    assert int(c.status) == 0 and torch.equal(outs[0] * scale, outs[1]) and outs[0].abs().max() > 0


def test_attention_odd_scales_and_side_stream():
    side = torch.cuda.Stream()
    attend_and_compare(np.random.default_rng(17), "e4m3", 128, 4, 2, [700, 90], [32], 0.7, odd_scales=True, stream=side)


def test_attention_bad_pages_and_counts_are_reported():
    """A page outside the pool, a block past the end, a count above the row: reported, the other
    units right, nothing read out of bounds."""
    rng = np.random.default_rng(18)
    for what in ("page", "block", "count"):
        c = Cache([64, 64], 1, 64, "int8", rng)
        d = c.dims
        d.max_sel_per_unit = d.max_blocks_per_unit = 4
        d.max_gather_pages_per_unit = 4
        sel, cnt = i32([[0, 1, 2, 3]] * 2), i32([4, 4])
        if what == "page":
            c.t_table[0, 1] = c.n_pages
        elif what == "block":
            sel[0, 3] = 7
        else:
            cnt[0] = 9
        q = torch.ones((2, 1, 64), device="cuda", dtype=torch.bfloat16)
        out, lse = torch.zeros((2, 1, 64), device="cuda"), torch.zeros((2, 1), device="cuda")
        g = i32([16, 16])
        B.sparse_decode_attn(d, q, c.kv, B.HeadCfg(block_tokens=g.data_ptr()), sel, cnt, out, lse,
                             torch.zeros(B.workspace_size(d) // 4, device="cuda"), c.status)
        torch.cuda.synchronize()
        assert int(c.status) in (B.BS_ERR_DEVICE_BOUNDS, B.BS_ERR_INVALID_ARG)
        K, V = c.unit(1)
        want, _ = O.sparse_attention(np.ones((1, 64)), K, V, [0, 1, 2, 3], 16, 64)
        assert np.abs(out[1].cpu().numpy() - want).max() <= 1e-4


def test_attention_selection_beyond_the_dims_is_refused_whole():
    """Workspace plan: a unit that selects more pages than max_gather_pages_per_unit allows for is
    reported and gets zeros; the others are right, and so is the next call on the workspace."""
    rng = np.random.default_rng(21)
    c = Cache([12000] + [1000] * 23, 1, 64, "int8", rng, G=2)
    d = c.dims
    nb = -(-c.T // 32)
    d.max_sel_per_unit = d.max_blocks_per_unit = int(nb.max())
    d.max_gather_pages_per_unit = 300                      # unit 0 selects 750 pages
    sel, g, cnt = i32(np.where(np.arange(nb.max()) < nb[:, None], np.arange(nb.max()), -1)), i32([32] * 24), i32(nb)
    q = torch.as_tensor(rng.normal(size=(24, 2, 64)), device="cuda").bfloat16()
    out, lse = torch.ones((24, 2, 64), device="cuda"), torch.ones((24, 2), device="cuda")
    ws = torch.zeros(B.workspace_size(d) // 4, device="cuda")
    K, V = c.unit(5)
    want, _ = O.sparse_attention(q[5].double().cpu().numpy(), K, V, list(range(nb[5])), 32, 1000)
    first = O.sparse_attention(q[0].double().cpu().numpy(), *c.unit(0), [0, 1, 9], 32, 12000)[0]
    for k in range(3):
        c.status.zero_()
        if k == 2:                                         # now within the dims
            cnt[0] = 3
            sel[0, :3] = i32([0, 1, 9])
        B.sparse_decode_attn(d, q, c.kv, B.HeadCfg(block_tokens=g.data_ptr()), sel, cnt, out, lse, ws, c.status)
        torch.cuda.synchronize()
        assert int(c.status) == (B.BS_ERR_DEVICE_BOUNDS if k < 2 else 0)
        assert np.abs(out[5].cpu().numpy() - want).max() <= 1e-4
        assert (out[0] == 0).all() if k < 2 else np.abs(out[0].cpu().numpy() - first).max() <= 1e-4
        assert torch.equal(ws.view(torch.int32)[:48], torch.zeros(48, dtype=torch.int32, device="cuda"))   # tickets


def test_attention_in_a_captured_graph():
    """Captured once, replayed over new queries, codes and lengths."""
    rng = np.random.default_rng(19)
    c = Cache([500, 300], 2, 128, "e4m3", rng, G=4)
    d = c.dims
    d.max_sel_per_unit, d.max_blocks_per_unit, d.max_gather_pages_per_unit = 4, 16, 8
    q = torch.zeros((2, 8, 128), device="cuda", dtype=torch.bfloat16)
    g, sel, cnt = i32([32] * 4), i32([[0, 3, 5, 9]] * 4), i32([4] * 4)
    cfg = B.HeadCfg(block_tokens=g.data_ptr())
    out, lse = torch.zeros((2, 8, 128), device="cuda"), torch.zeros((2, 8), device="cuda")
    ws = torch.zeros(B.workspace_size(d) // 4, device="cuda")
    x = torch.zeros((2, 4 * 128), device="cuda", dtype=torch.bfloat16)
    lens, begin, row0 = i32([500, 300]), i32([499, 299]), i32([0, 1])

    def step(stream=None):
        B.quant_append(d, c.pool_ptrs, c.t_table, lens, begin, row0, x[:, :256], x[:, 256:], 512, 2, 1, c.status, stream)
        B.sparse_decode_attn(d, q, c.kv, cfg, sel, cnt, out, lse, ws, c.status, stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        q.copy_(torch.as_tensor(rng.normal(size=q.shape), device="cuda"))
        x.copy_(torch.as_tensor(rng.normal(size=x.shape), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for u in range(4):
            b, h = divmod(u, 2)
            K, V = c.unit(u)
            want, _ = O.sparse_attention(q[b, 4 * h:4 * h + 4].double().cpu().numpy(), K, V, [0, 3, 5, 9], 32, int(c.T[u]))
            assert np.abs(out[b, 4 * h:4 * h + 4].cpu().numpy() - want).max() <= 1e-4
    assert int(c.status) == 0


def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 bytes: append, attention, means and page copies at its far end."""
    n, d = (1 << 21) + 64, 128                        # 2 KB pages: 4.3 GB each of K and V
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    rng = np.random.default_rng(20)
    k, v = (torch.zeros((n, 16, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n, device="cuda") for _ in range(2))
    T, last = 50, n - 1
    table = i32([[last, last - 1, last - 2, last - 3]])
    dims = B.Dims(batch=1, n_q_heads=4, n_kv_heads=1, head_dim=d, page_size=16, max_pages_per_unit=4,
                  max_blocks_per_unit=2, max_sel_per_unit=2, max_subs_per_unit=4, max_gather_pages_per_unit=4, n_pages=n,
                  kv_dtype=B.BS_INT8, q_dtype=B.BS_BF16)
    status, lens = i32([0]), i32([T])
    pools = B.Pools(k_pool=k.data_ptr(), v_pool=v.data_ptr(), k_scale=ks.data_ptr(), v_scale=vs.data_ptr())
    x = torch.as_tensor(rng.normal(size=(T, 2 * d)), device="cuda").bfloat16()
    B.quant_append(dims, pools, table, lens, i32([0]), i32([0]), x[:, :d], x[:, d:], 2 * d, T, T, status)
    K, V = (np.concatenate([Q.decode(u8(p[last - j]), "int8") * float(s[last - j]) for j in range(4)])[:T]
            for p, s in ((k, ks), (v, vs)))
    xs = x.float().cpu().numpy()
    # INT8: within half a step, and the fp32 rounding of quotient and scale
    assert (np.abs(K - xs[:, :d]) <= np.abs(xs[:, :d]).max() / 127 * 0.5001).all()
    q = torch.as_tensor(rng.normal(size=(1, 4, d)), device="cuda").bfloat16()
    kv = B.KV(k_pool=k.data_ptr(), v_pool=v.data_ptr(), page_table=table.data_ptr(), seq_lens=lens.data_ptr(),
              k_scale=ks.data_ptr(), v_scale=vs.data_ptr())
    out, lse = torch.zeros((1, 4, d), device="cuda"), torch.zeros((1, 4), device="cuda")
    g = i32([32])
    ws = torch.zeros(B.workspace_size(dims) // 4, device="cuda")

    def attend(kv):
        B.sparse_decode_attn(dims, q, kv, B.HeadCfg(block_tokens=g.data_ptr()), i32([[0, 1]]), i32([2]), out, lse, ws,
                             status)
        torch.cuda.synchronize()
        want, _ = O.sparse_attention(q[0].double().cpu().numpy(), K, V, [0, 1], 32, T)
        assert np.abs(out[0].cpu().numpy() - want).max() <= 1e-4

    attend(kv)
    one = {n_: i32([v_]) for n_, v_ in dict(cls=1, bt=32, st=16, k=1, ke=0, sink=16, loc=16, rows=4).items()}
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    cfg = B.HeadCfg(cls=one["cls"].data_ptr(), block_tokens=one["bt"].data_ptr(), sub_tokens=one["st"].data_ptr(),
                    k_total=one["k"].data_ptr(), k_evict=one["ke"].data_ptr(), sink_tokens=one["sink"].data_ptr(),
                    local_tokens=one["loc"].data_ptr(), sum_off=off.data_ptr(), sum_rows=one["rows"].data_ptr())
    summ = torch.zeros(4 * d, device="cuda")
    B.build_block_summaries(dims, kv, cfg, i32([0]), T, summ, status)
    means = np.stack([K[16 * j:16 * (j + 1)].mean(0) for j in range(4)])
    assert np.abs(summ.view(4, d).cpu().numpy() - means).max() <= 1e-5
    # the four pages to the front, and attended there
    pairs, count = i32([[last - j, j] for j in range(4)]), i32([4])
    B.pages_copy(dims, pools, B.PageCopies(pairs=pairs.data_ptr(), count=count.data_ptr(), capacity=4), status)
    front = i32([[0, 1, 2, 3]])
    kv.page_table = front.data_ptr()
    k[last - 3:].zero_()
    attend(kv)
    assert int(status) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its own cache and workspace: bitwise those of one at a time."""
    rng = np.random.default_rng(22)
    jobs = []
    for Hkv, lens, kind in ((4, [9000, 8000], "e4m3"), (8, [3000] * 6, "int8")):
        c = Cache(lens, Hkv, 128, kind, rng, G=4)
        U, nb = c.B * Hkv, -(-max(lens) // 64)
        c.dims.max_sel_per_unit = c.dims.max_blocks_per_unit = nb
        c.dims.max_gather_pages_per_unit = 4 * nb
        sel = np.where(np.arange(nb) < -(-c.T[:, None] // 64), np.arange(nb), -1)
        job = dict(c=c, sel=i32(sel), cnt=i32((sel >= 0).sum(1)), g=i32([64] * U), s=torch.cuda.Stream(),
                   q=torch.as_tensor(rng.normal(size=(c.B, 4 * Hkv, 128)), device="cuda").bfloat16(),
                   ws=torch.zeros(B.workspace_size(c.dims) // 4, device="cuda"),
                   out=torch.zeros((c.B, 4 * Hkv, 128), device="cuda"), lse=torch.zeros((c.B, 4 * Hkv), device="cuda"))
        job["cfg"] = B.HeadCfg(block_tokens=job["g"].data_ptr())
        jobs.append(job)

    def go(j, stream=None):
        B.sparse_decode_attn(j["c"].dims, j["q"], j["c"].kv, j["cfg"], j["sel"], j["cnt"], j["out"], j["lse"], j["ws"],
                             j["c"].status, stream)

    alone = []
    for j in jobs:
        go(j)
        torch.cuda.synchronize()
        alone.append((j["out"].clone(), j["lse"].clone()))
        j["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            go(j, j["s"])
    torch.cuda.synchronize()
    for j, (out, lse) in zip(jobs, alone):
        assert int(j["c"].status) == 0 and torch.equal(j["out"], out) and torch.equal(j["lse"], lse)


# ----------------------------------------------------------------------------------
# The decode loop over an 8-bit cache
# ----------------------------------------------------------------------------------
LOOPS = {"llama-T2900x4": (2, dict(T=2900, steps=4)), "mixed-g-T5000x3": (3, dict(B=1, T=5000, steps=3)),
         "ragged-batch": (4, dict(B=3, T=1700)), "dual-T900x6": (5, dict(B=3, T=900, steps=6)),
         "workspace-plan": (3, dict(B=4, T=20000, steps=2)), "fp32-d64": (1, dict(T=600))}


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("name", sorted(LOOPS))
def test_decode_loop(name, kind):
    """append -> fused step, and append -> the five calls, over the same 8-bit cache: the caches
    are equal, so are the selections (given their scores), and the attention of sampled units is
    that of the dequantised values; summaries equal a rebuild bit for bit."""
    cfg, kw = LOOPS[name]
    wl = make_workload(cfg, seed=31, **kw)
    fused, apart = PagedLayer(wl, kv8=kind), PagedLayer(wl, kv8=kind)
    fused.prefill()
    apart.prefill()
    rng = np.random.default_rng(1)
    for step in range(wl.steps):
        fused.append(step)
        apart.append(step)
        fused.fused_step(step)
        apart.step(step)
        torch.cuda.synchronize()
        assert fused.read_status() == 0 and apart.read_status() == 0
        assert torch.equal(fused.k_pool.view(torch.uint8), apart.k_pool.view(torch.uint8))
        assert torch.equal(fused.summaries.nan_to_num(), apart.summaries.nan_to_num())
        assert fused.selection(1 - fused.cur) == apart.selection(1 - apart.cur)
        assert torch.allclose(fused.lse, apart.lse, rtol=0, atol=1e-4)
        again = torch.full_like(fused.summaries, float("nan"))
        B.build_block_summaries(fused.dims, fused.kv_at(fused.seq_lens[step]), fused.cfg, fused.zeros_b,
                                int(wl.T_cap), again, fused.status)
        assert torch.equal(again.nan_to_num(), fused.summaries.nan_to_num())
        sel = fused.selection(1 - fused.cur)
        pools = [u8(p) for p in (fused.k_pool, fused.v_pool)]
        scales = [s.cpu().numpy() for s in (fused.k_scale, fused.v_scale)]
        for u in sorted(set(rng.integers(0, wl.U, 5).tolist())):
            b, h = divmod(u, wl.Hkv)
            T, g = int(wl.T(step, b)), int(wl.g[u])
            K, V = (Q.dequant_unit(p, s, wl.page_table[u], T, kind) for p, s in zip(pools, scales))
            n_sub = -(-T // int(wl.s[u]))
            means = np.stack([K[j * wl.s[u]:(j + 1) * wl.s[u]].mean(0) for j in range(n_sub)])
            assert np.abs(fused.unit_summaries(u, n_sub) - means).max() <= 1e-4 * max(1.0, np.abs(means).max())
            qh = fused.q[step][b, h * wl.G:(h + 1) * wl.G].double().cpu().numpy()
            t = O.selected_tokens(sel[u], g, T)
            to, tl = bound(qh, K[t], V[t], len(sel[u]) * g / 16, wl.d)
            want, want_l = O.sparse_attention(qh, K, V, sel[u], g, T)
            assert np.abs(fused.out[b, h * wl.G:(h + 1) * wl.G].cpu().numpy() - want).max() <= to
            assert np.abs(apart.out[b, h * wl.G:(h + 1) * wl.G].cpu().numpy() - want).max() <= to
            assert np.abs(fused.lse[b, h * wl.G:(h + 1) * wl.G].cpu().numpy() - want_l).max() <= tl


def test_decode_loop_block_logits():
    """ED-DMA block logits through the fused step over an 8-bit cache."""
    wl = make_workload(5, seed=33, B=2, T=1200, steps=3)
    layer = PagedLayer(wl, kv8="e4m3", ed_dma=True)
    layer.prefill()
    for step in range(wl.steps):
        layer.append(step)
        layer.fused_step(step)
    torch.cuda.synchronize()
    assert layer.read_status() == 0
    step, sel = wl.steps - 1, layer.selection(1 - layer.cur)
    pools = [(u8(p), s.cpu().numpy()) for p, s in ((layer.k_pool, layer.k_scale), (layer.v_pool, layer.v_scale))]
    for u in (0, 7, 15):
        b, h = divmod(u, wl.Hkv)
        T, g = int(wl.T(step, b)), int(wl.g[u])
        K, V = (Q.dequant_unit(p, s, wl.page_table[u], T, "e4m3") for p, s in pools)
        qh = layer.q[step][b, h * wl.G:(h + 1) * wl.G].double().cpu().numpy()
        want, _ = O.ed_dma_attention(qh, K, V, sel[u], g, T, wl.evict[u].astype(np.float64))
        t = O.selected_tokens(sel[u], g, T)
        to, _ = bound(qh, K[t], V[t], len(sel[u]) * g / 16, wl.d)
        assert np.abs(layer.out[b, h * wl.G:(h + 1) * wl.G].cpu().numpy() - want).max() <= 2 * to


def test_fused_step_wait_runs_out_and_recovers():
    """A selection held back (through the caller's own workspace words): the 8-bit attention's
    bounded wait gives up, reports it, and the next step is right."""
    wl = make_workload(2, seed=35, T=3001)
    layer = PagedLayer(wl, kv8="int8")
    layer.prefill()
    layer.append(0)
    torch.cuda.synchronize()
    u = next(x for x in range(wl.U) if wl.cls[x] != O.STREAMING)
    default = B.wait_limit_ns()
    B.set_wait_limit_ns(2_000_000)
    try:
        layer.workspace.view(torch.int32)[u] = 1 << 20       # the unit's selection ticket
        layer.fused_step(0)
        torch.cuda.synchronize()
        assert layer.read_status() == B.BS_ERR_TIMEOUT
    finally:
        B.set_wait_limit_ns(default)
    layer.workspace.zero_()
    layer.status.zero_()
    for cnt in layer.cnt:
        cnt.zero_()
    layer.fused_step(0)
    torch.cuda.synchronize()
    assert layer.read_status() == 0
    T, g, h = int(wl.T(0, 0)), int(wl.g[u]), u % wl.Hkv
    K, V = (Q.dequant_unit(u8(p), s.cpu().numpy(), wl.page_table[u], T, "int8")
            for p, s in ((layer.k_pool, layer.k_scale), (layer.v_pool, layer.v_scale)))
    sel = layer.selection(1 - layer.cur)[u]
    qh = layer.q[0][0, h * wl.G:(h + 1) * wl.G].double().cpu().numpy()
    want, _ = O.sparse_attention(qh, K, V, sel, g, T)
    t = O.selected_tokens(sel, g, T)
    assert np.abs(layer.out[0, h * wl.G:(h + 1) * wl.G].cpu().numpy() - want).max() <= \
        bound(qh, K[t], V[t], len(sel) * g / 16, wl.d)[0]


def test_layer_refuses_an_unknown_type():
    with pytest.raises(ValueError, match="kv8"):
        PagedLayer(make_workload(1, seed=0, T=64), kv8="fp4")
