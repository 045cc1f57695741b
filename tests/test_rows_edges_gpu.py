"""Prompt and tree attention where rows are split: rows of NaN through the merge,
values at the end of the range in many pieces; a key that dominates; rotation by more
than a turn a position; long caches; a tree beside others."""
import itertools

import numpy as np
import pytest
import torch

import _quant as Q
import _rows as R
from _rows import i32
from long_context_serving_gb300 import bsattn as B
from test_rows_gpu import Prefill, Tree, _sync_status

pytestmark = pytest.mark.gpu


def _tree(kind, form, n, d=64, **kw):
    """A tree in each of its plans: whole, a CTA a key tile, pieces that the units share."""
    B_, lens, gather = {"whole": (1, [40], 4), "tiles": (1, [4000], 256), "shared": (3, [4000, 2500, 3000], 512)}[form]
    c = R.Cache(B_, 2, 4, d, lens, kind, max_gather_pages_per_unit=gather)
    t = Tree(c, [n] * B_, **kw)
    assert (B.tree_workspace_size(c.dims, n) > 0) == (form != "whole")
    return c, t


def _prefill(kind, form, rows, d=64):
    lens, pages = ([120, 100], None) if form == "whole" else ([5000, 3111], 600)
    c = R.Cache(2, 1, 4, d, lens, kind, max_pages=pages)
    p = Prefill(c, [rows, rows])
    assert (B.prefill_workspace_size(c.dims, p.rows, p.max_new) > 0) == (form != "whole")
    return c, p


def _k_nan(c, units):
    """Every K of the units is NaN (by its code, or by its scale)."""
    for u in units:
        pages = torch.as_tensor(c.table_np[u][c.table_np[u] >= 0].astype(np.int64), device="cuda")
        if c.kind == "bf16":
            c.k[pages] = float("nan")
        elif c.kind == "e4m3":
            c.k.view(torch.uint8)[pages] = 0x7F
        else:
            c.ks[pages] = float("nan")


def _set_row(x, row, head, value):
    d = x.c.d
    x.q[row, head * d:(head + 1) * d] = value


CASES = [("prefill", form, rows) for form in ("whole", "split") for rows in (1, 20, 60)] + \
        [("tree", form, n) for form in ("whole", "tiles", "shared") for n in (3, 20, 60)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("call,form,n", CASES)
def test_a_query_of_nan_is_a_row_of_nan(call, form, n, kind):
    """However its keys are shared out; the other rows keep their bits."""
    c, x = _prefill(kind, form, n) if call == "prefill" else _tree(kind, form, n)
    x.run()
    assert _sync_status(c) == 0
    clean, lse = x.out.clone(), x.lse.clone()
    row, head = int(x.row0[0]) + n - 1, 1
    _set_row(x, row, head, float("nan"))
    x.run()
    assert _sync_status(c) == 0
    assert torch.isnan(x.out[row, head].float()).all() and torch.isnan(x.lse[row, head])
    others = torch.ones(x.out.shape[:2], dtype=torch.bool, device="cuda")
    others[row, head] = False
    assert torch.equal(x.out[others], clean[others]) and torch.equal(x.lse[others], lse[others])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("call,form,n", CASES)
def test_keys_of_nan_are_rows_of_nan(call, form, n, kind):
    """All K of the first sequence's units; rows of a tree that see no draft, so nothing else."""
    if call == "prefill":
        c, x = _prefill(kind, form, n)
    else:
        c, x = _tree(kind, form, n, masks=lambda i, rng: 0)
    _k_nan(c, range(c.Hkv))
    x.run()
    assert _sync_status(c) == 0
    mine = slice(int(x.row0[0]), int(x.row0[0]) + n)
    assert torch.isnan(x.out[mine].float()).all() and torch.isnan(x.lse[mine]).all()
    if c.B > 1:
        next_ = slice(int(x.row0[1]), int(x.row0[1]) + n)
        assert torch.isfinite(x.out[next_].float()).all() and torch.isfinite(x.lse[next_]).all()


def _fill_keys(c, value):
    """K[t] = value(t) in its first element, 0 in the others (bf16 caches)."""
    for u, T in ((u, int(c.lens[u // c.Hkv])) for u in range(c.B * c.Hkv)):
        t = torch.arange(T, device="cuda")
        at = torch.as_tensor(c.table_np[u].astype(np.int64), device="cuda")[t // 16]
        c.k[at, t % 16] = 0.0
        x = np.array([value(i) for i in range(T)])
        c.k[at, t % 16, 0] = torch.as_tensor(x, device="cuda").bfloat16()
        c.K[u] = np.zeros((T, c.d))
        c.K[u][:, 0] = x


@pytest.mark.parametrize("call,form,n", [c for c in CASES if c[2] != 20])
def test_the_largest_values_in_many_pieces(call, form, n):
    """V of 2^90 where the second half of every key tile passes the first by 2^28.9: a piece's sums are
    relative to its first half's maximum, and as many of them as there are stay finite together. Every
    weighted mean is 2^90, a number of bf16, up to the weights' rounding."""
    c, x = _prefill("bf16", form, n) if call == "prefill" else _tree("bf16", form, n, masks=lambda i, rng: 0)
    _fill_keys(c, lambda t: 20.0 if t % 128 >= 64 else 0.0)
    c.v[:] = 2.0 ** 90
    x.q[:] = 0.0
    for h in range(c.Hkv * c.G):
        x.q[:, h * c.d] = 8.0                     # a logit of 8 K / sqrt(64) = K: 20 log2(e) = 28.85
    x.run()
    assert _sync_status(c) == 0
    for b in range(c.B):
        out = x.out[x.row0[b]:x.row0[b] + n].double()
        assert ((out - 2.0 ** 90).abs() <= 2 * R.HALF_BF16 * 2.0 ** 90).all(), out.max()


def _two_keys(c, u, a, b, rng):
    """Unit u with keys of which a has the logit 0 and b one of 4.375 for a query of sqrt(d) in the first
    place, all others far below; V zero but for b. c.K and c.V, float64, follow."""
    T = int(c.lens[u // c.Hkv])
    row = c.table_np[u][:-(-T // 16)]
    pages = torch.as_tensor(row.astype(np.int64), device="cuda")
    K, V = np.zeros((T, c.d)), np.zeros((T, c.d))
    if c.kind == "bf16":
        K[:, 0], K[a, 0], K[b, 0] = -60.0, 0.0, 4.375
        V[b] = R.bf16(rng.uniform(1, 2, c.d))
        for pool, x in ((c.k, K), (c.v, V)):
            pool[pages] = torch.as_tensor(np.pad(x, ((0, 16 * len(row) - T), (0, 0)))).cuda().bfloat16().view(-1, 16, c.d)
    else:
        low, one, scale = (0xFE, 0x50, 4.375 / 8) if c.kind == "e4m3" else (0x81, 64, 4.375 / 64)    # -448 and 8; -127 and 64
        kc, vc = np.zeros((16 * len(row), c.d), np.uint8), np.zeros((16 * len(row), c.d), np.uint8)
        kc[:, 0], kc[a, 0], kc[b, 0] = low, 0, one
        vc[b] = rng.integers(1, 120, c.d)
        for pool, x in ((c.k, kc), (c.v, vc)):
            pool.view(torch.uint8)[pages] = torch.as_tensor(x.reshape(-1, 16, c.d)).cuda()
        c.ks[pages], c.vs[pages] = scale, 1.375
        K, V = Q.decode(kc[:T], c.kind) * scale, Q.decode(vc[:T], c.kind) * 1.375
    c.K[u], c.V[u] = K, V


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("call,form,n", CASES)
def test_a_key_that_dominates_comes_back(call, form, n, kind):
    """A first key sets the reference; a later one, in the second half of its tile or in another, weighs
    2^6.3 times as much, a number that bf16 does not hold. Its share p of the row is over 0.9: both parts of the
    quotient take the same rounded weight, so that its half step, 2^-8 of it at most, leaves 1 - p of
    itself, and the other weights as much; logits are within 2^-16 (1 + their terms) in both
    parts, the result is rounded once, half a step of its own binade."""
    if call == "prefill" and form == "whole":
        c = R.Cache(2, 1, 4, 64, [128, 128], kind)
        x = Prefill(c, [n, n])
    else:
        c, x = _prefill(kind, form, n) if call == "prefill" else _tree(kind, form, n, masks=lambda i, rng: 0)
    H, T = c.Hkv * c.G, int(min(c.lens))
    qs = R.bf16(np.random.default_rng(3).uniform(7.5, 8.5, (x.rows, H)))
    x.q[:] = 0.0
    x.q.view(x.rows, H, c.d)[..., 0] = torch.as_tensor(qs).cuda().bfloat16()
    for at in sorted({min(66, T - 1), (T - n - 1 if call == "prefill" else T - 1)}):
        for u in range(c.B * c.Hkv):
            _two_keys(c, u, 7, at, np.random.default_rng(u))
        x.run()
        assert _sync_status(c) == 0
        out = x.out.double().cpu().numpy()
        for b, h, i, g in itertools.product(range(c.B), range(c.Hkv), range(n), range(c.G)):
            u, row = b * c.Hkv + h, int(x.row0[b]) + i
            seen = int(c.lens[b]) - (n - i - 1 if call == "prefill" else 0)
            w = np.exp(c.K[u][:seen, 0] * float(qs[row, h * c.G + g]) / np.sqrt(c.d))
            p = w[at] / w.sum()
            assert p > 0.9
            want = p * c.V[u][at]
            half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 1e-30))) - 8)
            tol = half + np.abs(want) * (2 * R.HALF_BF16 * (1 - p) + 2.0 ** -15 * (1 + 5))
            err = np.abs(out[row, h * c.G + g] - want)
            assert (err <= tol).all(), (b, h, i, g, at, float((err / half).max()))


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_more_than_a_turn_a_position(inter):
    """Frequencies up to 32 radians a position at positions near 2^24: the angle's fraction of a turn is
    right to 2^-23 (2^-24 up to one radian), sine and cosine in fp32 to 2^-22."""
    d, rows = 64, 4096
    freq = np.zeros(d // 2)
    freq[:8] = [1.0, 0.77, 2 * np.pi, 3.3, 10.7, 25.1327, 31.9, 32.0]
    c = R.Cache(1, 1, 1, d, [16], "bf16", q_dtype=B.BS_FP32)
    pos = np.random.default_rng(1).integers(1 << 23, 1 << 24, rows)
    x = torch.zeros(rows, 3, d, device="cuda")
    x[:, :, 0 if inter else 0:(16 if inter else 8):2 if inter else 1] = 1.0       # the first of each pair
    q, k = torch.empty(rows, 1, d, device="cuda"), torch.empty(rows, 1, d, device="cuda")
    f_t = torch.as_tensor(freq, device="cuda")
    rope = B.Rope(inv_freq=f_t.data_ptr(), rot_dim=d, interleaved=int(inter), magnitude=1.0, eps=0.0)
    B.rope_append(c.dims, rope, x, x[:, 1], x[:, 2], 3 * d, rows, i32(pos), None, None, None, q, k, c.status)
    assert _sync_status(c) == 0
    got = q[:, 0].double().cpu().numpy()
    a, b = (got[:, 0:16:2], got[:, 1:16:2]) if inter else (got[:, :8], got[:, d // 2:d // 2 + 8])
    wide = np.longdouble
    turns = pos[:, None].astype(wide) * freq[:8].astype(wide) * wide("0.15915494309189533576888376337251436")
    angle = (2 * np.pi * (turns - np.rint(turns))).astype(np.float64)
    tol = 2 * np.pi * np.where(freq[:8] <= 1, 2.0 ** -24, 2.0 ** -23) + 2.0 ** -22
    assert (np.abs(a - np.cos(angle)) <= tol).all() and (np.abs(b - np.sin(angle)) <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 30, 200])
def test_prompts_behind_a_long_cache(kind, new):
    """Tens of thousands of tokens before the new ones, dense and windowed heads."""
    c = R.Cache(1, 2, 4, 128, [40961], kind)
    p = Prefill(c, [new], cls=[1, 0], sink=70, local=9000)
    p.run()
    assert _sync_status(c) == 0
    p.check(rows=6)


def test_a_tree_beside_others():
    """Other sequences' selections may move a tree's split points, and so the last bits of its sums: with
    either it is what the formula gives, the same bits again in the same batch."""
    for other in (60, 5):
        c = R.Cache(2, 2, 4, 64, [3000, 3000], "bf16", seed=5, max_gather_pages_per_unit=512)
        t = Tree(c, [12, 12])
        t.cnt.copy_(i32([188, 188, other, other]))
        t.sel[2] = t.sel[3] = list(range(other))
        t.run()
        assert _sync_status(c) == 0
        t.check()
        first = t.out.clone()
        t.ws.fill_(0xFF)
        t.run()
        assert _sync_status(c) == 0 and torch.equal(first, t.out)
