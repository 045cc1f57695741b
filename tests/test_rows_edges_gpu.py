"""Prompt and tree attention where rows are split: rows of NaN through the merge,
values at the end of the range in many pieces."""
import numpy as np
import pytest
import torch

import _rows as R
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
