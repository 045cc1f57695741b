"""Prompt attention with page scales and logits that are not finite: rows that see such a key show it,
rows that do not are what the formula gives over the keys that they see."""
import itertools

import numpy as np
import pytest
import torch

import _rows as R
from test_rows_gpu import Prefill, _sync_status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [6, 40, 150])      # the forms of 32, 128 and 256 rows
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_v_scales_that_are_not_finite(kind, what, rows):
    """The last page's V scale: rows before the page do not see any of its keys."""
    T = 212 if rows > 6 else 195
    c = R.Cache(1, 1, 4, 64, [T], kind)
    p = Prefill(c, [rows])
    lp = (T - 1) // 16
    c.vs[int(c.table_np[0, lp])] = float(what)
    p.run()
    assert _sync_status(c) == 0
    out = p.out.double().cpu().numpy()
    seen_by_some = 0
    for i, g in itertools.product(range(rows), range(4)):
        pos, row = T - rows + i, out[p.row0[0] + i, g]
        if pos >= lp * 16:
            seen_by_some += 1
            assert not np.isfinite(row).any(), (i, g)
            continue
        want = R.attend_row(p.q_np[p.row0[0] + i, g].astype(np.float64), c.K[0][:pos + 1], c.V[0][:pos + 1])
        R.check_row(row, float(p.lse[p.row0[0] + i, g]), want, (i, g))
    assert 0 < seen_by_some < 4 * rows


@pytest.mark.parametrize("rows", [6, 40, 150])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("page", ["first", "last"])
def test_k_scales_that_are_nan(kind, page, rows):
    """A NaN logit: every row that sees a key of the page is NaN, its lse too; the others are as ever."""
    T = 212 if rows > 6 else 195
    c = R.Cache(1, 1, 4, 64, [T], kind)
    p = Prefill(c, [rows])
    lp = 0 if page == "first" else (T - 1) // 16
    c.ks[int(c.table_np[0, lp])] = float("nan")
    p.run()
    assert _sync_status(c) == 0
    out = p.out.double().cpu().numpy()
    for i, g in itertools.product(range(rows), range(4)):
        pos, row, z = T - rows + i, out[p.row0[0] + i, g], float(p.lse[p.row0[0] + i, g])
        if pos >= lp * 16:
            assert np.isnan(row).all() and np.isnan(z), (i, g)
            continue
        want = R.attend_row(p.q_np[p.row0[0] + i, g].astype(np.float64), c.K[0][:pos + 1], c.V[0][:pos + 1])
        R.check_row(row, z, want, (i, g))


@pytest.mark.parametrize("rows", [6, 40, 150])
def test_a_logit_of_minus_infinity_weighs_nothing(rows):
    """Beside it a V that only the last row sees is NaN: the other rows, computed again without it, still
    take the key of weight zero for one."""
    T = 195
    c = R.Cache(1, 1, 4, 64, [T], "bf16")
    p = Prefill(c, [rows])
    p.q_np[..., 3] = 1.0
    p.q.view(p.rows, 4, 64)[..., 3] = 1.0
    low = 140                                            # in the last key's tile, whatever the split
    c.k[int(c.table_np[0, low // 16]), low % 16, 3] = float("-inf")
    c.v[int(c.table_np[0, (T - 1) // 16]), (T - 1) % 16] = float("nan")
    p.run()
    assert _sync_status(c) == 0
    out = p.out.double().cpu().numpy()
    for i, g in itertools.product(range(rows), range(4)):
        pos, row = T - rows + i, out[p.row0[0] + i, g]
        if pos == T - 1:
            assert np.isnan(row).all()
            continue
        s = np.arange(T) <= pos
        s[low] = False
        want = R.attend_row(p.q_np[p.row0[0] + i, g].astype(np.float64), c.K[0][s], c.V[0][s])
        R.check_row(row, float(p.lse[p.row0[0] + i, g]), want, (i, g))


@pytest.mark.parametrize("rows", [6, 40, 150])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_row_of_one_key_is_its_value_rounded_once(kind, rows):
    """The first token sees itself alone. Its weight, taken with the V scale's mantissa, is the reference:
    1 up to the fp32 steps of a logit of a few units and of exp2 (under 2^-18 together), so 1 in bf16, and
    the quotient is V within 2^-17 before the one rounding to bf16, half a step of 2^-8 of it."""
    for seed in range(8):
        c = R.Cache(1, 4, 4, 64, [rows], kind, seed=seed)
        p = Prefill(c, [rows])
        p.run()
        assert _sync_status(c) == 0
        out = p.out.double().cpu().numpy()[p.row0[0]]
        for u, g in itertools.product(range(4), range(4)):
            v = np.asarray(c.V[u][0], np.float64)
            err = np.abs(out[u * 4 + g] - v)
            assert (err <= (R.HALF_BF16 + 2.0 ** -16) * np.abs(v)).all(), (seed, u, g, (err / np.maximum(np.abs(v), 1e-30)).max())
