"""Calls on rows of new tokens, on the host: refusals before any launch and workspace sizes."""
import ctypes

import pytest

from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build

ref = ctypes.byref
ST = 0x60000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return B.lib()


def _dims(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, max_pages_per_unit=64,
                max_blocks_per_unit=32, max_sel_per_unit=16, max_subs_per_unit=128, max_gather_pages_per_unit=32,
                n_pages=128, kv_dtype=B.BS_BF16, q_dtype=B.BS_BF16)
    base.update(kw)
    return B.Dims(**base)


def _kv(**kw):
    return B.KV(**{**dict(k_pool=0x10000, v_pool=0x20000, page_table=0x30000, seq_lens=0x40000, k_scale=0x7000, v_scale=0x8000), **kw})


def _rope(d=None, pools=None, no_rope=False, **kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, stride=12 * 128, rows=4, pos=0x1000, seq=0x2000, table=0x3000, q_out=0x40000,
             k_out=0x50000, st=ST, inv_freq=0x9000, rot_dim=128, interleaved=0, magnitude=1.0, q_weight=0, k_weight=0, eps=1e-6)
    a.update(kw)
    r = B.Rope(**{n: a[n] for n in ("inv_freq", "rot_dim", "interleaved", "magnitude", "q_weight", "k_weight", "eps")})
    return B.lib().bs_rope_append(ref(d or _dims()), None if no_rope else ref(r), a["q"], a["k"], a["v"], a["stride"], a["rows"],
                                  a["pos"], a["seq"], ref(pools) if pools else None, a["table"], a["q_out"], a["k_out"],
                                  a["st"], None)


def test_rope_refusals():
    pools = B.Pools(k_pool=0x100000, v_pool=0x200000)
    assert _rope(rows=0) == B.BS_OK                                   # nothing to do, nothing launched
    assert _rope(rows=0, pools=pools, k_out=None) == B.BS_OK
    for kw in (dict(q=None), dict(k=None), dict(pos=None), dict(q_out=None), dict(st=None), dict(inv_freq=0), dict(no_rope=True),
               dict(k_out=None), dict(rows=-1), dict(stride=7 * 128), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(magnitude=float("nan")), dict(magnitude=float("inf")),
               dict(pools=pools, table=None), dict(pools=pools, seq=None), dict(pools=pools, v=None),
               dict(pools=B.Pools(k_pool=0, v_pool=0x1000)), dict(pools=B.Pools(k_pool=0x1000, v_pool=0)),
               dict(pools=pools, d=_dims(kv_dtype=B.BS_E4M3)), dict(pools=pools, d=_dims(kv_dtype=B.BS_INT8))):
        assert _rope(**kw) == B.BS_ERR_INVALID_ARG, kw
    for rot in (0, 8, 24, 144, -16):
        assert _rope(rot_dim=rot) == B.BS_ERR_SHAPE, rot
    assert _rope(d=_dims(head_dim=64), rot_dim=128) == B.BS_ERR_SHAPE
    for kw in (dict(q=0x10008), dict(k=0x10002), dict(q_out=0x40008), dict(k_out=0x50004), dict(stride=12 * 128 + 4),
               dict(inv_freq=0x9004), dict(pools=pools, v=0x30008), dict(pools=B.Pools(k_pool=0x100008, v_pool=0x200000))):
        assert _rope(**kw) == B.BS_ERR_ALIGN, kw
    assert _rope(d=_dims(head_dim=96)) == B.BS_ERR_SHAPE


def _prefill(d=None, kv=None, cfg=None, **kw):
    a = dict(q=0x10000, stride=8 * 128, rows=4, begin=0x1000, row0=0x2000, max_new=2, out=0x40000, lse=0x50000, ws=0x100000,
             ws_bytes=1 << 40, st=ST)
    a.update(kw)
    cfg = cfg or B.HeadCfg(cls=0x1000, sink_tokens=0x2000, local_tokens=0x3000)
    return B.lib().bs_prefill_attn(ref(d or _dims()), a["q"], a["stride"], a["rows"], ref(kv or _kv()), ref(cfg), a["begin"],
                                   a["row0"], a["max_new"], a["out"], a["lse"], a["ws"], a["ws_bytes"], a["st"], None)


def test_prefill_refusals():
    assert _prefill(rows=0) == B.BS_OK
    for kw in (dict(q=None), dict(begin=None), dict(row0=None), dict(out=None), dict(st=None), dict(rows=-1), dict(max_new=0),
               dict(stride=7 * 128), dict(kv=_kv(k_pool=0)), dict(kv=_kv(v_pool=0)), dict(kv=_kv(page_table=0)),
               dict(kv=_kv(seq_lens=0)), dict(cfg=B.HeadCfg(sink_tokens=1, local_tokens=1)),
               dict(cfg=B.HeadCfg(cls=1, local_tokens=1)), dict(cfg=B.HeadCfg(cls=1, sink_tokens=1)),
               dict(d=_dims(q_dtype=B.BS_FP32)), dict(d=_dims(kv_dtype=B.BS_FP32)),
               dict(d=_dims(kv_dtype=B.BS_E4M3), kv=_kv(k_scale=0)), dict(d=_dims(kv_dtype=B.BS_INT8), kv=_kv(v_scale=0)),
               dict(ws=None)):
        assert _prefill(**kw) == B.BS_ERR_INVALID_ARG, kw
    for kw in (dict(q=0x10008), dict(out=0x40008), dict(stride=8 * 128 + 4), dict(kv=_kv(k_pool=0x10008)), dict(ws=0x100008)):
        assert _prefill(**kw) == B.BS_ERR_ALIGN, kw
    need = B.prefill_workspace_size(_dims(), 4, 2)
    assert need > 0 and need % 16 == 0
    assert _prefill(ws_bytes=need - 1) == B.BS_ERR_CAPACITY
    assert _prefill(rows=1 << 31) == B.BS_ERR_CAPACITY


def _tree(d=None, kv=None, cfg=None, drop=None, **kw):
    a = dict(q=0x10000, stride=8 * 128, sel=0x1000, cnt=0x2000, out=0x40000, lse=0x50000, ws=0x100000, ws_bytes=1 << 40, st=ST,
             k_new=0x10000, v_new=0x20000, row_stride=512, n_rows=4, row_begin=0x3000, n_draft=0x4000, visible=0x5000, max_draft=8)
    a.update(kw)
    dr = B.Drafts(**{n: a[n] for n, _ in B.Drafts._fields_})
    cfg = cfg or B.HeadCfg(block_tokens=0x1000)
    return B.lib().bs_tree_decode_attn(ref(d or _dims()), a["q"], a["stride"], ref(kv or _kv()), ref(cfg), a["sel"], a["cnt"],
                                       None if drop else ref(dr), a["out"], a["lse"], a["ws"], a["ws_bytes"], a["st"], None)


def test_tree_refusals():
    assert _tree(n_rows=0) == B.BS_OK
    for kw in (dict(q=None), dict(sel=None), dict(cnt=None), dict(out=None), dict(st=None), dict(drop=True), dict(k_new=0), dict(v_new=0),
               dict(row_begin=0), dict(n_draft=0), dict(visible=0), dict(max_draft=0), dict(max_draft=65), dict(n_rows=-1),
               dict(row_stride=248), dict(stride=7 * 128), dict(cfg=B.HeadCfg()), dict(d=_dims(q_dtype=B.BS_FP32)),
               dict(d=_dims(kv_dtype=B.BS_FP32)), dict(d=_dims(kv_dtype=B.BS_E4M3), kv=_kv(k_scale=0)), dict(ws=None)):
        assert _tree(**kw) == B.BS_ERR_INVALID_ARG, kw
    for kw in (dict(q=0x10008), dict(out=0x40004), dict(k_new=0x10008), dict(v_new=0x20002), dict(row_stride=516),
               dict(visible=0x5004), dict(ws=0x100004)):
        assert _tree(**kw) == B.BS_ERR_ALIGN, kw
    need = B.tree_workspace_size(_dims(), 8)
    assert need > 0 and need % 16 == 0
    assert _tree(ws_bytes=need - 1) == B.BS_ERR_CAPACITY


def _commit(d=None, pools=None, no_pools=False, **kw):
    a = dict(table=0x1000, lens=0x2000, begin=0x3000, row0=0x4000, path=0x5000, stride=4, k=0x10000, v=0x20000, row_stride=512,
             rows=16, st=ST)
    a.update(kw)
    pools = pools or B.Pools(k_pool=0x30000, v_pool=0x40000, k_scale=0x50000, v_scale=0x50004)
    return B.lib().bs_tree_commit(ref(d or _dims()), None if no_pools else ref(pools), a["table"], a["lens"], a["begin"], a["row0"],
                                  a["path"], a["stride"], a["k"], a["v"], a["row_stride"], a["rows"], a["st"], None)


def test_commit_refusals():
    for kw in (dict(table=None), dict(lens=None), dict(begin=None), dict(row0=None), dict(path=None), dict(k=None), dict(v=None),
               dict(st=None), dict(no_pools=True), dict(stride=0), dict(stride=65), dict(row_stride=248), dict(rows=-1),
               dict(pools=B.Pools(k_pool=0, v_pool=0x40000)), dict(pools=B.Pools(k_pool=0x40000, v_pool=0)),
               dict(d=_dims(kv_dtype=B.BS_E4M3), pools=B.Pools(k_pool=0x30000, v_pool=0x40000, v_scale=0x50000)),
               dict(d=_dims(kv_dtype=B.BS_INT8), pools=B.Pools(k_pool=0x30000, v_pool=0x40000, k_scale=0x50000))):
        assert _commit(**kw) == B.BS_ERR_INVALID_ARG, kw
    for kw in (dict(k=0x10008), dict(v=0x20008), dict(row_stride=516), dict(pools=B.Pools(k_pool=0x30008, v_pool=0x40000))):
        assert _commit(**kw) == B.BS_ERR_ALIGN, kw


def test_workspace_sizes():
    """0 for bad arguments; bounded by 64 MB of records and their maxima; none for a full grid."""
    for bad in (dict(head_dim=96), dict(n_q_heads=9), dict(batch=0)):
        assert B.prefill_workspace_size(_dims(**bad), 4, 2) == 0 and B.tree_workspace_size(_dims(**bad), 8) == 0
    assert B.prefill_workspace_size(_dims(), 0, 2) == 0 and B.prefill_workspace_size(_dims(), 4, 0) == 0
    assert B.tree_workspace_size(_dims(), 0) == 0 and B.tree_workspace_size(_dims(), 65) == 0
    long = dict(max_pages_per_unit=8192, max_gather_pages_per_unit=8192)
    assert B.prefill_workspace_size(_dims(**long, batch=1), 20000, 20000) == 0
    for b in (1, 2, 16, 64, 1000):
        for n in (1, 7, 64):
            for size in (B.prefill_workspace_size(_dims(**long, batch=b), b * n, n), B.tree_workspace_size(_dims(**long, batch=b), n)):
                assert size <= (64 << 20) * 65 // 64 + (1 << 20)
