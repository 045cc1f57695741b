"""The 8-bit cache and page calls on the host: refusals before any launch (nothing here
touches a GPU), sizes, and the tests' own plain forms checked against each other."""
import ctypes

import numpy as np
import pytest
import torch

import _quant as Q
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return B.lib()


def _dims(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, max_pages_per_unit=64,
                max_blocks_per_unit=32, max_sel_per_unit=16, max_subs_per_unit=128, max_gather_pages_per_unit=32,
                n_pages=128, kv_dtype=B.BS_E4M3, q_dtype=B.BS_BF16)
    base.update(kw)
    return B.Dims(**base)


ref = ctypes.byref
ST = 0x60000


def test_eight_bit_dims():
    assert B.workspace_size(_dims()) == B.workspace_size(_dims(kv_dtype=B.BS_BF16)) > 0
    assert B.workspace_size(_dims(kv_dtype=B.BS_INT8)) > 0
    for bad in (dict(kv_dtype=4), dict(kv_dtype=-1), dict(q_dtype=B.BS_E4M3), dict(q_dtype=B.BS_INT8)):
        assert B.workspace_size(_dims(**bad)) == 0, bad


def test_attention_and_summaries_need_scales():
    L = B.lib()
    cfg = B.HeadCfg(*([0x50000] * 9))
    full = dict(k_pool=0x10000, v_pool=0x20000, page_table=0x30000, seq_lens=0x40000, k_scale=0x7000, v_scale=0x8000)
    io = B.StepIO(**{n: 0x1000 * (i + 1) for i, (n, _) in enumerate(B.StepIO._fields_)})
    io.workspace_bytes = 1 << 30
    for gone in ("k_scale", "v_scale"):
        kv = B.KV(**{**full, gone: 0})
        for d in (_dims(), _dims(kv_dtype=B.BS_INT8)):
            assert L.bs_sparse_decode_attn(ref(d), 0x1000, ref(kv), ref(cfg), 0x2000, 0x3000, None, 0x4000, 0x5000,
                                           0x8000, 1 << 30, ST, None) == B.BS_ERR_INVALID_ARG
            assert L.bs_sparse_decode_attn_noalloc(ref(d), 0x1000, ref(kv), ref(cfg), 0x2000, 0x3000, None, 0x4000,
                                                   0x5000, ST, None) == B.BS_ERR_INVALID_ARG
            assert L.bs_decode_step(ref(d), ref(kv), ref(cfg), ref(io), 0, None) == B.BS_ERR_INVALID_ARG
    kv = B.KV(**{**full, "k_scale": 0})
    assert L.bs_build_block_summaries(ref(_dims()), ref(kv), ref(cfg), 0x1000, 1, 0x70000, ST, None) == \
        B.BS_ERR_INVALID_ARG


def test_calls_without_page_scales_refuse_eight_bit_caches():
    L = B.lib()
    cfg = B.HeadCfg(*([0x50000] * 9))
    host = B.HostKV(k_pool=0x10000, v_pool=0x20000, page_table=0x30000, n_pages=128)
    cache = B.BlockCache(k_pool=0x40000, v_pool=0x50000, page_table=0x60000, slot_block=0x70000, block_slot=0x80000,
                         slots_per_unit=8, pages_per_slot=2)
    tables = B.HostTables(page_table=0x1000, seq_lens=0x2000, block_tokens=0x3000)
    for d in (_dims(), _dims(kv_dtype=B.BS_INT8)):
        assert L.bs_block_swap(ref(d), ref(cfg), 0x1000, ref(host), ref(cache), 0x1100, 0x2000, 0x3000, 0x4000, ST,
                               None) == B.BS_ERR_INVALID_ARG
        assert L.bs_cpu_sparse_attn(ref(d), 0x1000, ref(host), ref(tables), 0x4000, 0x5000, 0x6000, 0x7000, 4) == \
            B.BS_ERR_INVALID_ARG


def _append(d, pools=None, k_new=0x10000, v_new=0x20000, stride=256, rows=4, max_new=1, table=0x1000, lens=0x2000,
            begin=0x3000, row0=0x4000, st=ST):
    pools = pools or B.Pools(k_pool=0x30000, v_pool=0x40000, k_scale=0x50000, v_scale=0x50004)
    return B.lib().bs_quant_append(ref(d) if d else None, ref(pools), table, lens, begin, row0, k_new, v_new, stride,
                                   rows, max_new, st, None)


def test_append_refusals():
    d = _dims()
    assert _append(None) == B.BS_ERR_INVALID_ARG
    assert _append(_dims(head_dim=96)) == B.BS_ERR_SHAPE
    for kv in (B.BS_BF16, B.BS_FP32):
        assert _append(_dims(kv_dtype=kv)) == B.BS_ERR_INVALID_ARG
    for name in ("k_new", "v_new", "table", "lens", "begin", "row0", "st"):
        assert _append(d, **{name: None}) == B.BS_ERR_INVALID_ARG, name
    whole = dict(k_pool=0x30000, v_pool=0x40000, k_scale=0x50000, v_scale=0x50004)
    for name in whole:
        assert _append(d, pools=B.Pools(**{**whole, name: 0})) == B.BS_ERR_INVALID_ARG, name
    assert _append(d, stride=248) == B.BS_ERR_INVALID_ARG          # shorter than a row of KV heads
    assert _append(d, rows=-1) == B.BS_ERR_INVALID_ARG
    assert _append(d, max_new=0) == B.BS_ERR_INVALID_ARG
    assert _append(d, stride=260) == B.BS_ERR_ALIGN                # 520 bytes
    assert _append(_dims(q_dtype=B.BS_FP32), stride=258) == B.BS_ERR_ALIGN
    assert _append(d, k_new=0x10002) == B.BS_ERR_ALIGN
    assert _append(d, v_new=0x20008) == B.BS_ERR_ALIGN
    assert _append(d, pools=B.Pools(**{**whole, "v_pool": 0x40008})) == B.BS_ERR_ALIGN


def test_page_call_refusals():
    L = B.lib()
    d = _dims()
    m = B.PageMap(page_table=0x1000, ref_count=0x2000, seq_lens=0x3000)
    ws, nb = 0x10000, B.pages_workspace_size(d)
    cp = B.PageCopies(pairs=0x4000, count=0x5000, capacity=8)
    pools = B.Pools(k_pool=0x30000, v_pool=0x40000, k_scale=0x50000, v_scale=0x60000)
    assert nb > 0 and nb % 16 == 0 and B.pages_workspace_size(_dims(head_dim=96)) == 0

    def reserve(d=d, m=m, lens=0x6000, ws=ws, nb=nb, st=ST):
        return L.bs_pages_reserve(ref(d), ref(m), lens, ws, nb, st, None)

    def fork(d=d, m=m, src=0x6000, dst=0x7000, n=2, cp=cp, ws=ws, nb=nb, st=ST):
        return L.bs_pages_fork(ref(d), ref(m), src, dst, n, ref(cp), ws, nb, st, None)

    def free(d=d, m=m, seqs=0x6000, n=2, st=ST):
        return L.bs_pages_free(ref(d), ref(m), seqs, n, st, None)

    def compact(d=d, m=m, cp=cp, live=0x6000, ws=ws, nb=nb, st=ST):
        return L.bs_pages_compact(ref(d), ref(m), ref(cp), live, ws, nb, st, None)

    def copy(d=d, pools=pools, cp=cp, st=ST):
        return L.bs_pages_copy(ref(d), ref(pools), ref(cp), st, None)

    for call in (reserve, fork, free, compact, copy):
        assert call(d=_dims(page_size=8)) == B.BS_ERR_SHAPE
        assert call(st=None) == B.BS_ERR_INVALID_ARG
    for call in (reserve, fork, free, compact):
        for name in ("page_table", "ref_count", "seq_lens"):
            bad = B.PageMap(page_table=0x1000, ref_count=0x2000, seq_lens=0x3000)
            setattr(bad, name, 0)
            assert call(m=bad) == B.BS_ERR_INVALID_ARG, name
    for call in (reserve, fork, compact):
        assert call(ws=None) == B.BS_ERR_INVALID_ARG
        assert call(ws=0x10004) == B.BS_ERR_ALIGN
        assert call(nb=nb - 16) == B.BS_ERR_CAPACITY
    assert reserve(lens=None) == fork(src=None) == fork(dst=None) == free(seqs=None) == compact(live=None) == \
        B.BS_ERR_INVALID_ARG
    for call in (fork, free):
        assert call(n=0) == call(n=3) == B.BS_ERR_INVALID_ARG          # 1 <= n <= batch
    for call in (fork, compact, copy):
        assert call(cp=B.PageCopies(pairs=0, count=0x5000, capacity=8)) == B.BS_ERR_INVALID_ARG
        assert call(cp=B.PageCopies(pairs=0x4000, count=0, capacity=8)) == B.BS_ERR_INVALID_ARG
        assert call(cp=B.PageCopies(pairs=0x4000, count=0x5000, capacity=0)) == B.BS_ERR_INVALID_ARG
        assert call(cp=B.PageCopies(pairs=0x4004, count=0x5000, capacity=8)) == B.BS_ERR_ALIGN
    assert fork(cp=B.PageCopies(pairs=0x4000, count=0x5000, capacity=3)) == B.BS_ERR_CAPACITY   # 2 x 2 heads
    assert copy(pools=B.Pools(k_pool=0x30000, v_pool=0x40000, k_scale=0, v_scale=0x60000)) == B.BS_ERR_INVALID_ARG
    assert copy(pools=B.Pools(k_pool=0x30008, v_pool=0x40000, k_scale=0x50000, v_scale=0x60000)) == B.BS_ERR_ALIGN
    with pytest.raises(ValueError, match="differ in length"):
        B.pages_fork(d, m, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), cp,
                     torch.zeros(4), torch.zeros(1, dtype=torch.int32), stream=0)


# ---- the tests' plain forms ------------------------------------------------------------
def test_code_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(Q.E4M3)) and np.array_equal(t[~np.isnan(t)], Q.E4M3[~np.isnan(t)])
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.6, 4000), Q.E4M3[:127],
                        (Q.E4M3[:126] + Q.E4M3[1:127]) / 2]).astype(np.float32)     # values and exact ties
    y = np.concatenate([y, -y])
    y = y[np.abs(y) <= 448]
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.round_half_even(y, "e4m3"), want)
    assert Q.round_half_even([2.5, 3.5, -2.5, 300, -300, np.nan], "int8").view(np.int8).tolist() == \
        [2, 4, -2, 127, -127, 0]


def test_scale_rule():
    for a in (1.0, 447.9, 448.0, 448.1, 3.5, 1e-3, 2.0 ** -130, 3e38, 7.0, 7.01):
        s = Q.scale_for(a, "e4m3")
        assert np.log2(float(s)) == int(np.log2(float(s))) and np.float32(a) / float(s) <= 448
        assert s == Q.TINY or np.float32(a) / (float(s) / 2) > 448
    assert Q.scale_for(0, "e4m3") == 0 and Q.scale_for(0, "int8") == 0
    assert Q.scale_for(127, "int8") == 1 and Q.scale_for(1e-40, "int8") == Q.TINY
