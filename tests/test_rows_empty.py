"""Calls on no rows at all do nothing: row tensors of no elements have no address (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build
from long_context_serving_gb300.layer import PagedLayer
from workloads import make_workload

ref, ST = ctypes.byref, 0x60000


@pytest.fixture(scope="module")
def layer():
    build()
    return PagedLayer(make_workload(2, seed=3, T=100), device="cpu")


def test_attention_of_no_rows(layer):
    kv = B.KV(k_pool=0x10000, v_pool=0x20000, page_table=0x30000, seq_lens=0x40000)
    cfg = B.HeadCfg(cls=0x1000, sink_tokens=0x2000, local_tokens=0x3000, block_tokens=0x4000)
    stride = layer.wl.Hq * layer.wl.d
    B.prefill_attn(layer.dims, None, stride, 0, kv, cfg, 0x1000, 0x2000, 1, None, None, None, ST, 0)
    drafts = B.Drafts(k_new=0, v_new=0, row_stride=stride, n_rows=0, row_begin=0x1000, n_draft=0x2000, visible=0, max_draft=1)
    B.tree_decode_attn(layer.dims, None, stride, kv, cfg, 0x1000, 0x2000, drafts, None, None, None, ST, 0)


def test_a_commit_of_nothing(layer):
    """No drafts, none accepted, a path of no columns."""
    wl = layer.wl
    for rows, path in ((0, np.empty((1, 0))), (0, [[-1, -1]]), (3, np.empty((1, 0))), (3, [[-1]])):
        kv = torch.zeros(rows, wl.Hkv * wl.d, dtype=torch.bfloat16)
        layer.commit_drafts(kv, kv, [rows], path, [99])


def test_rotation_of_no_rows(layer):
    wl = layer.wl
    rope = B.Rope(inv_freq=0x9000, rot_dim=wl.d, interleaved=0, magnitude=1.0, eps=1e-6)
    none = torch.empty(0, wl.Hq * wl.d, dtype=torch.bfloat16)
    at = torch.empty(0, dtype=torch.int32)
    B.rope_append(layer.dims, rope, none, none, none, (wl.Hq + 2 * wl.Hkv) * wl.d, 0, at, at, None, None, none, none, ST, 0)
    pools = B.Pools(k_pool=0x10000, v_pool=0x20000)
    B.rope_append(layer.dims, rope, none, none, none, (wl.Hq + 2 * wl.Hkv) * wl.d, 0, at, at, pools, 0x3000, none, None, ST, 0)


def test_rows_that_exist_need_their_addresses(layer):
    """The same calls of one row are refused."""
    wl = layer.wl
    rope = B.Rope(inv_freq=0x9000, rot_dim=wl.d, interleaved=0, magnitude=1.0, eps=1e-6)
    call = B.lib().bs_rope_append
    for missing in range(5):
        p = [0x10000, 0x20000, 0x1000, 0x40000, 0x50000]
        p[missing] = None
        assert call(ref(layer.dims), ref(rope), p[0], p[1], None, (wl.Hq + 2 * wl.Hkv) * wl.d, 1, p[2], None, None, None, p[3], p[4], ST,
                    None) == B.BS_ERR_INVALID_ARG
