"""PagedLayer's calls on rows of new tokens: what they compute, over every cache type, and what a commit
leaves for the next step."""
import itertools

import numpy as np
import pytest
import torch

import _quant as Q
import _rows as R
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.layer import PagedLayer
from workloads import make_workload

pytestmark = pytest.mark.gpu
KV8 = [None, "e4m3", "int8"]


def _cache64(layer, u, T):
    """K and V of unit u's first T tokens as the pool holds them."""
    row = layer.page_table[u].cpu().numpy()
    if layer.kv8:
        return tuple(Q.dequant_unit(p.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), row, T, layer.kv8)
                     for p, s in ((layer.k_pool, layer.k_scale), (layer.v_pool, layer.v_scale)))
    flat = lambda p: p[torch.as_tensor(row[:-(-T // 16)].astype(np.int64), device=p.device)].double().cpu().numpy()  # noqa: E731
    return tuple(flat(p).reshape(-1, layer.wl.d)[:T] for p in (layer.k_pool, layer.v_pool))


def _rows(rng, *shape):
    return torch.as_tensor(R.bf16(rng.standard_normal(shape))).cuda().bfloat16()


@pytest.mark.parametrize("kv8", KV8)
def test_prompts_and_drafts_against_the_formula(kv8):
    wl = make_workload(2, seed=3, T=700)
    layer = PagedLayer(wl, kv8=kv8)
    layer.prefill()
    layer.append(0)
    layer.fused_step(0)                           # the selection that drafts attend
    T, n, rng = int(wl.T_prefill[0]), 9, np.random.default_rng(5)
    lo, hi = np.array([T - 90]), np.array([T])
    q = _rows(rng, 90, wl.Hq, wl.d)
    out, lse = (x.double().cpu().numpy() for x in layer.prefill_attend(q, lo, hi))
    keys = [_cache64(layer, u, T + 1) for u in range(wl.U)]
    q64 = q.double().cpu().numpy()
    for i, u in itertools.product((0, 40, 89), range(wl.U)):
        s = np.flatnonzero(R.prefill_seen(T - 90 + i, T, wl.cls[u] == B.BS_STREAMING, int(wl.sink[u]), int(wl.local[u])))
        for h in range(u * wl.G, (u + 1) * wl.G):
            R.check_row(out[i, h], lse[i, h], R.attend_row(q64[i, h], keys[u][0][s], keys[u][1][s]), (i, h))
    k, v = _rows(rng, n, wl.Hkv, wl.d), _rows(rng, n, wl.Hkv, wl.d)
    masks = [1 << i | (int(rng.integers(0, 1 << 30)) & ((1 << i) - 1)) for i in range(n)]
    out, lse = layer.draft_attend(q[:n], k, v, [n], torch.tensor(masks, dtype=torch.int64, device="cuda"), [T + 1])
    assert layer.read_status() == 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    k64, v64 = k.double().cpu().numpy(), v.double().cpu().numpy()
    last = 1 - layer.cur
    for u in range(wl.U):
        blocks = layer.sel[last][u, :int(layer.cnt[last][u])].cpu().numpy()
        t = np.concatenate([np.arange(b * wl.g[u], min((b + 1) * wl.g[u], T + 1)) for b in blocks])
        for i in range(n):
            js = [j for j in range(n) if masks[i] >> j & 1]
            K, V = np.concatenate([keys[u][0][t], k64[js, u]]), np.concatenate([keys[u][1][t], v64[js, u]])
            for h in range(u * wl.G, (u + 1) * wl.G):
                R.check_row(out[i, h], lse[i, h], R.attend_row(q64[i, h], K, V), (i, h))


@pytest.mark.parametrize("kv8", KV8)
def test_the_step_behind_a_commit_scores_what_was_committed(kv8):
    """Forty accepted drafts cross sub-blocks and pages: the step that follows has the means, scores,
    selection and output of a layer whose tokens were appended and summed."""
    n = 40
    wl = make_workload(2, seed=4, T=700, steps=n + 1)
    T = wl.T_prefill.astype(np.int64)
    layers = [PagedLayer(wl, kv8=kv8) for _ in range(2)]
    for x in layers:
        x.prefill()
    a, b = layers
    new = [p[:, int(T[0]):int(T[0]) + n].transpose(0, 1).contiguous() for p in (a._K, a._V)]      # [n][Hkv][d]
    a.commit_drafts(new[0], new[1], [n], np.arange(n)[None], T)
    b._write_tokens(T, T + n)
    at, begin = (torch.as_tensor(x.astype(np.int32), device="cuda") for x in (T + n, T))
    B.build_block_summaries(b.dims, b.kv_at(at), b.cfg, begin, n, b.summaries, b.status)
    assert a.read_status() == 0 and b.read_status() == 0
    assert torch.equal(a.summaries.view(torch.int32), b.summaries.view(torch.int32))
    for x in layers:
        x.append(n)
        x.fused_step(n)
        assert x.read_status() == 0
    for name in ("scores", "out", "lse", "summaries"):
        assert torch.equal(getattr(a, name).view(torch.int32), getattr(b, name).view(torch.int32)), name
    assert torch.equal(a.sel[0], b.sel[0]) and torch.equal(a.cnt[0], b.cnt[0])


@pytest.mark.parametrize("kv8", [None, "int8"])
def test_appends_of_no_rows(kv8):
    """No row and no accepted draft is nothing to do; an accepted draft without a row is reported."""
    wl = make_workload(2, seed=3, T=100)
    layer = PagedLayer(wl, kv8=kv8)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    before = layer.k_pool.view(torch.uint8).clone()
    empty = torch.empty(0, wl.Hkv * wl.d, dtype=torch.bfloat16, device="cuda")
    pools = layer.pools if kv8 else B.Pools(k_pool=layer.k_pool.data_ptr(), v_pool=layer.v_pool.data_ptr())
    for accepted, status in ((0, 0), (1, B.BS_ERR_DEVICE_BOUNDS)):
        B.tree_commit(layer.dims, pools, layer.page_table, i32(50 + accepted), i32(50), i32(0), i32(0, 0), 2, empty, empty,
                      wl.Hkv * wl.d, 0, layer.status)
        assert layer.read_status() == status
        if kv8:
            layer.status.zero_()
            B.quant_append(layer.dims, pools, layer.page_table, i32(50 + accepted), i32(50), i32(0), empty, empty, wl.Hkv * wl.d, 0, 1,
                           layer.status)
            assert layer.read_status() == status
    assert torch.equal(before, layer.k_pool.view(torch.uint8))


def test_attention_of_no_rows():
    """Empty tensors, which have no address, give empty results."""
    wl = make_workload(2, seed=3, T=100)
    layer = PagedLayer(wl)
    q = torch.empty(0, wl.Hq, wl.d, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, wl.Hkv * wl.d, dtype=torch.bfloat16, device="cuda")
    assert q.data_ptr() == 0
    for out, lse in (layer.prefill_attend(q, [99], [99]),
                     layer.draft_attend(q, kv, kv, [0], torch.empty(0, dtype=torch.int64, device="cuda"), [99])):
        assert out.shape == (0, wl.Hq, wl.d) and lse.shape == (0, wl.Hq)
    layer.commit_drafts(kv, kv, [0], [[-1]], [99])
    assert layer.read_status() == 0
