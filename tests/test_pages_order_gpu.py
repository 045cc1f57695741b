"""Page calls on maps with damaged entries, and directly ahead of the decode step, on the GPU."""
import numpy as np
import pytest
import torch

from test_pages_gpu import Map, Model, filled, i32
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build
from long_context_serving_gb300.layer import PagedLayer
from workloads import make_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build()
    B.lib()


@pytest.mark.parametrize("entry", [-2, -7, -2 ** 31])
def test_entries_below_minus_one_are_reported(entry):
    """-1 holds no page; a smaller entry lies outside the pool. free drops it, fork refuses to share
    it, compact leaves it; reserve gives its place a page."""
    m, g = filled(lens=(40, 32, 0, 0))
    m.table[0, 1] = entry
    g = Map(m)
    g.free([0])
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS
    m.table[0, 1] = -1
    m.ref[1] = 1                                    # (page 1, which the entry held, keeps its count)
    m.free([0])
    g.check(m)

    m, g = filled(lens=(40, 32, 0, 0))
    m.table[3, 1] = entry                           # a full page of sequence 1
    g = Map(m)
    g.fork([0, 1], [2, 3])
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS and int(g.count) == 0
    g.check(m)
    m.table[3, 1] = m.table[0, 2]                   # the partial page of sequence 0's first head
    m.table[0, 2] = entry
    g = Map(m)
    g.fork([0], [2])
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS and int(g.count) == 0
    g.check(m)

    m = Model(2, 1, 8, 64)
    m.ref[40:50] = 1
    m.table[0, :8], m.table[1, :2] = np.arange(40, 48), (48, 49)
    m.table[1, 5] = entry
    g = Map(m)
    g.compact()
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS
    m.compact()
    g.check(m)

    m, g = filled(lens=(40, 32, 0, 0))
    m.table[0, 1] = entry
    g = Map(m)
    g.reserve([40, 32, 0, 0])
    assert g.take_status() == m.reserve([40, 32, 0, 0]) == 0
    g.check(m)


# (name of the plan: workload, sizes; clusters, the workspace in two launches and in three)
STEPS = {"cluster": (2, dict(T=2900, steps=1)), "ragged": (4, dict(B=3, T=1700, steps=1)),
         "workspace": (3, dict(B=4, T=20000, steps=1))}


@pytest.mark.parametrize("kv8", [None, "e4m3"])
@pytest.mark.parametrize("name", sorted(STEPS))
def test_fused_step_directly_behind_a_compaction(name, kv8):
    """The step that follows compact on the stream, with no other launch between, reads the table
    that compact wrote: bitwise the step of a cache whose pages never moved. (The pages' contents
    were copied ahead, by the moves of a compaction of a copy of the map.)"""
    cfg, kw = STEPS[name]
    wl = make_workload(cfg, seed=61, **kw)
    still, moved = PagedLayer(wl, kv8=kv8), PagedLayer(wl, kv8=kv8)
    for layer in (still, moved):
        layer.prefill()
        layer.append(0)
    dev = "cuda"
    # a stretch of new pages ahead of all others is free
    extra = wl.n_pages // 3 + 5
    pools = [moved.k_pool, moved.v_pool] + ([moved.k_scale, moved.v_scale] if kv8 else [])
    pools = [torch.cat([p[:1].view(torch.uint8).expand(extra, *p[:1].view(torch.uint8).shape[1:]), p.view(torch.uint8)])
             .view(p.dtype) if p.dim() > 1 else torch.cat([p[:1].expand(extra), p]) for p in pools]
    moved.k_pool, moved.v_pool = pools[:2]
    if kv8:
        moved.k_scale, moved.v_scale = pools[2:]
    n_pages = wl.n_pages + extra
    moved.dims.n_pages = n_pages
    last = np.repeat(-(-(wl.T_prefill + 1) // 16), wl.Hkv)
    table = np.where(np.arange(wl.page_table.shape[1]) < last[:, None], wl.page_table + extra, -1).astype(np.int32)
    table0 = torch.as_tensor(table, device=dev)
    ref0 = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    ref0[table0[table0 >= 0].long()] = 1
    assert int(ref0.max()) == 1 and int(ref0[:extra].max()) == 0
    moved.page_table.copy_(table0)
    moved.kv = B.KV(k_pool=moved.k_pool.data_ptr(), v_pool=moved.v_pool.data_ptr(),
                    page_table=moved.page_table.data_ptr(), seq_lens=0,
                    k_scale=moved.k_scale.data_ptr() if kv8 else 0, v_scale=moved.v_scale.data_ptr() if kv8 else 0)
    lens = moved.seq_lens[0].clone()
    ref = ref0.clone()
    page_map = B.PageMap(page_table=moved.page_table.data_ptr(), ref_count=ref.data_ptr(), seq_lens=lens.data_ptr())
    pairs, count = torch.zeros((n_pages, 2), dtype=torch.int32, device=dev), i32([0])
    copies = B.PageCopies(pairs=pairs.data_ptr(), count=count.data_ptr(), capacity=n_pages)
    n_live, ws = i32([0]), torch.zeros(B.pages_workspace_size(moved.dims) // 4, dtype=torch.int32, device=dev)
    ptrs = B.Pools(k_pool=moved.k_pool.data_ptr(), v_pool=moved.v_pool.data_ptr(), k_scale=moved.kv.k_scale,
                   v_scale=moved.kv.v_scale)

    def compact():
        B.pages_compact(moved.dims, page_map, copies, n_live, ws, moved.status)

    compact()
    B.pages_copy(moved.dims, ptrs, copies, moved.status)
    torch.cuda.synchronize()
    assert int(count) >= extra // 2 and moved.read_status() == 0
    still.fused_step(0)
    for _ in range(10):
        moved.page_table.copy_(table0)
        ref.copy_(ref0)
        for x in (moved.out, moved.lse, moved.scores):
            x.zero_()
        moved.cur = 0
        moved.cnt[1].zero_()
        if moved.alive is not None:
            moved.alive.fill_(1)
        compact()
        moved.fused_step(0)
        torch.cuda.synchronize()
        assert moved.read_status() == 0 and int(n_live) == int(ref0.sum())
        assert moved.selection(0) == still.selection(0)
        assert torch.equal(moved.out, still.out) and torch.equal(moved.lse, still.lse)
        assert torch.equal(moved.summaries.nan_to_num(), still.summaries.nan_to_num())
