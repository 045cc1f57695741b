"""PagedLayer's calls on rows of new tokens: tensors that do not fit are refused before any launch
(CPU), and calls on two streams share nothing (GPU)."""
import numpy as np
import pytest
import torch

from long_context_serving_gb300.build import build
from long_context_serving_gb300.layer import PagedLayer
from workloads import make_workload

ROWS = 6


@pytest.fixture(scope="module")
def layer():
    build()
    return PagedLayer(make_workload(2, seed=3, T=100), device="cpu")


def _q(wl, rows=ROWS, dtype=torch.bfloat16):
    return torch.zeros(rows, wl.Hq, wl.d, dtype=dtype)


@pytest.mark.parametrize("bad", ["transposed", "padded", "fp32", "heads", "flat"])
def test_queries_that_are_not_rows_are_refused(layer, bad):
    wl = layer.wl
    q = {"transposed": torch.zeros(wl.Hq, ROWS, wl.d, dtype=torch.bfloat16).transpose(0, 1),
         "padded": torch.zeros(ROWS, wl.Hq, 2 * wl.d, dtype=torch.bfloat16)[:, :, :wl.d],
         "fp32": _q(wl, dtype=torch.float32),
         "heads": torch.zeros(ROWS, wl.Hq + 1, wl.d, dtype=torch.bfloat16),
         "flat": torch.zeros(ROWS, wl.Hq * wl.d, dtype=torch.bfloat16)}[bad]
    with pytest.raises(ValueError):
        layer.prefill_attend(q, [94], [100])
    kv = torch.zeros(ROWS, wl.Hkv * wl.d, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.draft_attend(q, kv, kv, [ROWS], torch.ones(ROWS, dtype=torch.int64), [100])


@pytest.mark.parametrize("bad", ["short", "narrow", "strides", "fp32", "columns"])
def test_new_keys_that_do_not_fit_are_refused(layer, bad):
    wl = layer.wl
    w = wl.Hkv * wl.d
    good = torch.zeros(ROWS, w, dtype=torch.bfloat16)
    k = {"short": good[:ROWS - 1], "narrow": good[:, :w - 8], "strides": torch.zeros(ROWS, 2 * w, dtype=torch.bfloat16)[:, :w],
         "fp32": good.float(), "columns": torch.zeros(w, ROWS, dtype=torch.bfloat16).t()}[bad]
    masks = torch.ones(ROWS, dtype=torch.int64)
    for pair in ((k, good), (good, k)):
        with pytest.raises(ValueError):
            layer.draft_attend(_q(wl), *pair, [ROWS], masks, [100])
        with pytest.raises(ValueError):
            layer.commit_drafts(*pair, [ROWS], [[0, 1]], [100])


def test_masks_paths_and_lengths_that_do_not_fit_are_refused(layer):
    wl = layer.wl
    kv = torch.zeros(ROWS, wl.Hkv * wl.d, dtype=torch.bfloat16)
    for m in (torch.ones(ROWS - 1, dtype=torch.int64), torch.ones(ROWS, dtype=torch.int32),
              torch.ones(2 * ROWS, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            layer.draft_attend(_q(wl), kv, kv, [ROWS], m, [100])
    for path in ([[0, -1, 2]], [[ROWS]], [0, 1], [[0], [1]]):      # a hole, no such draft, not a row a sequence
        with pytest.raises(ValueError):
            layer.commit_drafts(kv, kv, [ROWS], path, [100])
    for lo, hi in (([94, 0], [100, 0]), ([94], [100, 0]), (94, 100)):
        with pytest.raises(ValueError):
            layer.prefill_attend(_q(wl), lo, hi)


@pytest.mark.gpu
def test_streams_share_nothing():
    """Prompt rows and drafts attended on two streams in turn, each behind work that keeps its stream
    busy, are bitwise what each call gives alone; a fused projection's columns serve as rows."""
    wl = make_workload(2, seed=3, T=3000)
    layer = PagedLayer(wl)
    layer.prefill()
    layer.append(0)
    layer.fused_step(0)
    T = int(wl.T_prefill[0])
    gen = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn(90, wl.Hq * wl.d + 64, device="cuda", generator=gen).bfloat16()
    q = wide[:, :wl.Hq * wl.d].unflatten(1, (wl.Hq, wl.d))
    kv = torch.randn(8, 2, wl.Hkv * wl.d, device="cuda", generator=gen).bfloat16()
    masks = torch.tensor([(1 << (i + 1)) - 1 for i in range(8)], dtype=torch.int64, device="cuda")
    calls = [lambda s: layer.prefill_attend(q[:3], [T - 3], [T], s),        # rows few enough to be split
             lambda s: layer.draft_attend(q[:8], kv[:, 0], kv[:, 1], [8], masks, [T + 1], s),
             lambda s: layer.prefill_attend(q, [T - 90], [T], s)]
    alone = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    busy = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        s = streams[i % 2]
        with torch.cuda.stream(s):
            busy @ busy
        got.append(calls[i % 3](s if i < 6 else s.cuda_stream))
    torch.cuda.synchronize()
    assert layer.read_status() == 0
    for i, (out, lse) in enumerate(got):
        assert out.is_contiguous() and torch.equal(out, alone[i % 3][0]) and torch.equal(lse, alone[i % 3][1]), i
