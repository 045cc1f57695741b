"""Page calls on maps with damaged entries, and directly ahead of the decode step, on the GPU."""
import numpy as np
import pytest
import torch

from test_pages_gpu import Map, Model, filled
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build

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
