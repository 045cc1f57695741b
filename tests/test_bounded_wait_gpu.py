"""The kernels' wait on a shared-memory barrier (mbar_wait_bounded), by a kernel of the test's own: a phase
that nothing completes ends with the status and leaves the GPU usable, one that completes late does not."""
import ctypes
import subprocess

import pytest
import torch

from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300 import build as Bd

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "bs_internal.cuh"
// Warp 0 waits for a barrier of one arrival; warp 1 arrives after `late_ns`, or not at all.
__global__ void waits(int arrives, uint64_t late_ns, uint64_t limit_ns, int32_t *st, int32_t *ok, uint64_t *took) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) bsi::mbar_init(&bar, 1);
  __syncthreads();
  const uint64_t t0 = bsi::global_ns();
  if (threadIdx.x < 32) {
    const bool done = __all_sync(0xffffffffu, bsi::mbar_wait_bounded(&bar, 0, st, limit_ns));
    if (threadIdx.x == 0) {
      *ok = done;
      *took = bsi::global_ns() - t0;
    }
  } else if (threadIdx.x == 32 && arrives) {
    for (int i = 0; i < 100000 && bsi::global_ns() - t0 < late_ns; ++i) __nanosleep(100);
    bsi::mbar_arrive(&bar);
  }
}
extern "C" int run(int arrives, uint64_t late_ns, uint64_t limit_ns, int32_t *st, int32_t *ok, uint64_t *took, void *stream) {
  waits<<<1, 64, 0, (cudaStream_t)stream>>>(arrives, late_ns, limit_ns, st, ok, took);
  return cudaGetLastError();
}
"""


def test_waits_end(tmp_path):
    src, so = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(SOURCE)
    r = subprocess.run([Bd.nvcc(), *Bd.FLAGS, *Bd.ARCH, "-shared", "-o", str(so), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    run = ctypes.CDLL(str(so)).run
    run.argtypes = [ctypes.c_int, ctypes.c_uint64, ctypes.c_uint64] + [ctypes.c_void_p] * 4
    st, ok = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    took = torch.zeros(1, dtype=torch.int64, device="cuda")
    limit = 20_000_000
    for arrives, late, want_ok, want_st in ((1, 0, 1, 0), (0, 0, 0, B.BS_ERR_TIMEOUT), (1, 1_000_000, 1, 0)):
        st.zero_()
        ok.fill_(-1)
        assert run(arrives, late, limit, st.data_ptr(), ok.data_ptr(), took.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert int(ok) == want_ok and int(st) == want_st
        if not want_ok:
            assert limit <= int(took) < 50 * limit
        assert int(took) >= late
