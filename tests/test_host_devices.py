"""The library's host code against a stand-in for the CUDA runtime (CPU only): the objects
of the build are linked with a small C++ runtime that launches nothing. It keeps kernel
attributes per device, as CUDA does, and refuses a launch whose dynamic shared memory or
cluster the current device was not told of."""
import os
import shutil
import subprocess

import pytest

from long_context_serving_gb300 import build as Bd

RUNTIME = r"""
#include <cstdio>
#include <cstring>
#include <map>
#include <utility>
#include <cuda.h>
#include <cuda_runtime_api.h>
#include "bsattn.h"

static int g_device = 0, g_launches = 0;
static cudaError_t g_last = cudaSuccess;
static std::map<std::pair<int, const void *>, std::map<int, int>> g_attrs;

static cudaError_t launched(const void *f, size_t smem, unsigned cluster) {
  auto &a = g_attrs[{g_device, f}];
  ++g_launches;
  if ((smem > 48 * 1024 && size_t(a[cudaFuncAttributeMaxDynamicSharedMemorySize]) < smem) ||
      (cluster > 8 && a[cudaFuncAttributeNonPortableClusterSizeAllowed] != 1))
    return g_last = cudaErrorInvalidValue;
  return cudaSuccess;
}
static struct { dim3 grid, block; size_t smem; void *stream; } g_conf;

extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = g_device; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v) {
  g_attrs[{g_device, f}][a] = v;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { const cudaError_t e = g_last; g_last = cudaSuccess; return e; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *f, int, size_t smem, unsigned) {
  // (like the runtime: none for shared memory the device was not told of)
  *n = smem > 48 * 1024 && size_t(g_attrs[{g_device, f}][cudaFuncAttributeMaxDynamicSharedMemorySize]) < smem ? 0 : 2;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *) { *p = (void *)0x100000; return cudaSuccess; }
static CUresult encode(...) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *r) {
  *p = (void *)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
  unsigned cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  return launched(f, c->dynamicSmemBytes, cluster);
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, struct CUstream_st *st) {
  g_conf = {g, b, s, st};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *g, dim3 *b, size_t *s, void *st) {
  *g = g_conf.grid;
  *b = g_conf.block;
  *s = g_conf.smem;
  *(void **)st = g_conf.stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) { *k = (cudaKernel_t)f; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void **, size_t s, cudaStream_t) {
  return launched((const void *)k, s, 1);
}
cudaError_t cudaLaunchKernel(const void *f, dim3, dim3, void **, size_t s, cudaStream_t) { return launched(f, s, 1); }
void **__cudaRegisterFatBinary(void *) { static void *h; return &h; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
}

static int32_t *P(int i) { return (int32_t *)(uintptr_t)(0x1000000 + 0x10000 * i); }   // never looked at
static bs_dims dims_for(int kv, int units, int gather, int blocks) {
  bs_dims d{};
  d.batch = units / 2; d.n_kv_heads = 2; d.n_q_heads = 8; d.head_dim = 128; d.page_size = 16;
  d.max_pages_per_unit = 4 * blocks; d.max_blocks_per_unit = blocks; d.max_sel_per_unit = 4096 < blocks ? 4096 : blocks;
  d.max_subs_per_unit = 8 * blocks; d.max_gather_pages_per_unit = gather; d.n_pages = 1 << 20;
  d.kv_dtype = (bs_dtype)kv; d.q_dtype = BS_BF16;
  return d;
}
static bs_head_cfg cfg() {
  return bs_head_cfg{P(1), P(2), P(3), P(4), P(5), P(6), P(7), (const int64_t *)P(8), P(9)};
}
static bs_kv cache() { return bs_kv{P(10), P(11), P(12), P(13), (const float *)P(14), (const float *)P(15)}; }
static bs_step_io step_io(size_t bytes) {
  bs_step_io io{};
  io.q = P(20); io.summaries = (float *)P(21); io.scores = (float *)P(22); io.evict_logits = (float *)P(23);
  io.alive = (uint8_t *)P(24); io.prev_idx = P(25); io.prev_cnt = P(26); io.cur_idx = P(27); io.cur_cnt = P(28);
  io.added = P(29); io.added_cnt = P(30); io.removed = P(31); io.removed_cnt = P(32); io.out = (float *)P(33);
  io.lse = (float *)P(34); io.workspace = P(35); io.workspace_bytes = bytes; io.dev_status = P(36);
  return io;
}
"""

DEVICES = RUNTIME + r"""
int main() {
  int fails = 0;
  // clusters; workspace mode in two launches, in three
  const int plans[][3] = {{4, 200, 400}, {60, 200, 400}, {60, 600, 1500}, {60, 600, 8000}, {4, 3000, 8000}};
  for (int device : {0, 1, 0, 3, 70})
    for (int kv : {BS_BF16, BS_FP32, BS_E4M3, BS_INT8})
      for (auto &p : plans) {
        g_device = device;
        const bs_dims d = dims_for(kv, p[0], p[1], p[2]);
        const bs_head_cfg c = cfg();
        const bs_kv k = cache();
        const size_t ws = bs_workspace_size(&d);
        const bs_step_io io = step_io(ws);
        auto check = [&](const char *name, bs_status s) {
          if (s == BS_OK) return;
          std::printf("%s on device %d: kv %d, %d units, %d pages, %d blocks: %s\n", name, device, kv, p[0], p[1], p[2],
                      bs_status_string(s));
          ++fails;
        };
        check("bs_build_block_summaries",
              bs_build_block_summaries(&d, &k, &c, P(40), 1, (float *)P(21), P(36), nullptr));
        check("bs_score_blocks",
              bs_score_blocks(&d, P(20), &c, P(13), (float *)P(21), BS_GROUP_MAX, (float *)P(22), P(36), nullptr));
        check("bs_select_topk", bs_select_topk(&d, &c, P(13), (float *)P(22), (float *)P(23), (uint8_t *)P(24), P(27), P(28),
                                               P(36), nullptr));
        check("bs_sparse_decode_attn", bs_sparse_decode_attn(&d, P(20), &k, &c, P(27), P(28), nullptr, (float *)P(33),
                                                             (float *)P(34), P(35), ws, P(36), nullptr));
        check("bs_block_setdiff",
              bs_block_setdiff(&d, P(25), P(26), P(27), P(28), P(29), P(30), P(31), P(32), P(36), nullptr));
        check("bs_decode_step", bs_decode_step(&d, &k, &c, &io, BS_GROUP_MAX, nullptr));
      }
  std::printf("launches %d\nfails %d\n", g_launches, fails);
  return fails != 0;
}
"""


def run_host(tmp_path, source, *args):
    nvcc, cxx = Bd.nvcc(), shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    objs = [os.path.join(Bd.BUILD, s.replace(".cu", ".o")) for s in Bd.SOURCES]
    Bd.build(force=not all(os.path.exists(o) for o in objs))
    src, exe = tmp_path / "host.cpp", tmp_path / "host"
    src.write_text(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-w", "-I", cuda, "-I", Bd.INCLUDE, str(src), *objs, "-lpthread", "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=120)


def test_every_call_runs_on_every_device_of_a_process(tmp_path):
    """Kernel attributes hold for one device: a second one gets its own, in each call and plan."""
    r = run_host(tmp_path, DEVICES)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split("launches ")[1].split()[0]) >= 5 * 4 * 5 * 7


OLD_KV = RUNTIME + r"""
#include <sys/mman.h>
#include <unistd.h>
#include <cstddef>
// bs_kv as it was before it had scales, at the very end of readable memory.
int main() {
  const size_t page = sysconf(_SC_PAGESIZE), old = offsetof(bs_kv, k_scale);
  char *m = (char *)mmap(nullptr, 2 * page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  if (m == MAP_FAILED || mprotect(m + page, page, PROT_NONE) != 0) return 2;
  const bs_kv k = cache();
  const bs_kv *kv = (const bs_kv *)std::memcpy(m + page - old, &k, old);
  int fails = 0;
  for (int type : {BS_BF16, BS_FP32})
    for (int units : {4, 60}) {
      const bs_dims d = dims_for(type, units, 600, 8000);
      const bs_head_cfg c = cfg();
      const size_t ws = bs_workspace_size(&d);
      const bs_step_io io = step_io(ws);
      fails += bs_build_block_summaries(&d, kv, &c, P(40), 1, (float *)P(21), P(36), nullptr) != BS_OK;
      fails += bs_sparse_decode_attn(&d, P(20), kv, &c, P(27), P(28), nullptr, (float *)P(33), (float *)P(34), P(35), ws,
                                     P(36), nullptr) != BS_OK;
      fails += bs_sparse_decode_attn_noalloc(&d, P(20), kv, &c, P(27), P(28), nullptr, (float *)P(33), (float *)P(34),
                                             P(36), nullptr) != BS_OK;
      fails += bs_decode_step(&d, kv, &c, &io, BS_GROUP_MAX, nullptr) != BS_OK;
    }
  std::printf("fails %d\n", fails);
  return fails != 0;
}
"""


def test_a_bs_kv_without_scales_is_enough_for_other_caches(tmp_path):
    """A program built when bs_kv ended at seq_lens passes 32 bytes: no more of them are read unless
    the cache is 8-bit."""
    r = run_host(tmp_path, OLD_KV)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
