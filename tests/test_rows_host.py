"""The calls on rows of new tokens, host code against the stand-in for the CUDA runtime (CPU only):
every form on several devices, a bs_kv without scales; and the sources' loads."""
import os
import re

import pytest

from long_context_serving_gb300 import build as Bd
from test_host_devices import RUNTIME, run_host

MAIN = RUNTIME + r"""
#include <sys/mman.h>
#include <unistd.h>
#include <cstddef>
static bs_kv *at_the_end() {      // bs_kv as it was before it had scales, at the very end of readable memory
  const size_t page = sysconf(_SC_PAGESIZE), old = offsetof(bs_kv, k_scale);
  char *m = (char *)mmap(nullptr, 2 * page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  if (m == MAP_FAILED || mprotect(m + page, page, PROT_NONE) != 0) return nullptr;
  const bs_kv k = cache();
  return (bs_kv *)std::memcpy(m + page - old, &k, old);
}
int main() {
  int fails = 0;
  const bs_kv full = cache(), *old = at_the_end();
  if (old == nullptr) return 2;
  for (int device : {0, 1, 0, 3, 70})
    for (int kv : {BS_BF16, BS_FP32, BS_E4M3, BS_INT8})
      for (int dim : {64, 128})
        for (int units : {2, 60, 400}) {
          g_device = device;
          bs_dims d = dims_for(kv, units, 600, 8000);
          d.head_dim = dim;
          const bs_head_cfg c = cfg();
          const bs_kv *k = kv == BS_BF16 ? old : &full;
          auto check = [&](const char *name, bs_status s) {
            if (s == BS_OK) return;
            std::printf("%s on device %d: kv %d, %d units, d %d: %s\n", name, device, kv, units, dim, bs_status_string(s));
            ++fails;
          };
          const bool quant = kv == BS_E4M3 || kv == BS_INT8;
          const bs_pools pools{P(10), P(11), (float *)P(14), (float *)P(15)};
          for (float *w : {(float *)nullptr, (float *)P(7)}) {
            const bs_rope rope{(const double *)P(40), dim, 0, 1.0f, w, w, 1e-6f};
            check("bs_rope_append", bs_rope_append(&d, &rope, P(20), P(21), P(22), 16 * dim, 100, P(23), P(24), quant ? nullptr : &pools,
                                                   P(12), P(33), P(34), P(36), nullptr));
          }
          check("bs_tree_commit", bs_tree_commit(&d, &pools, P(12), P(13), P(2), P(3), P(4), 7, P(20), P(21), 16 * dim, 1000, P(36), nullptr));
          if (kv == BS_FP32) continue;
          for (int n : {1, 20, 60}) {      // the forms of 32, 128 and 256 rows
            const size_t pw = bs_prefill_workspace_size(&d, 1000, n), tw = bs_tree_workspace_size(&d, n);
            check("bs_prefill_attn", bs_prefill_attn(&d, P(20), 16 * dim, 1000, k, &c, P(2), P(3), n, P(33), (float *)P(34), P(35), pw,
                                                     P(36), nullptr));
            const bs_drafts dr{P(21), P(22), 16 * dim, 1000, P(3), P(4), (const uint64_t *)P(5), n};
            check("bs_tree_decode_attn", bs_tree_decode_attn(&d, P(20), 16 * dim, k, &c, P(27), P(28), &dr, P(33), nullptr, P(35), tw,
                                                             P(36), nullptr));
          }
        }
  std::printf("launches %d\nfails %d\n", g_launches, fails);
  return fails != 0;
}
"""

FILES = ["bs_rope.cu", "bs_rows.cuh", "bs_rows_attn.cuh", "bs_rows_mma.cuh", "bs_rows_attn.cu", "bs_umma.cuh"]


def test_every_form_runs_on_every_device(tmp_path):
    r = run_host(tmp_path, MAIN)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
    assert int(r.stdout.split("launches ")[1].split()[0]) >= 5 * 2 * 3 * (4 * 3 + 3 * 6)


@pytest.mark.parametrize("name", FILES)
def test_no_non_coherent_loads(name):
    """These kernels are in place before the work ahead of them has finished: see the other sources' test."""
    text = open(os.path.join(Bd.CSRC, name), encoding="utf-8").read()
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    assert not re.search(r"\b__ldg\s*\(|\.nc\b|__restrict__", text)
