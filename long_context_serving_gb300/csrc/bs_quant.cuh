// 8-bit codes of the quantised caches (E4M3 and INT8): conversions shared by the append,
// the sub-block summaries and the attention.
#pragma once

#include <cuda_fp16.h>

#include "bs_internal.cuh"

namespace bsi {

__host__ __device__ __forceinline__ bool is_quant(int kv_dtype) { return kv_dtype == BS_E4M3 || kv_dtype == BS_INT8; }

// The caller's struct; its scales, which it did not always have, are read for 8-bit caches only.
inline bs_kv kv_of(const bs_dims &dims, const bs_kv *kv) {
  bs_kv k{kv->k_pool, kv->v_pool, kv->page_table, kv->seq_lens, nullptr, nullptr};
  if (is_quant(dims.kv_dtype)) {
    k.k_scale = kv->k_scale;
    k.v_scale = kv->v_scale;
  }
  return k;
}

// A load of data read once, from L2. (Neither ld.global.nc nor an L1 line: a kernel that is in
// place before the work ahead of it has finished reads what that wrote.)
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
  uint4 w;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p)
               : "memory");
  return w;
}

// Four codes of a word as two fp16 pairs (exact): bytes 0, 1 in lo, bytes 2, 3 in hi.
template <bool I8>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (I8) {
    // c + 128 as the low mantissa bits of 1024 + (c + 128), less 1152.
    const uint32_t x = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
    const __half2 hb = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&ha);
    hi = *reinterpret_cast<const uint32_t *>(&hb);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Four codes as floats (exact).
template <bool I8>
__device__ __forceinline__ void codes_to_f32(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  codes_to_f16<I8>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

}  // namespace bsi
