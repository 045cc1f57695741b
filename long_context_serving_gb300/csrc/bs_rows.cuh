// Rows of new tokens: eight elements at a time from and to bf16 or fp32 memory.
#pragma once

#include "bs_quant.cuh"

namespace bsi {

// Eight elements from or to memory, fp32 (F32) or bf16.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *base, int64_t i) {
    const char *p = static_cast<const char *>(base) + i * (F32 ? 4 : 2);
    w[0] = ld_stream16(p);
    if constexpr (F32) w[1] = ld_stream16(p + 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (F32) {
      x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y); x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
      x[4] = __uint_as_float(w[1].x); x[5] = __uint_as_float(w[1].y); x[6] = __uint_as_float(w[1].z); x[7] = __uint_as_float(w[1].w);
    } else {
      x[0] = bf16lo(w[0].x); x[1] = bf16hi(w[0].x); x[2] = bf16lo(w[0].y); x[3] = bf16hi(w[0].y);
      x[4] = bf16lo(w[0].z); x[5] = bf16hi(w[0].z); x[6] = bf16lo(w[0].w); x[7] = bf16hi(w[0].w);
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t i, const float (&x)[8]) {
  char *p = static_cast<char *>(base) + i * (F32 ? 4 : 2);
  if constexpr (F32) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

}  // namespace bsi
