// Quantising append: new tokens' K and V into the pages of an 8-bit cache (the rule of
// scales and codes stands with bs_quant_append in bsattn.h).
//
// One warp per (page, K or V): a page is the unit of a scale, so the whole of its new rows
// sit in one warp's registers (16-byte loads, every row's in flight together), one warp
// reduction gives the largest magnitude, and the codes leave as full rows of 8-byte stores.
// One pass: each new value is read once, each code written once; bound by HBM for prompts,
// by latency for single tokens (one chain of lengths -> page index -> old scale).
#include "bs_quant.cuh"

namespace bsi {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;

struct AppendArgs {
  bs_dims dims;
  bs_pools pools;
  const int32_t *page_table, *seq_lens, *tok_begin, *row_begin;
  const void *k_new, *v_new;
  int64_t row_stride, n_rows;
  int32_t *st;
};

// Scale of a page whose largest finite magnitude is a.
template <bool I8>
__device__ __forceinline__ float page_scale(float a) {
  if (!(a > 0.0f)) return 0.0f;
  constexpr float kTiny = 1.17549435e-38f;   // 2^-126
  if (I8) return fmaxf(__fdiv_rn(a, 127.0f), kTiny);
  // a = 1.m * 2^k; 448 = 1.75 * 2^8: 2^(k - 8), doubled when 1.m > 1.75.
  const uint32_t bits = __float_as_uint(a);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

// Four codes of four quotients.
template <bool I8>
__device__ __forceinline__ uint32_t encode4(const float (&y)[4]) {
  if constexpr (I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (NaN: fmaxf / fminf would return the bound)
      const int q = y[i] == y[i] ? __float2int_rn(fminf(fmaxf(y[i], -127.0f), 127.0f)) : 0;
      w |= static_cast<uint32_t>(q & 0xff) << (8 * i);
    }
    return w;
  } else {
    uint32_t w;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return w;
  }
}

// x / s in fp32 for every value; a power-of-two s multiplies by its reciprocal (the same
// rounding of the same number).
struct Quotient {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale) {
    const uint32_t bits = __float_as_uint(scale);
    // 2^e with 2^-e normal: e in [-126, 126]
    pow2 = (bits & 0x7fffffu) == 0 && bits >= (1u << 23) && bits <= (253u << 23);
    inv = pow2 ? __uint_as_float((254u << 23) - bits) : 0.0f;
  }
  __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : __fdiv_rn(x, s); }
};

template <int D, bool I8, bool Q32>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanesPerRow = D / 8;              // 8 dimensions a lane
  constexpr int kRowsPerIter = 32 / kLanesPerRow;
  constexpr int kIters = kPage / kRowsPerIter;
  const bs_dims &dims = a.dims;
  const int u = blockIdx.x, b = u / dims.n_kv_heads, h = u % dims.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = a.seq_lens[b], t_begin = a.tok_begin[b];
  const bool first_warp = blockIdx.y == 0 && threadIdx.x == 0;
  if (t_begin < 0 || T < t_begin) {
    if (first_warp) report(a.st, BS_ERR_INVALID_ARG);
    return;
  }
  if (t_begin == T) return;
  if ((static_cast<int64_t>(T) + kPage - 1) / kPage > dims.max_pages_per_unit) {
    if (first_warp) report(a.st, BS_ERR_CAPACITY);
    return;
  }
  const int64_t row0 = a.row_begin[b];
  if (row0 < 0 || row0 + (T - t_begin) > a.n_rows) {
    if (first_warp) report(a.st, BS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int lp0 = t_begin / kPage, n_lp = (T - 1) / kPage - lp0 + 1;
  const int sub = lane / kLanesPerRow, col = lane % kLanesPerRow;
  for (int64_t item = static_cast<int64_t>(blockIdx.y) * kAppendWarps + warp; item < 2ll * n_lp;
       item += static_cast<int64_t>(gridDim.y) * kAppendWarps) {
    const int lp = lp0 + static_cast<int>(item >> 1);
    const bool is_v = item & 1;
    const int phys = a.page_table[static_cast<size_t>(u) * dims.max_pages_per_unit + lp];
    if (phys < 0 || phys >= dims.n_pages) {
      if (lane == 0) report(a.st, BS_ERR_DEVICE_BOUNDS);
      continue;
    }
    const int base = lp * kPage;
    const int s0 = max(t_begin - base, 0), s1 = min(T - base, kPage);   // slots of new tokens
    uint8_t *page = static_cast<uint8_t *>(is_v ? a.pools.v_pool : a.pools.k_pool) + static_cast<size_t>(phys) * (kPage * D);
    float *scale = (is_v ? a.pools.v_scale : a.pools.k_scale) + phys;
    const float had = s0 > 0 ? *scale : 0.0f;
    // ---- the new rows, every load in flight -----------------------------------------
    constexpr int kVecs = Q32 ? 2 : 1;
    uint4 raw[kIters][kVecs];
    const int64_t first = row0 + (base - t_begin);                       // row of slot 0
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int slot = i * kRowsPerIter + sub;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) raw[i][j] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= s0 && slot < s1) {
        const int64_t at = (first + slot) * a.row_stride + static_cast<int64_t>(h) * D + col * 8;
        const char *src = static_cast<const char *>(is_v ? a.v_new : a.k_new) + at * (Q32 ? 4 : 2);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) raw[i][j] = ldg_stream16(src + 16 * j);
      }
    }
    auto value = [&](int i, int j) -> float {       // value j (0..7) of iteration i
      if constexpr (Q32) {
        const uint4 w = raw[i][j >> 2];
        const uint32_t x = (j & 3) == 0 ? w.x : (j & 3) == 1 ? w.y : (j & 3) == 2 ? w.z : w.w;
        return __uint_as_float(x);
      } else {
        const uint4 w = raw[i][0];
        const uint32_t x = (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w;
        return (j & 1) ? bf16hi(x) : bf16lo(x);
      }
    };
    uint32_t big = 0u;   // magnitudes order like their bits
#pragma unroll
    for (int i = 0; i < kIters; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = __float_as_uint(value(i, j)) & 0x7fffffffu;
        big = max(big, m < 0x7f800000u ? m : 0u);
      }
    big = __reduce_max_sync(0xffffffffu, big);
    const float to = fmaxf(had, page_scale<I8>(__uint_as_float(big)));
    const Quotient quo(to);
    // ---- codes already there, at the new scale -----------------------------------------
    if (s0 > 0 && to > had) {
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const int slot = i * kRowsPerIter + sub;
        if (slot < s0) {
          uint2 *p = reinterpret_cast<uint2 *>(page + slot * D + col * 8);
          const uint2 old = *p;
          float f[4];
          uint2 now;
          codes_to_f32<I8>(old.x, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = quo(__fmul_rn(f[j], had));
          now.x = encode4<I8>(f);
          codes_to_f32<I8>(old.y, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = quo(__fmul_rn(f[j], had));
          now.y = encode4<I8>(f);
          *p = now;
        }
      }
    }
    // ---- the new codes ------------------------------------------------------------------
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int slot = i * kRowsPerIter + sub;
      if (slot >= s0 && slot < s1) {
        float f[4];
        uint2 now = make_uint2(0u, 0u);
        if (to > 0.0f) {
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = quo(value(i, j));
          now.x = encode4<I8>(f);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = quo(value(i, 4 + j));
          now.y = encode4<I8>(f);
        }
        *reinterpret_cast<uint2 *>(page + slot * D + col * 8) = now;
      }
    }
    if (lane == 0) *scale = to;
  }
}

template <int D, bool I8, bool Q32>
bs_status launch_append(const AppendArgs &a, int max_new, cudaStream_t cs) {
  const int units = a.dims.batch * a.dims.n_kv_heads;
  const int64_t items = 2 * ((static_cast<int64_t>(max_new) + kPage - 2) / kPage + 1);   // pages that max_new tokens can touch
  const int64_t gy = (items + kAppendWarps - 1) / kAppendWarps;
  append_kernel<D, I8, Q32><<<dim3(units, static_cast<unsigned>(gy < 65535 ? gy : 65535)), kAppendThreads, 0, cs>>>(a);
  return launch_status();
}

template <int D>
bs_status dispatch_types(const AppendArgs &a, int max_new, cudaStream_t cs) {
  const bool i8 = a.dims.kv_dtype == BS_INT8, q32 = a.dims.q_dtype == BS_FP32;
  if (i8) return q32 ? launch_append<D, true, true>(a, max_new, cs) : launch_append<D, true, false>(a, max_new, cs);
  return q32 ? launch_append<D, false, true>(a, max_new, cs) : launch_append<D, false, false>(a, max_new, cs);
}

}  // namespace
}  // namespace bsi

extern "C" bs_status bs_quant_append(const bs_dims *dims, const bs_pools *pools, const int32_t *page_table,
                                     const int32_t *seq_lens, const int32_t *tok_begin, const int32_t *row_begin,
                                     const void *k_new, const void *v_new, int64_t row_stride, int64_t n_rows,
                                     int32_t max_new_tokens, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (!is_quant(dims->kv_dtype)) return BS_ERR_INVALID_ARG;
  if (!pools || !pools->k_pool || !pools->v_pool || !pools->k_scale || !pools->v_scale || !page_table || !seq_lens ||
      !tok_begin || !row_begin || !k_new || !v_new || !dev_status)
    return BS_ERR_INVALID_ARG;
  if (n_rows < 0 || max_new_tokens < 1) return BS_ERR_INVALID_ARG;
  if (row_stride < static_cast<int64_t>(dims->n_kv_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(pools->k_pool) || !aligned16(pools->v_pool) || !aligned16(k_new) || !aligned16(v_new) ||
      row_stride % (dims->q_dtype == BS_FP32 ? 4 : 8) != 0)
    return BS_ERR_ALIGN;
  AppendArgs a{*dims, *pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status};
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return dims->head_dim == 128 ? dispatch_types<128>(a, max_new_tokens, cs) : dispatch_types<64>(a, max_new_tokens, cs);
}
