// Quantising append: new tokens' K and V into the pages of an 8-bit cache (the rule of
// scales and codes stands with bs_quant_append in bsattn.h).
//
// One warp per (page, K or V): a page is the unit of a scale, so the whole of its new rows
// sit in one warp's registers (16-byte loads, every row's in flight together), one warp
// reduction gives the largest magnitude, and the codes leave as full rows of 8-byte stores.
// One pass: each new value is read once, each code written once. Prompts are bound by HBM and by
// instruction issue together (53.7K tokens of 8 heads, bf16 to INT8: 64.5 us, 5.1 TB/s, issue
// slots 69 % busy; 59 us if no quotient ever lay next to a half), single tokens by latency (64
// sequences of 8 heads: 2.9 us; one chain of lengths -> page index -> rows and old scale).
#include "bs_attn_launch.cuh"
#include "bs_quant.cuh"
#include "bs_rows.cuh"

namespace bsi {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct AppendArgs {
  bs_dims dims;
  bs_pools pools;
  const int32_t *page_table, *seq_lens, *tok_begin, *row_begin;
  const void *k_new, *v_new;
  int64_t row_stride, n_rows;
  int32_t *st;
  const int32_t *path;   // bs_tree_commit: [batch][path_stride], the row of each new token; else null
  int32_t path_stride;
};

// Do the accepted drafts of a sequence fit? False: nothing to do (none, or they do not fit, which
// `first` reports). All lanes of a warp call it together.
__device__ __forceinline__ bool path_fits(const AppendArgs &a, int b, bool first, int T, int t_begin, int64_t row0) {
  int bad = 0;
  if (t_begin < 0 || T < t_begin) bad = BS_ERR_INVALID_ARG;
  else if (t_begin == T) return false;
  else if ((static_cast<int64_t>(T) + kPage - 1) / kPage > a.dims.max_pages_per_unit) bad = BS_ERR_CAPACITY;
  else if (T - t_begin > a.path_stride) bad = BS_ERR_CAPACITY;
  else if (row0 < 0 || row0 > a.n_rows) bad = BS_ERR_DEVICE_BOUNDS;
  if (bad == 0) {
    bool out = false;
    for (int i = threadIdx.x & 31; i < T - t_begin; i += 32) {
      const int node = a.path[static_cast<int64_t>(b) * a.path_stride + i];
      out |= node < 0 || row0 + node >= a.n_rows;
    }
    if (__any_sync(0xffffffffu, out)) bad = BS_ERR_DEVICE_BOUNDS;
  }
  if (bad != 0 && first) report(a.st, bad);
  return bad == 0;
}

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

// Codes of eight quotients x / s in fp32 by the rule of bs_quant_append, for any values.
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
// (Out of line: rarely taken, and its divisions are long.)
template <bool I8>
__device__ __noinline__ uint2 encode8_any(float4 a, float4 b, float s) {
  const float x[4] = {__fdiv_rn(a.x, s), __fdiv_rn(a.y, s), __fdiv_rn(a.z, s), __fdiv_rn(a.w, s)};
  const float y[4] = {__fdiv_rn(b.x, s), __fdiv_rn(b.y, s), __fdiv_rn(b.z, s), __fdiv_rn(b.w, s)};
  return make_uint2(encode4<I8>(x), encode4<I8>(y));
}
template <bool I8>
__device__ __forceinline__ uint2 encode8_any(const float (&x)[8], float s) {
  return encode8_any<I8>(make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]), s);
}

// The same without divisions, for finite x with |x| <= top * s (top 448 or 127) when `exact`.
// E4M3: a power-of-two s multiplies by its reciprocal, the same rounding of the same number.
// INT8: n = rint(x * inv), inv = fp32(1 / s), differs from the rule only where the quotient
// is next to a half: |x inv - x / s| <= 2^-17 and the quotient's own rounding is at most
// 2^-18 for |x / s| < 128, so a lane with a value within 2^-15 of a half divides. (bf16 has
// many: half a page's largest value is one. Dividing that value alone, not the lane's eight,
// was no faster, 64.3 us for 64.4, and settling the halves by their exact residuals in line,
// without a division, slower: 67.2.)
template <bool I8>
struct Encoder {
  float s, inv;
  bool exact;
  __device__ __forceinline__ Encoder(float scale, bool finite) : s(scale) {
    const uint32_t bits = __float_as_uint(scale);
    // A normal scale whose reciprocal is normal too.
    const bool normal = bits >= (1u << 23) && bits <= (252u << 23);
    inv = normal ? __frcp_rn(scale) : 0.0f;
    exact = finite && normal && (I8 || (bits & 0x7fffffu) == 0);
  }
  __device__ __forceinline__ uint2 operator()(const float (&x)[8]) const {
    if (!exact) return encode8_any<I8>(x, s);
    uint2 w;
    if constexpr (I8) {
      constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: the sum's low bits are the integer
      uint32_t n[8];
      float off = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = fmaf(x[j], inv, kMagic);
        n[j] = __float_as_uint(t);
        off = fmaxf(off, fabsf(fmaf(x[j], inv, -(t - kMagic))));
      }
      if (off > 0.5f - 0x1p-15f) return encode8_any<I8>(x, s);
      w.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
      w.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
    } else {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = x[j] * inv;
      w.x = encode4<I8>(y);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = x[4 + j] * inv;
      w.y = encode4<I8>(y);
    }
    return w;
  }
};

// The page item `it` of a unit: logical page lp0 + it / 2, K (even) or V (odd).
// Eight CTAs an SM for bf16 rows: 64 registers, at d = 128 with 40 bytes of them spilled a
// thread; seven CTAs (72 registers, 12 bytes spilled) took 65.9 us for the prompts above, six
// 68.1. fp32 rows are twice the registers (166 at d = 128, none spilled); not timed.
// kPath: new tokens' rows are those that the path names (bs_tree_commit).
template <int D, bool I8, bool Q32, bool kPath>
__global__ void __launch_bounds__(kAppendThreads, Q32 ? (D == 128 ? 3 : 5) : 8) append_kernel(const __grid_constant__ AppendArgs a, int per_warp) {
  constexpr int kLanesPerRow = D / 8;              // 8 dimensions a lane
  constexpr int kRowsPerIter = 32 / kLanesPerRow;
  constexpr int kIters = kPage / kRowsPerIter;
  const bs_dims &dims = a.dims;
  const int u = blockIdx.x, b = u / dims.n_kv_heads, h = u % dims.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();      // everything before this call has finished
  pdl_trigger();
  const int T = a.seq_lens[b], t_begin = a.tok_begin[b];
  const int64_t row0 = a.row_begin[b];
  const bool first_thread = blockIdx.y == 0 && threadIdx.x == 0;
  if constexpr (kPath) {
    if (!path_fits(a, b, first_thread, T, t_begin, row0)) return;
  } else {      // (in line: through a function of both forms 48 bytes are spilled, 66.2 us for 65.6)
    if (t_begin < 0 || T < t_begin) {
      if (first_thread) report(a.st, BS_ERR_INVALID_ARG);
      return;
    }
    if (t_begin == T) return;
    if ((static_cast<int64_t>(T) + kPage - 1) / kPage > dims.max_pages_per_unit) {
      if (first_thread) report(a.st, BS_ERR_CAPACITY);
      return;
    }
    if (row0 < 0 || row0 + (T - t_begin) > a.n_rows) {
      if (first_thread) report(a.st, BS_ERR_DEVICE_BOUNDS);
      return;
    }
  }
  const int lp0 = t_begin / kPage;
  const int64_t n_items = 2ll * ((T - 1) / kPage - lp0 + 1);
  const int sub = lane / kLanesPerRow, col = lane % kLanesPerRow;
  const int32_t *pt = a.page_table + static_cast<size_t>(u) * dims.max_pages_per_unit;
  const int64_t stride = static_cast<int64_t>(gridDim.y) * kAppendWarps * per_warp;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.y) * kAppendWarps + warp) * per_warp; i0 < n_items; i0 += stride)
    for (int64_t item = i0; item < i0 + per_warp && item < n_items; ++item) {
    const int lp = lp0 + static_cast<int>(item >> 1);
    const bool is_v = item & 1;
    const int phys = pt[lp];
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
    const char *src = static_cast<const char *>(is_v ? a.v_new : a.k_new) +
                      ((kPath ? row0 : first + sub) * a.row_stride + static_cast<int64_t>(h) * D + col * 8) * (Q32 ? 4 : 2);
    const int64_t step = kRowsPerIter * a.row_stride * (Q32 ? 4 : 2);
    const int32_t *nodes = kPath ? a.path + static_cast<int64_t>(b) * a.path_stride + (base - t_begin) : nullptr;   // of slot 0
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int slot = i * kRowsPerIter + sub;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) raw[i][j] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= s0 && slot < s1) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
          raw[i][j] = ld_stream16(src + (kPath ? nodes[slot] * a.row_stride * (Q32 ? 4 : 2) : i * step) + 16 * j);
      }
    }
    auto values = [&](int i, float (&x)[8]) {
      if constexpr (Q32) {
        x[0] = __uint_as_float(raw[i][0].x); x[1] = __uint_as_float(raw[i][0].y);
        x[2] = __uint_as_float(raw[i][0].z); x[3] = __uint_as_float(raw[i][0].w);
        x[4] = __uint_as_float(raw[i][1].x); x[5] = __uint_as_float(raw[i][1].y);
        x[6] = __uint_as_float(raw[i][1].z); x[7] = __uint_as_float(raw[i][1].w);
      } else {
        x[0] = bf16lo(raw[i][0].x); x[1] = bf16hi(raw[i][0].x); x[2] = bf16lo(raw[i][0].y); x[3] = bf16hi(raw[i][0].y);
        x[4] = bf16lo(raw[i][0].z); x[5] = bf16hi(raw[i][0].z); x[6] = bf16lo(raw[i][0].w); x[7] = bf16hi(raw[i][0].w);
      }
    };
    // The largest magnitude: bits order like magnitudes, bf16 pairs are compared two at a time,
    // and only a page with a non-finite value looks again, without those. keep(word): the
    // magnitudes of a word that count.
    auto largest = [&](auto keep) -> uint32_t {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < kIters; ++i)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const uint4 w = raw[i][j];
          if constexpr (Q32) m = max(m, max(max(keep(w.x), keep(w.y)), max(keep(w.z), keep(w.w))));
          else m = __vmaxu2(m, __vmaxu2(__vmaxu2(keep(w.x), keep(w.y)), __vmaxu2(keep(w.z), keep(w.w))));
        }
      if constexpr (!Q32) m = max(m << 16, m & 0xffff0000u);
      return __reduce_max_sync(0xffffffffu, m);
    };
    uint32_t big = largest([](uint32_t w) { return w & (Q32 ? 0x7fffffffu : 0x7fff7fffu); });
    const bool finite = big < 0x7f800000u;
    if (!finite)
      big = largest([](uint32_t w) {
        if constexpr (Q32) {
          const uint32_t m = w & 0x7fffffffu;
          return m < 0x7f800000u ? m : 0u;
        } else {
          const uint32_t m = w & 0x7fff7fffu;
          return m & __vcmpltu2(m, 0x7f807f80u);
        }
      });
    const float to = fmaxf(had, page_scale<I8>(__uint_as_float(big)));
    const Encoder<I8> enc(to, finite);
    // ---- codes already there, at the new scale (divisions for E4M3 too; one page a unit) ---
    if (s0 > 0 && to > had) {
#pragma unroll 1
      for (int slot = sub; slot < s0; slot += kRowsPerIter) {
        uint2 *p = reinterpret_cast<uint2 *>(page + slot * D + col * 8);
        const uint2 old = *p;
        float f[8], lo[4], hi[4];
        codes_to_f32<I8>(old.x, lo);
        codes_to_f32<I8>(old.y, hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = __fmul_rn(lo[j], had);
          f[4 + j] = __fmul_rn(hi[j], had);
        }
        *p = encode8_any<I8>(f, to);
      }
    }
    // ---- the new codes ------------------------------------------------------------------
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int slot = i * kRowsPerIter + sub;
      if (slot >= s0 && slot < s1) {
        float x[8];
        values(i, x);
        *reinterpret_cast<uint2 *>(page + slot * D + col * 8) = to > 0.0f ? enc(x) : make_uint2(0u, 0u);
      }
    }
    if (lane == 0) *scale = to;
  }
}

// Into a cache that is not quantised (bs_tree_commit): eight elements a thread, one CTA a unit.
// A few rows; the launch and one chain of loads (lengths, path entry, page and row) are its time: 1.9 us
// in a graph (E4M3, 64 sequences of 8 heads, through append_kernel: 3.8).
template <int D, bool Q32, bool C32>
__global__ void __launch_bounds__(kAppendThreads) commit_rows_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kVecs = D / 8;
  const int u = blockIdx.x, b = u / a.dims.n_kv_heads, h = u % a.dims.n_kv_heads;
  pdl_wait();      // everything before this call has finished
  pdl_trigger();
  const int T = a.seq_lens[b], t_begin = a.tok_begin[b];
  const int64_t row0 = a.row_begin[b];
  if (!path_fits(a, b, threadIdx.x == 0, T, t_begin, row0)) return;
  const int32_t *pt = a.page_table + static_cast<size_t>(u) * a.dims.max_pages_per_unit;
  for (int i = threadIdx.x; i < (T - t_begin) * 2 * kVecs; i += kAppendThreads) {
    const int n = i / (2 * kVecs), at = i % kVecs, t = t_begin + n;
    const bool is_v = (i / kVecs) % 2 != 0;
    const int phys = pt[t / kPage];
    if (phys < 0 || phys >= a.dims.n_pages) {
      report(a.st, BS_ERR_DEVICE_BOUNDS);
      continue;
    }
    const int64_t row = row0 + a.path[static_cast<int64_t>(b) * a.path_stride + n];
    Raw8<Q32> raw;
    raw.load(is_v ? a.v_new : a.k_new, row * a.row_stride + static_cast<int64_t>(h) * D + at * 8);
    float x[8];
    raw.get(x);
    store8<C32>(is_v ? a.pools.v_pool : a.pools.k_pool, (static_cast<int64_t>(phys) * kPage + t % kPage) * D + at * 8, x);
  }
}

// Pages a warp takes in turn: one (K or V) while that keeps the launch short; four for long
// prompts, where a CTA's start is worth several pages.
template <int D, bool I8, bool Q32, bool kPath>
bs_status launch_append(const AppendArgs &a, int max_new, cudaStream_t cs) {
  const int units = a.dims.batch * a.dims.n_kv_heads;
  const int64_t items = 2 * ((static_cast<int64_t>(max_new) + kPage - 2) / kPage + 1);   // pages that max_new tokens can touch
  const int per_warp = units * items > 8 * 152 * kAppendWarps ? 4 : 1;
  const int64_t gy = (items + kAppendWarps * per_warp - 1) / (kAppendWarps * per_warp);
  // (a programmatic dependent: its CTAs are in place when the work before it ends)
  const dim3 grid(units, static_cast<unsigned>(gy < 65535 ? gy : 65535));
  return launch_ex(append_kernel<D, I8, Q32, kPath>, grid, kAppendThreads, 0, cs, 0, true, a, per_warp) == cudaSuccess ? BS_OK
                                                                                                                : BS_ERR_CUDA;
}

template <int D, bool kPath>
bs_status dispatch_types(const AppendArgs &a, int max_new, cudaStream_t cs) {
  const bool i8 = a.dims.kv_dtype == BS_INT8, q32 = a.dims.q_dtype == BS_FP32;
  if (i8) return q32 ? launch_append<D, true, true, kPath>(a, max_new, cs) : launch_append<D, true, false, kPath>(a, max_new, cs);
  return q32 ? launch_append<D, false, true, kPath>(a, max_new, cs) : launch_append<D, false, false, kPath>(a, max_new, cs);
}

template <int D>
bs_status commit_rows(const AppendArgs &a, cudaStream_t cs) {
  const bool q32 = a.dims.q_dtype == BS_FP32, c32 = a.dims.kv_dtype == BS_FP32;
  auto kernel = q32 ? (c32 ? commit_rows_kernel<D, true, true> : commit_rows_kernel<D, true, false>)
                    : (c32 ? commit_rows_kernel<D, false, true> : commit_rows_kernel<D, false, false>);
  const dim3 grid(a.dims.batch * a.dims.n_kv_heads);
  return launch_ex(kernel, grid, kAppendThreads, 0, cs, 0, true, a) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

// Host checks that both appends share (after those of the dims). Arrays of no rows have no address.
bs_status check_append(const bs_dims *dims, const bs_pools *pools, const void *page_table, const void *seq_lens,
                       const void *tok_begin, const void *row_begin, const void *k_new, const void *v_new,
                       int64_t row_stride, int64_t n_rows, const void *dev_status) {
  if (!pools || !pools->k_pool || !pools->v_pool || !page_table || !seq_lens || !tok_begin || !row_begin || !dev_status ||
      (n_rows != 0 && (!k_new || !v_new)))
    return BS_ERR_INVALID_ARG;
  if (is_quant(dims->kv_dtype) && (!pools->k_scale || !pools->v_scale)) return BS_ERR_INVALID_ARG;
  if (n_rows < 0 || row_stride < static_cast<int64_t>(dims->n_kv_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(pools->k_pool) || !aligned16(pools->v_pool) || !aligned16(k_new) || !aligned16(v_new) ||
      row_stride % (dims->q_dtype == BS_FP32 ? 4 : 8) != 0)
    return BS_ERR_ALIGN;
  return BS_OK;
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
  if (max_new_tokens < 1) return BS_ERR_INVALID_ARG;
  s = check_append(dims, pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status);
  if (s != BS_OK) return s;
  AppendArgs a{*dims, *pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status, nullptr, 0};
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return dims->head_dim == 128 ? dispatch_types<128, false>(a, max_new_tokens, cs) : dispatch_types<64, false>(a, max_new_tokens, cs);
}

extern "C" bs_status bs_tree_commit(const bs_dims *dims, const bs_pools *pools, const int32_t *page_table,
                                    const int32_t *seq_lens, const int32_t *tok_begin, const int32_t *row_begin,
                                    const int32_t *path, int32_t path_stride, const void *k_new, const void *v_new,
                                    int64_t row_stride, int64_t n_rows, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (!path || path_stride < 1 || path_stride > BS_MAX_DRAFT) return BS_ERR_INVALID_ARG;
  s = check_append(dims, pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status);
  if (s != BS_OK) return s;
  // (the scales of a cache that has none are not the kernel's to see)
  bs_pools to{pools->k_pool, pools->v_pool, nullptr, nullptr};
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (!is_quant(dims->kv_dtype)) {
    AppendArgs a{*dims, to, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status, path, path_stride};
    return dims->head_dim == 128 ? commit_rows<128>(a, cs) : commit_rows<64>(a, cs);
  }
  AppendArgs a{*dims, *pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride, n_rows, dev_status, path, path_stride};
  return dims->head_dim == 128 ? dispatch_types<128, true>(a, path_stride, cs) : dispatch_types<64, true>(a, path_stride, cs);
}
