// Norm, rotation and cache write of new tokens' queries and keys (formulas with bs_rope_append
// in bsattn.h), one pass: every element is read once and written once.
//
// A row is the heads of one token, and all of them turn by the same angles. A lane holds 16
// elements of a head, the eight pairs that it turns, so a rotation needs no exchange and a norm
// three shuffles (head_dim / 16 lanes a head); it keeps the pairs' cosines and sines in registers
// while its warp walks the row's heads, four (d = 128) or eight (d = 64) at a time. Few rows are
// split over several warps each.
// Loads of the next heads fly beside this turn's work, a row's first ones beside its angles. Bound by
// HBM in prompts (29K rows of 28 + 8 heads, bf16: 97 us, 5.5 TB/s, with norms 99; fp32 6.25 TB/s), by one
// chain of loads in decode steps (64 rows with norms, 3.1 us in a graph).
// Angles: position * inv_freq in turns, inv_freq / 2 pi, less its whole turns, held as two floats (high
// and low part, from one fp64 product a frequency and block), the product's rounding error taken back by
// an fma: the fraction of a turn is right to 2^-24 at any position below 2^24 for frequencies of up to
// a radian (parts of 1/4 a turn: roundings of 2^-25, 2^-27 and less), to 2^-23 up to 32 radians (parts of 1/2 a turn
// and fp64's own 2^-52 of the angle), without fp64 in the loop (fp64 runs at 1/64 of fp32's rate here).
#include "bs_attn_launch.cuh"
#include "bs_rows.cuh"

namespace bsi {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kMaxPosition = 1 << 24;   // positions are exact in fp32

struct RopeArgs {
  bs_dims dims;
  bs_rope rope;
  const void *q, *k, *v;
  int64_t row_stride, n_rows;
  const int32_t *positions, *row_seq;
  void *k_pool, *v_pool;   // null: no cache
  const int32_t *page_table;
  void *q_out, *k_out;
  int32_t parts;           // warps that share a row
  int32_t *st;
};

// Q32, C32: rows and outputs, cache in fp32 (else bf16). kNorm: with norms (of queries, keys or both).
template <int D, bool Q32, bool C32, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, Q32 ? 2 : 3) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16;          // lanes a head
  constexpr int kHeads = 32 / kLanes;     // heads a warp takes at once
  const bs_dims &dims = a.dims;
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int rot = a.rope.rot_dim;
  const bool inter = a.rope.interleaved != 0;
  __shared__ float2 turns[D / 2];         // inv_freq / 2 pi: high part, low part
  asm volatile("griddepcontrol.wait;" ::: "memory");      // everything before this call has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x < rot / 2) {
    const double turn = a.rope.inv_freq[threadIdx.x] * 0.15915494309189533577;   // 1 / (2 pi)
    const double f = turn - rint(turn);           // (positions are whole: whole turns fall out)
    const float hi = static_cast<float>(f);
    turns[threadIdx.x] = make_float2(hi, static_cast<float>(f - hi));
  }
  // This lane's elements of a head: [ea, ea + 8) and [eb, eb + 8); pairs 8l .. 8l + 7 where it
  // lies in the rotated part.
  const bool turning = l < rot / 16;
  const int ea = turning && !inter ? 8 * l : 16 * l;
  const int eb = turning && !inter ? rot / 2 + 8 * l : 16 * l + 8;
  const bool norm_q = kNorm && a.rope.q_weight != nullptr, norm_k = kNorm && a.rope.k_weight != nullptr;
  __shared__ __align__(16) float weights[kNorm ? 2 : 1][kNorm ? D : 4];   // of queries, of keys (registers hold no room for them)
  if constexpr (kNorm) {
    for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
      const float *w = i < D ? a.rope.q_weight : a.rope.k_weight;
      weights[i / D][i % D] = w != nullptr ? w[i % D] : 1.0f;
    }
  }
  __syncthreads();
  const int Hq = dims.n_q_heads, Hkv = dims.n_kv_heads;
  const bool cache = a.k_pool != nullptr;
  const int n_heads = Hq + Hkv + (cache ? Hkv : 0), step = a.parts * kHeads;
  const int64_t n_items = a.n_rows * a.parts;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kRopeWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5); item < n_items; item += n_warps) {
    const int64_t row = a.parts == 1 ? item : item / a.parts;
    const int part = a.parts == 1 ? 0 : static_cast<int>(item - row * a.parts);
    const int b = a.row_seq != nullptr ? a.row_seq[row] : 0;
    const int pos = a.positions[row];
    const int64_t row_at = row * a.row_stride;
    // The heads of one turn: this lane's, and its elements on their way.
    struct Head {
      int head;
      Raw8<Q32> a, b;
    };
    auto fetch = [&](int h0) -> Head {
      Head x{};
      x.head = h0 + sub;
      if (x.head < n_heads) {
        const void *src = x.head < Hq ? a.q : x.head < Hq + Hkv ? a.k : a.v;
        const int64_t at = row_at + static_cast<int64_t>(x.head < Hq ? x.head : x.head < Hq + Hkv ? x.head - Hq : x.head - Hq - Hkv) * D;
        x.a.load(src, at + ea);
        x.b.load(src, at + eb);
      }
      return x;
    };
    Head next = fetch(part * kHeads);     // (beside the row's position and its angles)
    if (b < 0) continue;                  // padding
    int bad = 0;
    if (pos < 0 || pos >= kMaxPosition) bad = BS_ERR_INVALID_ARG;
    else if (a.row_seq != nullptr && b >= dims.batch) bad = BS_ERR_DEVICE_BOUNDS;
    else if (cache && pos / kPage >= dims.max_pages_per_unit) bad = BS_ERR_CAPACITY;
    if (bad != 0) {
      if (lane == 0 && part == 0) report(a.st, bad);
      continue;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = 1.0f;
      sn[j] = 0.0f;
    }
    if (turning) {
      const float p = static_cast<float>(pos);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = turns[8 * l + j];
        const float t = p * f.x;
        const float low = fmaf(p, f.y, fmaf(p, f.x, -t));
        const float r = (t - rintf(t)) + low;
        sincospif(2.0f * r, &sn[j], &cs[j]);
        sn[j] *= a.rope.magnitude;
        cs[j] *= a.rope.magnitude;
      }
    }
    for (int h0 = part * kHeads; h0 < n_heads; h0 += step) {
      const Head x = next;
      next = fetch(h0 + step < n_heads ? h0 + step : n_heads);   // (past the last: nothing)
      const int head = x.head;
      const bool live = head < n_heads, is_q = head < Hq, is_v = head >= Hq + Hkv;
      const int hk = is_q ? 0 : is_v ? head - Hq - Hkv : head - Hq;
      int page = 0;
      if (cache && live && !is_q)
        page = a.page_table[(static_cast<int64_t>(b) * Hkv + hk) * dims.max_pages_per_unit + pos / kPage];
      float xa[8], xb[8];
      x.a.get(xa);
      x.b.get(xb);
      if constexpr (kNorm) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], sum));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (is_q ? norm_q : (!is_v && norm_k)) {
          const float inv = rsqrtf(fmaf(sum, 1.0f / D, a.rope.eps));
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 wa = *reinterpret_cast<const float4 *>(&weights[is_q ? 0 : 1][ea + j]);
            const float4 wb = *reinterpret_cast<const float4 *>(&weights[is_q ? 0 : 1][eb + j]);
            xa[j] *= inv * wa.x; xa[j + 1] *= inv * wa.y; xa[j + 2] *= inv * wa.z; xa[j + 3] *= inv * wa.w;
            xb[j] *= inv * wb.x; xb[j + 1] *= inv * wb.y; xb[j + 2] *= inv * wb.z; xb[j + 3] *= inv * wb.w;
          }
        }
      }
      if (turning && !is_v) {
        if (inter) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float &u = j < 4 ? xa[2 * j] : xb[2 * j - 8];
            float &w = j < 4 ? xa[2 * j + 1] : xb[2 * j - 7];
            const float u0 = u, w0 = w;
            u = fmaf(u0, cs[j], -(w0 * sn[j]));
            w = fmaf(w0, cs[j], u0 * sn[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float u = xa[j], w = xb[j];
            xa[j] = fmaf(u, cs[j], -(w * sn[j]));
            xb[j] = fmaf(w, cs[j], u * sn[j]);
          }
        }
      }
      if (!live) continue;
      if (is_q) {
        const int64_t to = (row * Hq + head) * D;
        store8<Q32>(a.q_out, to + ea, xa);
        store8<Q32>(a.q_out, to + eb, xb);
        continue;
      }
      if (!is_v && a.k_out != nullptr) {
        const int64_t to = (row * Hkv + hk) * D;
        store8<Q32>(a.k_out, to + ea, xa);
        store8<Q32>(a.k_out, to + eb, xb);
      }
      if (cache) {
        if (page < 0 || page >= dims.n_pages) {
          if (l == 0) report(a.st, BS_ERR_DEVICE_BOUNDS);
          continue;
        }
        const int64_t to = (static_cast<int64_t>(page) * kPage + pos % kPage) * D;
        store8<C32>(is_v ? a.v_pool : a.k_pool, to + ea, xa);
        store8<C32>(is_v ? a.v_pool : a.k_pool, to + eb, xb);
      }
    }
  }
}

template <int D, bool Q32, bool C32>
bs_status launch_rope(RopeArgs &a, cudaStream_t cs) {
  constexpr int kHeads = 512 / D;
  const int groups = (a.dims.n_q_heads + 2 * a.dims.n_kv_heads + kHeads - 1) / kHeads;
  const bool norm = a.rope.q_weight != nullptr || a.rope.k_weight != nullptr;
  const int64_t most = static_cast<int64_t>(attn_target_ctas()) / 2 * (Q32 ? 2 : 3);   // CTAs that are on the GPU at once
  // A row's angles are worth about one group of its heads: it is shared out only while warps lack work.
  const int64_t spare = most * kRopeWarps / a.n_rows;
  a.parts = static_cast<int>(spare < 1 ? 1 : spare < groups ? spare : groups);
  const int64_t ctas = (a.n_rows * a.parts + kRopeWarps - 1) / kRopeWarps;
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
  auto kernel = norm ? rope_kernel<D, Q32, C32, true> : rope_kernel<D, Q32, C32, false>;
  return launch_ex(kernel, grid, kRopeThreads, 0, cs, 0, true, a) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

template <int D>
bs_status dispatch_types(RopeArgs &a, cudaStream_t cs) {
  const bool q32 = a.dims.q_dtype == BS_FP32, c32 = a.dims.kv_dtype == BS_FP32;
  if (q32) return c32 ? launch_rope<D, true, true>(a, cs) : launch_rope<D, true, false>(a, cs);
  return c32 ? launch_rope<D, false, true>(a, cs) : launch_rope<D, false, false>(a, cs);
}

}  // namespace
}  // namespace bsi

extern "C" bs_status bs_rope_append(const bs_dims *dims, const bs_rope *rope, const void *q, const void *k,
                                    const void *v, int64_t row_stride, int64_t n_rows, const int32_t *positions,
                                    const int32_t *row_seq, const bs_pools *pools, const int32_t *page_table,
                                    void *q_out, void *k_out, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (n_rows < 0 || n_rows > (int64_t(1) << 40)) return BS_ERR_INVALID_ARG;
  const bool some = n_rows > 0;      // (arrays of no rows have no address)
  if (!rope || !rope->inv_freq || !dev_status || (some && (!q || !k || !positions || !q_out))) return BS_ERR_INVALID_ARG;
  if (pools != nullptr) {
    if (is_quant(dims->kv_dtype)) return BS_ERR_INVALID_ARG;
    if (!pools->k_pool || !pools->v_pool || !page_table || (some && (!row_seq || !v))) return BS_ERR_INVALID_ARG;
  } else if (some && !k_out) {
    return BS_ERR_INVALID_ARG;
  }
  if (rope->rot_dim < 16 || rope->rot_dim > dims->head_dim || rope->rot_dim % 16 != 0) return BS_ERR_SHAPE;
  if (rope->interleaved != 0 && rope->interleaved != 1) return BS_ERR_INVALID_ARG;
  // (written so that NaN fails too)
  if (!(rope->eps >= 0.0f && rope->eps <= 3.4e38f) || !(rope->magnitude >= -3.4e38f && rope->magnitude <= 3.4e38f))
    return BS_ERR_INVALID_ARG;
  if (row_stride < static_cast<int64_t>(dims->n_q_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || (pools && (!aligned16(v) || !aligned16(pools->k_pool) || !aligned16(pools->v_pool))) ||
      !aligned16(q_out) || (k_out && !aligned16(k_out)) || row_stride % (dims->q_dtype == BS_FP32 ? 4 : 8) != 0 ||
      reinterpret_cast<uintptr_t>(rope->inv_freq) % 8 != 0)
    return BS_ERR_ALIGN;
  if (n_rows == 0) return BS_OK;
  RopeArgs a{};
  a.dims = *dims;
  a.rope = *rope;
  a.q = q;
  a.k = k;
  a.v = v;
  a.row_stride = row_stride;
  a.n_rows = n_rows;
  a.positions = positions;
  a.row_seq = row_seq;
  if (pools != nullptr) {
    a.k_pool = pools->k_pool;
    a.v_pool = pools->v_pool;
    a.page_table = page_table;
  }
  a.q_out = q_out;
  a.k_out = k_out;
  a.st = dev_status;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return dims->head_dim == 128 ? dispatch_types<128>(a, cs) : dispatch_types<64>(a, cs);
}
