// Attention over 8-bit caches (E4M3 or INT8 codes, one fp32 scale per page for K and one
// for V): the kernels and their launcher. The unit's block list, the split plan and the
// merges are those of the other caches (bs_attn_impl.cuh); only the page math differs.
//
// With ks, vs the scales of token t's page and K8, V8 its codes:
//   x_h(t) = ks (q_h . K8[t]) / sqrt(d) + e,   o_h += vs (exp(x_h(t) - m) V8[t]).
//
// Logits and maxima are kept as they are, not times log2(e), so that every finite block logit e
// counts (the type's lowest times log2(e) would be -inf); log2(e) enters x - m, whose
// exponential is 2 to that power.
//
// A warp takes whole pages, two at a time, through two buffers of its own in shared memory,
// one for a pair's K and one for its V, filled by 16-byte asynchronous copies (cp.async) and
// drained without a CTA barrier. K of the next pair is in flight from the end of this pair's
// scores, its V from the end of this pair's values: 4 to 8 KB a warp, eight warps an SM. (Rings
// of two and three pairs were slower, as were codes loaded straight into registers.)
// Rows are stored with their 16-byte chunks permuted (swz8), so that the reads below are free
// of bank conflicts (D = 64: V two-way). Fragment layouts are chosen around 16-byte reads;
// lane = 4 r + c:
//   K: lane reads chunks 2c, 2c + 1 (D = 64: c) of tokens r and r + 8. A k-step of the MMA may
//     take any 16 dimensions as long as q agrees, so the four words of a chunk feed four
//     k-steps: S[16 x 8] = q K8^T with the heads as rows (rows 8..15: the low parts of q,
//     for an fp32 query) and eight tokens as columns, two such tiles a page.
//   S leaves lane (r, c) with head r, tokens 2c, 2c + 1, 8 + 2c, 9 + 2c: already the B
//     fragment of P^T in O^T = V8^T P^T (k = tokens, n = heads).
//   V: lane reads chunk r (D / 8 dimensions) of those same four tokens, and pairs the tokens'
//     bytes with one byte permutation per four codes before converting.
// Precision: the codes are exact in fp16. A query row is multiplied by the power of two that
// brings its largest element to [2^14, 2^15) and enters as fp16 hi + lo: an element keeps 2^-22
// of itself, or 2^-39 of the row's largest where that is more. bf16 queries enter as hi alone,
// exact down to 2^-31 of the row's largest and within 2^-39 of it below. The weights of a page
// enter in the same way, at the power of two of that page's largest weight: within 2^-22 of
// themselves or 2^-38 of that largest, however the pages' V scales differ (down to weights of
// 2^-112 of the warp's largest; those below keep fewer bits).
// (One power for all pages, 21.7 us for the 128K batch below, would lose a page whose weights are
// below 2^-38 of the largest, however large its V scale.) Sums are fp32; the scales are applied to
// each page's product in fp32, so none can leave fp16's range.
//
// Measured (G = 4, d = 128, E4M3, 32 units of a 128K batch, 69.5 MB of selected codes): 22.1 us
// a call, 3.1 TB/s over the whole call and 5.8 TB/s of random 2 KB pages in the loop itself;
// bound by memory there (without the V products 21.1 us), by the chain of launch, block list,
// page indices and first copies (3.8 us) before it and the workspace merge (3 us) after it.
// Short calls are that chain: 8.3 us for 8 units of 32K, 4.0 us for one token.
#include <algorithm>

#include "bs_attn_impl.cuh"
#include "bs_attn_launch.cuh"
#include "bs_quant.cuh"

namespace bsi {
namespace {

constexpr int kQuantThreads = 128;   // 4 warps
constexpr int kQuantWarps = kQuantThreads / 32;
constexpr int kCtasPerSm = 2;
constexpr int kMinSplit = 8;
constexpr int kStepSplit = 40;

// Shared memory: the staged selection entries, then the warps' buffers; after the loop the
// warps' states take the buffers' place.
template <int D>
struct QuantLayout {
  static constexpr int kPageBytes = kPage * D;
  static constexpr int kOffBuf = kSelPreload * 4;                           // per warp: a pair of K, a pair of V
  static constexpr int kWarpBytes = 4 * kPageBytes;
  static constexpr int kOffO = kOffBuf;                                     // [4][8][D]
  static constexpr int kOffMl = kOffO + kQuantWarps * kMaxG * D * 4;         // m, l: [2][4][8]
  static constexpr int kEnd = kOffMl + 2 * kQuantWarps * kMaxG * 4;
  static constexpr int kBufEnd = kOffBuf + kQuantWarps * kWarpBytes;
  // What a cluster's other CTAs send while this one may still be in its loop: per column
  // entry, o (float4) and (m, l).
  static constexpr int kOffRecvO = kEnd > kBufEnd ? kEnd : kBufEnd;
  static constexpr int kOffRecvMl = kOffRecvO + kMaxG * D * 4;
  static constexpr int kBytes = kOffRecvMl + kMaxG * (D / 4) * 8;
};

// Byte offset of 16-byte chunk `ch` of row `row` of a page in its buffer.
template <int D>
__device__ __forceinline__ int swz8(int row, int ch) {
  return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A page's codes into its buffer (all 32 lanes; whole rows a warp instruction).
template <int D>
__device__ __forceinline__ void copy_page(uint32_t slot, const uint8_t *pool, int phys) {
  constexpr int kChunks = D / 16;
  const int lane = threadIdx.x & 31;
  const uint8_t *src = pool + static_cast<size_t>(phys) * (kPage * D) + lane * 16;
#pragma unroll
  for (int i = 0; i < kPage * kChunks / 32; ++i) {
    const int at = i * 32 + lane;
    cp_async16(slot + swz8<D>(at / kChunks, at % kChunks), src + i * 512);
  }
}

// D = A B + D, m16n8k16, fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo_f(uint32_t w) { return __half2float(__ushort_as_half(w & 0xffffu)); }
__device__ __forceinline__ float f16_hi_f(uint32_t w) { return __half2float(__ushort_as_half(w >> 16)); }

// A page in flight and what its codes mean; no valid tokens: it does not count and nothing
// of it is read.
struct PageMeta {
  uint32_t page;   // physical page << 5 | valid tokens (pools hold less than 2^27 pages)
  float ks, vs, bias;
  __device__ __forceinline__ int valid() const { return static_cast<int>(page & 31u); }
  __device__ __forceinline__ int phys() const { return static_cast<int>(page >> 5); }
};

// A lane's part of the query rows of a unit: row lane / 4 (zeros past the last head), the
// dimensions of its K chunks. Loaded first, converted once the block list is known, so that
// the loads are in flight beside the list's.
template <int D, bool Q32>
struct RawQ {
  static constexpr int kVecs = D / (Q32 ? 16 : 32);
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const void *q, size_t orow0, int G) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const char *src = static_cast<const char *>(q) + ((orow0 + r) * D + (D / 4) * c) * (Q32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = r < G ? ld_stream16(src + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
  }
  // Dimensions 4 s .. 4 s + 3 of the part.
  __device__ __forceinline__ void four(int s, float (&x)[4]) const {
    if constexpr (Q32) {
      x[0] = __uint_as_float(v[s].x); x[1] = __uint_as_float(v[s].y);
      x[2] = __uint_as_float(v[s].z); x[3] = __uint_as_float(v[s].w);
    } else {
      const uint32_t a = s & 1 ? v[s / 2].z : v[s / 2].x, b = s & 1 ? v[s / 2].w : v[s / 2].y;
      x[0] = bf16lo(a); x[1] = bf16hi(a); x[2] = bf16lo(b); x[3] = bf16hi(b);
    }
  }
};

// The query rows as A fragments in the dimension order of the K reads, times 2^e with the
// row's largest element near 2^14; *unscale gets 2^-e (head lane / 4).
template <int D, bool Q32>
__device__ __forceinline__ void q_to_f16(const RawQ<D, Q32> &raw, uint32_t (&hi)[D / 16][2], uint32_t (&lo)[D / 16][2],
                                         float *unscale) {
  float x[D / 16][4];
  float big = 0.0f;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    raw.four(s, x[s]);
#pragma unroll
    for (int i = 0; i < 4; ++i) big = fmaxf(big, fabsf(x[s][i]));
  }
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
  // 2^e with e = 14 - floor(log2 big), kept within fp32's normal range; zero and
  // non-finite rows stay as they are.
  int e = 0;
  if (big > 0.0f && big < INFINITY) {
    e = 14 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
    e = max(-120, min(120, e));
  }
  const float scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  *unscale = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = x[s][2 * i] * scale, b = x[s][2 * i + 1] * scale;
      hi[s][i] = pack_f16(a, b);
      lo[s][i] = Q32 ? pack_f16(a - f16_lo_f(hi[s][i]), b - f16_hi_f(hi[s][i])) : 0u;
    }
}

// A warp's running state: m and l of head lane / 4 (m replicated over the head's four lanes;
// l a partial sum of exp(x - m) per lane), and
// o[i][k] = O[heads 2 c, 2 c + 1][dim r D/8 + 2 i + k].
template <int D>
struct WarpState {
  float m, l;
  float2 o[D / 16][2];
};

// S = q K8^T of the page in `slot`: two tiles of eight tokens; x[i] of token 2c + (i & 1) +
// 8 (i >> 1).
template <int D, bool I8, bool Q32>
__device__ __forceinline__ void page_scores(const unsigned char *slot, const PageMeta &t, const uint32_t (&qh)[D / 16][2],
                                            const uint32_t (&ql)[D / 16][2], float q_scale, float *x) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    uint4 w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = *reinterpret_cast<const uint4 *>(slot + swz8<D>(r + 8 * i, D == 128 ? 2 * c + j : c));
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t b0, b1;
        codes_to_f16<I8>(k == 0 ? w[i].x : k == 1 ? w[i].y : k == 2 ? w[i].z : w[i].w, b0, b1);
        mma_f16(s[i], qh[4 * j + k][0], ql[4 * j + k][0], qh[4 * j + k][1], ql[4 * j + k][1], b0, b1);
      }
  }
  const float f = q_scale * t.ks;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float dot = Q32 ? s[i >> 1][i & 1] + s[i >> 1][2 + (i & 1)] : s[i >> 1][i & 1];
    x[i] = fmaf(dot, f, t.bias);
  }
}

// O^T += vs V8^T P^T of the page in `slot` (h, l: the page's weights at their power of two as
// fp16 pairs, hi and lo; back: its reciprocal for heads 2 c and 2 c + 1). The products come back
// to their size before the V scale enters: the two together may be subnormal. Two-wide fp32
// makes that free (the multiplication and the addition take the issue slots of one-wide
// additions). Codes of tokens that do not count may be anything (NaN too) and are zeroed.
template <int D, bool I8>
__device__ __forceinline__ void page_values(const unsigned char *slot, const PageMeta &t, const uint32_t (&h)[2],
                                            const uint32_t (&l)[2], float2 back, WarpState<D> &w) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  uint32_t v[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4 *>(slot + swz8<D>(tok, r));
      v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(slot + swz8<D>(tok, r >> 1) + 8 * (r & 1));
      v[i][0] = x.x; v[i][1] = x.y;
    }
  }
  if (t.valid() < kPage) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (2 * c + (i & 1) + 8 * (i >> 1) >= t.valid()) {
#pragma unroll
        for (int g = 0; g < D / 32; ++g) v[i][g] = 0u;
      }
  }
  const float2 vs = make_float2(t.vs, t.vs);
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {      // four dimensions of the lane's chunk
    const uint32_t v0 = v[0][g], v1 = v[1][g], v2 = v[2][g], v3 = v[3][g];
    uint32_t a[4], b[4];                   // fp16 pairs of tokens (2c, 2c+1) and (2c+8, 2c+9) per dimension
    codes_to_f16<I8>(__byte_perm(v0, v1, 0x5140), a[0], a[1]);
    codes_to_f16<I8>(__byte_perm(v0, v1, 0x7362), a[2], a[3]);
    codes_to_f16<I8>(__byte_perm(v2, v3, 0x5140), b[0], b[1]);
    codes_to_f16<I8>(__byte_perm(v2, v3, 0x7362), b[2], b[3]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(acc, a[2 * i], a[2 * i + 1], b[2 * i], b[2 * i + 1], h[0], h[1]);
      mma_f16(acc, a[2 * i], a[2 * i + 1], b[2 * i], b[2 * i + 1], l[0], l[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w.o[2 * g + i][k] = __ffma2_rn(__fmul2_rn(make_float2(acc[2 * k], acc[2 * k + 1]), back), vs, w.o[2 * g + i][k]);
    }
  }
}

// 2^x, results below 2^-126 as 0; exp(x) as 2^(x log2 e).
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_ftz(float x) { return exp2_ftz(x * kLog2e); }

// Online softmax of this lane's head over the 32 tokens of two pages: x becomes the weights
// exp(x - m), the running state is rescaled when the maximum rises.
//
// up[j] is the power of two that brings page j's largest weight near 2^14 (weights down to
// 2^-112) before it enters fp16, back[j] its reciprocal for heads 2 c and 2 c + 1: a page's
// weights keep their bits relative to that page's largest, so that pages may differ in their V
// scales as fp32 allows.
template <int D>
__device__ __forceinline__ void softmax_pair(float (&x)[8], WarpState<D> &w, float (&up)[2], float2 (&back)[2]) {
  const int c = threadIdx.x & 3;
  float top[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float mx = fmaxf(fmaxf(x[4 * j], x[4 * j + 1]), fmaxf(x[4 * j + 2], x[4 * j + 3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    top[j] = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  }
  const float mx = fmaxf(top[0], top[1]);
  if (__any_sync(0xffffffffu, mx > w.m)) {
    const float m_new = fmaxf(w.m, mx);
    const float alpha = m_new == -INFINITY ? 1.0f : exp_ftz(w.m - m_new);
    w.m = m_new;
    w.l *= alpha;
    const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c), a1 = __shfl_sync(0xffffffffu, alpha, 8 * c + 4);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) w.o[i][k] = __fmul2_rn(w.o[i][k], make_float2(a0, a1));
  }
  const float base = w.m == -INFINITY ? 0.0f : w.m;
  // The exponent e of the page's largest weight, -112 .. 0: the nearest integer by the low bits
  // of the sum with 1.5 * 2^23. back's exponent field is 113 + e (7 bits), up's 254 less it; the
  // two pages' go to the lanes of the products in one word.
  uint32_t field[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float t = fmaxf((top[j] - base) * kLog2e, -112.0f) + 12582912.0f;
    field[j] = __float_as_uint(t) - 0x4b400000u + 113u;
    up[j] = __uint_as_float((254u - field[j]) << 23);
  }
  const uint32_t fields = field[1] << 16 | field[0];
  const uint32_t f0 = __shfl_sync(0xffffffffu, fields, 8 * c), f1 = __shfl_sync(0xffffffffu, fields, 8 * c + 4);
  back[0] = make_float2(__uint_as_float(f0 << 23), __uint_as_float(f1 << 23));
  back[1] = make_float2(__uint_as_float(f0 << 7 & 0x7f800000u), __uint_as_float(f1 << 7 & 0x7f800000u));
#pragma unroll
  for (int i = 0; i < 8; i += 2) {   // (a weight below 2^-126 of the largest is 0)
    const float2 less = __fadd2_rn(make_float2(x[i], x[i + 1]), make_float2(-base, -base));
    const float2 y = __fmul2_rn(less, make_float2(kLog2e, kLog2e));
    x[i] = exp2_ftz(y.x);
    x[i + 1] = exp2_ftz(y.y);
  }
  w.l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}
__device__ __forceinline__ void split_weights(const float *x, float up, uint32_t (&h)[2], uint32_t (&l)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(up, up));
    h[i] = pack_f16(a.x, a.y);
    const float2 rest = __fadd2_rn(a, make_float2(-f16_lo_f(h[i]), -f16_hi_f(h[i])));
    l[i] = pack_f16(rest.x, rest.y);
  }
}

// One float4 column of the merge of n states of a head, visited in order, kFlight of them in
// flight at once: load(k, m, l, o) gives state k's maximum, sum and unnormalised column.
// A state with m = -inf has weight 0; a NaN stays one.
template <int kFlight, class Load>
__device__ __forceinline__ void merge_column(int n, Load load, float4 &o, float &m, float &l) {
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  m = -INFINITY;
  l = 0.0f;
  for (int k0 = 0; k0 < n; k0 += kFlight) {
    float mk[kFlight], lk[kFlight];
    float4 v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      mk[k] = -INFINITY;
      lk[k] = 0.0f;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < n) load(k0 + k, mk[k], lk[k], v[k]);
    }
    float m_new = m;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) m_new = fmaxf(m_new, mk[k]);
    const float base = m_new == -INFINITY ? 0.0f : m_new;
    const float a = exp2f((m - base) * kLog2e);
    o.x *= a; o.y *= a; o.z *= a; o.w *= a;
    l *= a;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const float wt = exp2f((mk[k] - base) * kLog2e);
      o.x = fmaf(v[k].x, wt, o.x);
      o.y = fmaf(v[k].y, wt, o.y);
      o.z = fmaf(v[k].z, wt, o.z);
      o.w = fmaf(v[k].w, wt, o.w);
      l = fmaf(lk[k], wt, l);
    }
    m = m_new;
  }
}

// o / l and lse = m + log l; a state with l = 0 (nothing attended) gives zeros and -inf.
__device__ __forceinline__ void write_column(const float4 &o, float m, float l, float *orow, float *lse_h, int dq) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  reinterpret_cast<float4 *>(orow)[dq] =
      l == 0.0f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (dq == 0) *lse_h = l == 0.0f ? -INFINITY : m + logf(l);
}

// The first barrier of a cluster's life, in two halves: arrived at on entry, waited for
// before the first access to a peer's memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_peer4(uint32_t a, const float4 &v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_peer2(uint32_t a, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}

// The end of a split: the four warps' states (ow [4][8][D], mw and lw [4][8], in shared
// memory and visible) merged, and merged with the unit's other splits: ns splits take part.
// One writes its output itself. A cluster's CTA r merges the columns r, r + ns, ...: every CTA
// sends its own to the owner's shared memory (each has started: attn_split_quant) and one
// cluster barrier later the owner merges what it got, in split order. (Reading the peers'
// memory instead needs a second barrier, which keeps every CTA until it has been read: 2.3 to
// 2.6 us from the last CTA's loop to the end, against 1.8 to 2.3.) In workspace mode each writes a record, takes an
// arrival ticket, and the last merges the records in split order.
template <int D>
__device__ void finish_quant(const AttnArgs &a, const UnitBlocks &ub, int u, int split, int ns, bool in_cluster, int G,
                             size_t orow0, unsigned char *smem) {
  using L = QuantLayout<D>;
  constexpr int NT = kQuantThreads, W = kQuantWarps, QD = D / 4, REC = attn_record_floats(D);
  const int tid = threadIdx.x;
  const float *ow = reinterpret_cast<const float *>(smem + L::kOffO);
  const float *mw = reinterpret_cast<const float *>(smem + L::kOffMl), *lw = mw + W * kMaxG;
  float4 *recv_o = reinterpret_cast<float4 *>(smem + L::kOffRecvO);
  float2 *recv_ml = reinterpret_cast<float2 *>(smem + L::kOffRecvMl);
  if (in_cluster && ns > 1) cluster_wait();   // every CTA of the cluster has started
  float *base = a.records + static_cast<size_t>(u) * kAttnMaxSplits * G * REC;
  for (int i = tid; i < G * QD; i += NT) {
    const int h = i / QD, dq = i % QD;
    float4 o;
    float m, l;
    merge_column<W>(W, [&](int k, float &mk, float &lk, float4 &v) {
      mk = mw[k * kMaxG + h];
      lk = lw[k * kMaxG + h];
      v = reinterpret_cast<const float4 *>(ow + (k * kMaxG + h) * D)[dq];
    }, o, m, l);
    if (ns == 1) {
      write_column(o, m, l, a.out + (orow0 + h) * D, a.lse + orow0 + h, dq);
      continue;
    }
    if (in_cluster) {
      const int owner = i % ns, at = i / ns * ns + split;   // (ns divides G * D / 4)
      st_peer4(peer_addr(recv_o + at, owner), o);
      st_peer2(peer_addr(recv_ml + at, owner), m, l);
      continue;
    }
    float *row = base + (static_cast<size_t>(split) * G + h) * REC;
    reinterpret_cast<float4 *>(row)[dq] = o;
    if (dq == 0) {
      row[D] = m;
      row[D + 1] = l;
    }
  }
  if (ns == 1) {
    if (ub.polled && tid == 0) a.expect[u] = ub.epoch;
    return;
  }
  if (in_cluster) {
    cluster_sync_all();
    const int rank = static_cast<int>(cluster_rank());
    for (int i = rank + ns * tid; i < G * QD; i += ns * NT) {
      const int h = i / QD, dq = i % QD, at = i / ns * ns;
      float4 o;
      float m, l;
      merge_column<8>(ns, [&](int k, float &mk, float &lk, float4 &v) {
        const float2 ml = recv_ml[at + k];
        mk = ml.x;
        lk = ml.y;
        v = recv_o[at + k];
      }, o, m, l);
      write_column(o, m, l, a.out + (orow0 + h) * D, a.lse + orow0 + h, dq);
    }
    // Every CTA of the cluster has read the unit's words: advance its epoch.
    if (ub.polled && split == 0 && tid == 0) a.expect[u] = ub.epoch;
    return;
  }
  // The CTA barrier orders every thread's record writes before thread 0's release; the last
  // split acquires.
  __shared__ int is_last;
  __syncthreads();
  if (tid == 0) is_last = atomic_add_acq_rel_gpu(a.arrivals + u, 1) == ns - 1;
  __syncthreads();
  if (!is_last) return;
  for (int i = tid; i < G * QD; i += NT) {
    const int h = i / QD, dq = i % QD;
    float4 o;
    float m, l;
    merge_column<16>(ns, [&](int k, float &mk, float &lk, float4 &v) {
      const float *row = base + (static_cast<size_t>(k) * G + h) * REC;
      mk = __ldcg(row + D);
      lk = __ldcg(row + D + 1);
      v = __ldcg(reinterpret_cast<const float4 *>(row) + dq);
    }, o, m, l);
    write_column(o, m, l, a.out + (orow0 + h) * D, a.lse + orow0 + h, dq);
  }
  if (tid == 0) {
    a.arrivals[u] = 0;  // ready for the next call
    if (ub.polled) a.expect[u] = ub.epoch;
  }
}

// Page gp of the split as resolve_page gives it, with the block's logit; its
// load flies beside the page's. 0 tokens for a page that does not count: past the end,
// outside the pool or the rows (reported), or of a block that dropped out (logit -inf).
__device__ __forceinline__ int resolve_quant_page(const UnitBlocks &ub, const AttnArgs &a, const int32_t *pt, int u, int gp,
                                                  int gp1, int *phys, float *bias) {
  *phys = -1;
  *bias = 0.0f;
  if (gp >= gp1) return 0;
  const bs_dims &dims = a.dims;
  const int ppb = ub.pg.ppb, i = gp / ppb;
  int blk = 0, valid;
  bool ok = true;
  const int32_t *where;
  if (ub.plist) {   // resolved by the selection; all full but the unit's last, which holds token T - 1
    where = ub.plist + gp;
    valid = gp == ub.pg.n_pages - 1 ? (ub.T - 1) % kPage + 1 : kPage;
    if (a.bias) blk = __ldcg(ub.sel + i);
  } else {
    blk = ub.block(i);
    const int64_t lp = static_cast<int64_t>(blk) * ppb + (gp - i * ppb);
    ok = blk >= 0 && lp < dims.max_pages_per_unit && lp * kPage < ub.T;
    where = pt + (ok ? lp : 0);
    valid = static_cast<int>(min(static_cast<int64_t>(kPage), ub.T - lp * kPage));
  }
  const bool logit = a.bias != nullptr;
  ok = ok && (!logit || (blk >= 0 && blk < dims.max_blocks_per_unit));
  const int p = __ldcg(where);
  const float e = logit ? __ldcg(a.bias + static_cast<size_t>(u) * dims.max_blocks_per_unit + (ok ? blk : 0)) : 0.0f;
  if (!ok || p < 0 || p >= dims.n_pages) {
    report(a.st, BS_ERR_DEVICE_BOUNDS);
    return 0;
  }
  *bias = e;
  if (e == -INFINITY) return 0;   // (nothing of it is read)
  *phys = p;
  return valid;
}

// Returns false for a split that took no part (it left at once; see step_ws_splits).
template <int D, bool I8, bool Q32>
__device__ bool attn_split_quant(const AttnArgs &a, unsigned char *smem, bool in_step, bool in_cluster) {
  using L = QuantLayout<D>;
  constexpr int NT = kQuantThreads, W = kQuantWarps;
  const bs_dims &dims = a.dims;
  int32_t *st = a.st;
  const int u = attn_unit_id(in_cluster), split = attn_split_id(in_cluster);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = dims.n_q_heads / dims.n_kv_heads;
  const int b = u / dims.n_kv_heads, hk = u % dims.n_kv_heads;
  const size_t orow0 = static_cast<size_t>(b) * dims.n_q_heads + static_cast<size_t>(hk) * G;
  int32_t *sel_sm = reinterpret_cast<int32_t *>(smem);
  const int n_part = in_step && !in_cluster ? step_ws_splits(a, u, attn_n_splits(false)) : attn_n_splits(in_cluster);
  if (split >= n_part) return false;   // (never in a cluster)
  if (in_cluster && n_part > 1) cluster_arrive();

  if (in_step) prefetch_page_row<NT>(dims, a.kv, a.cfg, a.plist, u, in_step);
  RawQ<D, Q32> raw_q;
  raw_q.load(a.q, orow0, G);
  UnitBlocks ub = load_unit_blocks<NT>(a, u, sel_sm, in_step, in_cluster);
  check_split_bound(ub, n_part, split, st);
  // A cluster's splits, and in the fused step those of step_ws_splits, all stay to the end.
  // The stand-alone call's know the unit's count at once: those past its pages leave (of a
  // unit that cannot be attended all but the first, which writes its zeros).
  const int ns = in_step || in_cluster ? n_part : ub.ok ? max(1, ub.pg.n_split) : 1;
  if (split >= ns) return false;
  const int n_pages = ub.ok ? ub.pg.n_pages : 0;
  const int gp0 = min(split * ub.pg.pps, n_pages);
  const int gp1 = min(gp0 + ub.pg.pps, n_pages);
  const int32_t *pt = a.kv.page_table + static_cast<size_t>(u) * dims.max_pages_per_unit;
  const uint8_t *kpool = static_cast<const uint8_t *>(a.kv.k_pool);
  const uint8_t *vpool = static_cast<const uint8_t *>(a.kv.v_pool);

  // This warp's pages: gp0 + warp + W i, i < n_mine; resolved 32 at a time, one per lane.
  const int n_mine = gp1 - gp0 > warp ? (gp1 - gp0 - warp + W - 1) / W : 0;
  uint32_t ch_page = 0;   // physical page (27 bits) and valid tokens (5 bits)
  float ch_ks = 0.0f, ch_vs = 0.0f, ch_bias = 0.0f;
  unsigned char *kbuf = smem + L::kOffBuf + warp * L::kWarpBytes, *vbuf = kbuf + 2 * L::kPageBytes;
  const uint32_t kslot = smem_u32(kbuf), vslot = smem_u32(vbuf);
  const bool biased = a.bias != nullptr;
  // Pages i, i + 1 (i even: both lie in one chunk of 32).
  auto meta = [&](int i, PageMeta (&t)[2]) {
    if (i >= n_mine) {
      t[0].page = t[1].page = 0u;
      return;
    }
    if ((i & 31) == 0) {
      int phys;
      const int valid = resolve_quant_page(ub, a, pt, u, gp0 + warp + W * (i + lane), gp1, &phys, &ch_bias);
      ch_page = valid > 0 ? static_cast<uint32_t>(phys) << 5 | static_cast<uint32_t>(valid) : 0u;
      ch_ks = valid > 0 ? __ldcg(a.kv.k_scale + phys) : 0.0f;   // (not waited for until the pair is computed)
      ch_vs = valid > 0 ? __ldcg(a.kv.v_scale + phys) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) t[j].page = __shfl_sync(0xffffffffu, ch_page, (i & 31) + j);
  };
  // What the pair's codes mean, once it is computed (before the next meta of a chunk's end).
  auto scales = [&](int i, PageMeta (&t)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t[j].ks = __shfl_sync(0xffffffffu, ch_ks, (i & 31) + j);
      t[j].vs = __shfl_sync(0xffffffffu, ch_vs, (i & 31) + j);
      t[j].bias = biased ? __shfl_sync(0xffffffffu, ch_bias, (i & 31) + j) : 0.0f;
    }
  };
  // One group of copies a pair and pool, empty past the end.
  auto copy_pair = [&](const PageMeta (&t)[2], uint32_t to, const uint8_t *pool) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (t[j].valid() > 0) copy_page<D>(to + j * L::kPageBytes, pool, t[j].phys());
    cp_commit();
  };

  WarpState<D> w;
  w.m = -INFINITY;
  w.l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) w.o[i][0] = w.o[i][1] = make_float2(0.0f, 0.0f);
  PageMeta t[2];
  meta(0, t);
  copy_pair(t, kslot, kpool);
  copy_pair(t, vslot, vpool);
  uint32_t qh[D / 16][2], ql[D / 16][2];
  float q_scale;
  q_to_f16<D, Q32>(raw_q, qh, ql, &q_scale);
  q_scale *= rsqrtf(static_cast<float>(D));
  for (int i = 0; i < n_mine; i += 2) {
    scales(i, t);
    const bool any = (t[0].page | t[1].page) != 0u;   // (none: dropped, or outside the pool)
    cp_wait<1>();            // this pair's K has landed
    __syncwarp();
    float x[8];
    if (any) {
#pragma unroll
      for (int j = 0; j < 2; ++j) page_scores<D, I8, Q32>(kbuf + j * L::kPageBytes, t[j], qh, ql, q_scale, x + 4 * j);
    }
    __syncwarp();
    PageMeta next[2];
    meta(i + 2, next);
    copy_pair(next, kslot, kpool);
    cp_wait<1>();            // its V too
    __syncwarp();
    if (any) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (t[j].valid() < kPage) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (2 * (lane & 3) + (k & 1) + 8 * (k >> 1) >= t[j].valid()) x[4 * j + k] = -INFINITY;
        }
      float up[2];
      float2 back[2];
      softmax_pair<D>(x, w, up, back);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h[2], l[2];
        split_weights(x + 4 * j, up[j], h, l);
        page_values<D, I8>(vbuf + j * L::kPageBytes, t[j], h, l, back[j], w);
      }
    }
    __syncwarp();
    copy_pair(next, vslot, vpool);
    t[0] = next[0];
    t[1] = next[1];
  }
  cp_wait<0>();
  __syncthreads();           // the buffers' place is taken by the states below

  // ---- combine the four warps' states ---------------------------------------------
  float *ow = reinterpret_cast<float *>(smem + L::kOffO);     // [4][8][D]
  float *mw = reinterpret_cast<float *>(smem + L::kOffMl);    // [4][8]
  float *lw = mw + W * kMaxG;                                 // [4][8]
  {
    const int r = lane >> 2, c = lane & 3;
    w.l += __shfl_xor_sync(0xffffffffu, w.l, 1);
    w.l += __shfl_xor_sync(0xffffffffu, w.l, 2);
    if (c == 0) {
      mw[warp * kMaxG + r] = w.m;
      lw[warp * kMaxG + r] = w.l;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float2 *>(ow + (warp * kMaxG + 2 * c + j) * D + r * (D / 8) + 2 * i) =
            j == 0 ? make_float2(w.o[i][0].x, w.o[i][1].x) : make_float2(w.o[i][0].y, w.o[i][1].y);
  }
  __syncthreads();
  finish_quant<D>(a, ub, u, split, ns, in_cluster, G, orow0, smem);
  return true;
}

template <int D, bool I8, bool Q32>
__global__ void __launch_bounds__(kQuantThreads, kCtasPerSm) attn_quant_kernel(const __grid_constant__ AttnArgs a, bool step, bool cluster) {
  extern __shared__ __align__(16) unsigned char smem[];
  // The stand-alone call is a programmatic dependent of whatever ran before it: its CTAs are in
  // place when that ends, and wait for it before they read anything.
  if (!step) pdl_wait();
  pdl_launch_dependents();
  const bool took_part = attn_split_quant<D, I8, Q32>(a, smem, step, cluster);
  // In the fused step, finish only after the selection kernel has (a split that took no
  // part leaves at once: split 0 of every unit takes part, so the grid still does).
  if (step && took_part) pdl_wait();
}

template <int D, bool I8, bool Q32>
bs_status launch_quant(AttnArgs a, bool step, cudaStream_t cs) {
  const int units = a.dims.batch * a.dims.n_kv_heads;
  const int mg = a.dims.max_gather_pages_per_unit;
  // Pages per split in workspace mode. The stand-alone call's units start together: as many
  // as fill one wave if every unit takes its largest selection. In the fused step units start
  // as they are published, and 36 to 48 pages a split were best (a layer step of the 128K
  // batch: 69 to 70 us; 77 at 16 pages, 75 at 24, 73 at 32, 72 at 56, 76 by the rule above).
  if (mg <= kClusterMaxPages) {
    const int slots = attn_target_ctas() / 2 * kCtasPerSm;
    const int64_t even = (static_cast<int64_t>(units) * mg + slots - 1) / slots;
    a.min_split = step ? kStepSplit
                       : static_cast<int>(std::max<int64_t>(kMinSplit, (even + kQuantWarps - 1) / kQuantWarps * kQuantWarps));
  }
  constexpr int smem = QuantLayout<D>::kBytes;
  auto kernel = attn_quant_kernel<D, I8, Q32>;
  static OncePerDevice attrs;
  if (!attrs([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
               cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
      }))
    return BS_ERR_CUDA;
  const bool cluster = attn_mode(units, mg) == kModeCluster;
  int splits = attn_grid_splits(units, mg, attn_target_ctas(), a.min_split);
  // A cluster's merge costs more than a few pages: no more splits than leave each kMinSplit.
  if (cluster)
    while (splits > 1 && mg < splits * kMinSplit) splits >>= 1;
  const dim3 grid = cluster ? dim3(splits, units) : dim3(units, splits);   // (workspace mode: unit-major)
  const cudaError_t e =
      launch_ex(kernel, grid, kQuantThreads, smem, cs, cluster && splits > 1 ? splits : 0, true, a, step, cluster);
  return e == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

template <int D>
bs_status dispatch_types(const AttnArgs &a, bool step, cudaStream_t cs) {
  const bool i8 = a.dims.kv_dtype == BS_INT8, q32 = a.dims.q_dtype == BS_FP32;
  if (i8) return q32 ? launch_quant<D, true, true>(a, step, cs) : launch_quant<D, true, false>(a, step, cs);
  return q32 ? launch_quant<D, false, true>(a, step, cs) : launch_quant<D, false, false>(a, step, cs);
}

}  // namespace

bs_status launch_attn_quant(const AttnArgs &a, bool step, cudaStream_t cs) {
  return a.dims.head_dim == 128 ? dispatch_types<128>(a, step, cs) : dispatch_types<64>(a, step, cs);
}

}  // namespace bsi
