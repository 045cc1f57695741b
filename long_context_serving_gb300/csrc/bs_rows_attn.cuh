// Attention of rows of new tokens over a paged cache (bs_prefill_attn, bs_tree_decode_attn): what
// the rows of a unit are, the keys that they see, and one row computed by a warp in fp32.
//
// The keys of a block of rows are a list of groups of 16: pages of the cache (prefill: the sink's
// pages, then those from the first row's window, or from 0, to the last row's own; tree: the
// selected blocks' pages), then for a tree its drafts, 16 rows of k_new and v_new at a time.
#pragma once

#include <cuda_bf16.h>

#include "bs_rows.cuh"

namespace bsi {

struct RowsArgs {
  bs_dims dims;
  const __nv_bfloat16 *q;
  int64_t q_stride, n_rows;
  bs_kv kv;
  const int32_t *row_begin;
  const int32_t *cls, *sink_tokens, *local_tokens, *tok_begin;   // prefill
  const int32_t *block_tokens, *sel_idx, *sel_cnt;               // tree
  bs_drafts drafts;                                              // tree
  int32_t max_new;        // tokens of one sequence, at most (prefill: max_new_tokens, tree: max_draft)
  __nv_bfloat16 *out;
  float *lse;
  int32_t *st;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The new tokens of a sequence: n of them, the first at position p0 (prefill) of T.
struct SeqRows {
  int n, p0, T;
  int64_t row0;
};

// What is told of a sequence: tokens, drafts or first new token, first row.
struct SeqWords {
  int T, x;
  int64_t row0;
};
template <bool kTree>
__device__ __forceinline__ SeqWords seq_words(const RowsArgs &a, int b) {
  return SeqWords{a.kv.seq_lens[b], kTree ? a.drafts.n_draft[b] : a.tok_begin[b], a.row_begin[b]};
}

// 0, or the status of a sequence that does not fit (its n is then 0).
template <bool kTree>
__device__ __forceinline__ int seq_rows(const RowsArgs &a, const SeqWords &w, SeqRows &r) {
  const int T = w.T, x = w.x;
  r.n = 0;
  r.row0 = w.row0;
  r.T = T;
  r.p0 = kTree ? 0 : x;
  if (T < 0 || x < 0 || x > (kTree ? a.max_new : T)) return BS_ERR_INVALID_ARG;
  const int n = kTree ? x : T - x;
  if (n == 0) return 0;
  if (T / kPage + (T % kPage != 0) > a.dims.max_pages_per_unit || n > a.max_new) return BS_ERR_CAPACITY;
  if (r.row0 < 0 || r.row0 + n > (kTree ? a.drafts.n_rows : a.n_rows)) return BS_ERR_DEVICE_BOUNDS;
  r.n = n;
  return 0;
}

// The keys of tokens [i0, i1) of a unit's rows.
struct Keys {
  int T, p0;                 // as in SeqRows
  bool windowed;             // prefill: a streaming unit
  int sink, local;
  int n_sink, first;         // prefill: pages of the sink, first page of the window
  int ppb;                   // tree: pages a block
  int n_cache, n_groups;     // groups that are pages, all groups
  int n_draft;
  const int32_t *sel;        // tree: the unit's blocks
  const int32_t *table;      // its page table
};

// What is told of a unit: tree, tokens of a block and selected blocks; prefill, class, sink and window.
struct UnitWords {
  int x, y, z;
};
template <bool kTree>
__device__ __forceinline__ UnitWords unit_words(const RowsArgs &a, int u) {
  if constexpr (kTree) return UnitWords{a.block_tokens[u], a.sel_cnt[u], 0};
  else return UnitWords{a.cls[u], a.sink_tokens[u], a.local_tokens[u]};
}

template <bool kTree>
__device__ __forceinline__ int unit_keys(const RowsArgs &a, const SeqRows &r, const UnitWords &w, int u, int i0, int i1, Keys &k) {
  k.T = r.T;
  k.p0 = r.p0;
  k.table = a.kv.page_table + static_cast<int64_t>(u) * a.dims.max_pages_per_unit;
  k.windowed = false;
  k.sink = k.local = k.n_sink = k.first = k.n_draft = 0;
  k.ppb = 1;
  k.sel = nullptr;
  k.n_cache = k.n_groups = 0;
  if constexpr (kTree) {
    const int g = w.x, cnt = w.y;
    if (g <= 0 || g % kPage != 0 || cnt < 0) return BS_ERR_INVALID_ARG;
    k.ppb = g / kPage;
    if (cnt > a.dims.max_sel_per_unit || static_cast<int64_t>(cnt) * k.ppb > a.dims.max_gather_pages_per_unit)
      return BS_ERR_CAPACITY;
    k.sel = a.sel_idx + static_cast<int64_t>(u) * a.dims.max_sel_per_unit;
    k.n_draft = r.n;
    k.n_cache = cnt * k.ppb;
    k.n_groups = k.n_cache + (r.n + kPage - 1) / kPage;
  } else {
    const int cls = w.x;
    if (cls < BS_STREAMING || cls > BS_DUAL) return BS_ERR_INVALID_ARG;
    const int pa = r.p0 + i0, pb = r.p0 + i1 - 1;
    if (cls == BS_STREAMING) {
      k.windowed = true;
      k.sink = w.y;
      k.local = w.z;
      if (k.sink < 0 || k.local < 1) return BS_ERR_INVALID_ARG;
      k.first = max(pa - k.local + 1, 0) / kPage;
      k.n_sink = min(k.sink / kPage + (k.sink % kPage != 0), k.first);
    }
    k.n_cache = k.n_groups = k.n_sink + pb / kPage - k.first + 1;
  }
  return 0;
}

// Group i of the list: its first key (a token of the cache, or a draft), the page that holds it.
// page -1: a draft group; -2: nothing there, or something that does not exist (then reported).
struct Group {
  int base, page;
};

template <bool kTree>
__device__ __forceinline__ Group key_group(const RowsArgs &a, const Keys &k, int i) {
  Group g;
  int64_t lp;
  if constexpr (kTree) {
    if (i >= k.n_cache) {
      g.base = (i - k.n_cache) * kPage;
      g.page = -1;
      return g;
    }
    const int blk = k.sel[i / k.ppb];
    lp = static_cast<int64_t>(blk) * k.ppb + i % k.ppb;
    g.base = 0;
    g.page = -2;
    if (lp * kPage >= k.T || blk < 0) {
      if (blk < 0 || (lp - i % k.ppb) * kPage >= k.T) report(a.st, BS_ERR_DEVICE_BOUNDS);
      return g;
    }
  } else {
    lp = i < k.n_sink ? i : k.first + (i - k.n_sink);
  }
  g.base = static_cast<int>(lp) * kPage;
  g.page = k.table[lp];
  if (g.page < 0 || g.page >= a.dims.n_pages) {
    report(a.st, BS_ERR_DEVICE_BOUNDS);
    g.page = -2;
  }
  return g;
}

// Does token i of the rows (prefill: at position p0 + i; tree: its mask of drafts) see key
// base + c of a group?
template <bool kTree>
__device__ __forceinline__ bool sees(const Keys &k, const Group &g, int c, int i, uint64_t mask) {
  const int t = g.base + c;
  if constexpr (kTree) return g.page == -1 ? t < k.n_draft && ((mask >> t) & 1) != 0 : t < k.T;
  const int p = k.p0 + i;
  return t <= p && (!k.windowed || t < k.sink || t > p - k.local);
}

// ---------------------------------------------------------------------------------------
// Columns of one row by one warp, in fp32: lane l holds elements [l * D / 32, ...) of q and of the
// output. `bad` (a bit an element) are columns that are not finite in a product that had an unseen
// key's infinity or NaN in it. A key that the row does not see is not looked at; one that it does see
// and that is not finite itself explains its columns (a logit of NaN or +inf, all of them), whose bits are
// cleared; one of -inf weighs nothing.
// From the last key back, for what is not finite tends to be near and the search ends when nothing is
// left to explain. For the columns that stay: o, unnormalised, relative to 2^m (log2 units).
// ---------------------------------------------------------------------------------------
template <int D, bool kTree>
__device__ __noinline__ void row_columns(const RowsArgs &a, const SeqRows &r, const Keys &k, int h, int i, int gq, int g_lo,
                                         int g_hi, uint32_t &bad, float &m, float (&o)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int G = a.dims.n_q_heads / a.dims.n_kv_heads;
  const float sc = kLog2e * rsqrtf(static_cast<float>(D));
  float q[E];
  const __nv_bfloat16 *qp = a.q + (r.row0 + i) * a.q_stride + static_cast<int64_t>(h * G + gq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qp[e]);
    o[e] = 0.0f;
  }
  const uint64_t mask = kTree ? a.drafts.visible[r.row0 + i] : 0;
  m = -INFINITY;
  const int dt = a.dims.kv_dtype;
  auto value = [&](const void *pool, int64_t at) -> float {
    if (dt == BS_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(pool)[at]);
    const uint8_t c = static_cast<const uint8_t *>(pool)[at];
    if (dt == BS_INT8) return static_cast<float>(static_cast<int8_t>(c));
    float f[4];
    codes_to_f32<false>(c, f);
    return f[0];
  };
  for (int gi = g_hi - 1; gi >= g_lo; --gi) {
    if (!__any_sync(0xffffffffu, bad != 0)) return;
    const Group g = key_group<kTree>(a, k, gi);
    if (g.page == -2) continue;
    const bool draft = g.page == -1;
    const bool quant = !draft && is_quant(dt);
    const float ks = quant ? a.kv.k_scale[g.page] : 1.0f, vs = quant ? a.kv.v_scale[g.page] : 1.0f;
    for (int c = kPage - 1; c >= 0; --c) {
      if (!sees<kTree>(k, g, c, i, mask)) continue;
      const int64_t at = draft ? (r.row0 + g.base + c) * a.drafts.row_stride + static_cast<int64_t>(h) * D + lane * E
                               : (static_cast<int64_t>(g.page) * kPage + c) * D + lane * E;
      float x = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        x = fmaf(q[e], draft ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.drafts.k_new)[at + e]) : value(a.kv.k_pool, at + e), x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
      x = x * ks * sc;
      if (!(x < INFINITY)) {
        bad = 0;
        return;
      }
      const float top = fmaxf(m, x), keep = m == -INFINITY ? 0.0f : exp2f(m - top), w = x == -INFINITY ? 0.0f : exp2f(x - top);
      m = top;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = draft ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.drafts.v_new)[at + e]) : value(a.kv.v_pool, at + e) * vs;
        if (!(fabsf(v) < INFINITY)) bad &= ~(1u << e);
        o[e] = fmaf(o[e], keep, w * v);
      }
    }
  }
}

}  // namespace bsi
