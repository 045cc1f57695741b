// Attention of new tokens over the paged cache: bs_prefill_attn and bs_tree_decode_attn, their
// plans, and the merge of split rows.
#include "bs_rows_mma.cuh"

namespace bsi {
namespace {

// ---------------------------------------------------------------------------------------
// Plan: from host-known bounds only (n_rows, the most tokens of a sequence, the dims) and the current
// device's SMs.
// ---------------------------------------------------------------------------------------
struct HostPlan {
  RowsPlan p;
  int rows;                // rows of a CTA: 32, 128 or 256
  int64_t items;
  size_t ml_at, heads_at, workspace_bytes;
};

HostPlan plan_rows(const bs_dims &d, int64_t n_rows, int max_new, bool tree) {
  HostPlan h{};
  const int G = d.n_q_heads / d.n_kv_heads;
  h.rows = static_cast<int64_t>(max_new) * G <= 32 ? 32 : max_new <= 128 / G ? 128 : 256;
  h.p.tokens = (h.rows == 32 ? 32 : 128) / G;
  h.p.block_tokens = h.rows == 256 ? 2 * h.p.tokens : h.p.tokens;
  const int64_t per_seq = (static_cast<int64_t>(max_new) + h.p.block_tokens - 1) / h.p.block_tokens;
  int64_t tiles;           // key tiles of a block, at most
  if (tree) {
    h.p.n_blocks = static_cast<int>(per_seq);
    h.items = static_cast<int64_t>(d.batch) * d.n_kv_heads * per_seq;
    tiles = (static_cast<int64_t>(d.max_gather_pages_per_unit) + (max_new + kPage - 1) / kPage + kTileGroups - 1) / kTileGroups;
  } else {
    const int64_t by_seq = per_seq * d.batch, by_rows = n_rows / h.p.block_tokens + (n_rows < d.batch ? n_rows : d.batch);
    const int64_t blocks = per_seq == 1 || by_seq < by_rows ? by_seq : by_rows;
    h.p.n_blocks = per_seq == 1 ? 0 : static_cast<int>(blocks < INT32_MAX ? blocks : INT32_MAX);
    h.items = blocks * d.n_kv_heads;
    tiles = (static_cast<int64_t>(d.max_pages_per_unit) + kTileGroups - 1) / kTileGroups;
  }
  h.p.record_rows = (max_new < h.p.block_tokens ? max_new : h.p.block_tokens) * G;
  const int at_once = attn_target_ctas() / (h.rows == 32 ? 1 : 2);      // CTAs
  int64_t splits = 1;
  if (tree && h.items * tiles <= at_once) {
    splits = tiles;             // a CTA a tile: no more than a wave whatever the selections are
  } else if (tree && h.items <= kShareItems && h.items <= at_once && tiles < (1 << 20)) {
    // One wave over the units' own tiles (128K trees of uneven units: 58 us, an even number of splits
    // 65; working it out takes a CTA 1 to 2 us, which the case above does without: 10.2 us for 12.7).
    h.p.even = at_once;
    splits = tiles;
  } else {
    // What one wave has room for. Fewer rows than a tensor core's worth are bound by memory, and by
    // how evenly CTAs get their keys: as many pieces as the longest row that the table can hold has
    // 24 tiles (32 sequences of 2K to 16K tokens, of 16K at most: 165 us; pieces by 48 tiles 174, by 12 tiles
    // 167, whole sequences 229), while that is no more than eight waves of CTAs. A shorter sequence is cut
    // into as many, smaller ones, or into its tiles. Two row tiles are bound by their products, and split no further.
    splits = at_once / h.items;
    if (h.rows < 256 && tiles > 32) {
      const int64_t pieces = (tiles + 23) / 24, room = 8 * at_once / h.items;
      if (splits < (pieces < room ? pieces : room)) splits = pieces < room ? pieces : room;
    }
  }
  if (splits > tiles) splits = tiles;
  const int64_t row_bytes = static_cast<int64_t>(h.p.record_rows) * d.head_dim * 4;
  if (h.p.even == 0) {
    const int64_t most = (int64_t(64) << 20) / row_bytes / h.items;   // records of 64 MB
    if (splits > most) splits = most;
  }
  h.p.splits = static_cast<int>(splits < 1 ? 1 : splits);
  if (h.p.splits > 1) {
    const size_t recs = h.p.even > 0 ? h.p.even : static_cast<size_t>(h.items) * h.p.splits;
    h.ml_at = recs * row_bytes;
    h.heads_at = h.ml_at + (recs * h.p.record_rows * sizeof(float2) + 15) / 16 * 16;
    h.workspace_bytes = h.heads_at + static_cast<size_t>(h.items) * sizeof(int4);
  }
  return h;
}

// ---------------------------------------------------------------------------------------
// Merge of split rows: a warp a row, a lane D / 32 elements. Two loads one after the other (what the
// item is; its records, sixteen of them at a time in flight beside the maxima).
// ---------------------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <int D, bool kTree>
__global__ void __launch_bounds__(kMergeWarps * 32) rows_merge_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ RowsPlan p) {
  constexpr int E = D / 32, kAtOnce = 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the splits' records
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int item = blockIdx.x, row = blockIdx.y * kMergeWarps + warp;
  const int4 head = p.heads[item];                         // CTAs, the first, first row, rows
  const int G = a.dims.n_q_heads / a.dims.n_kv_heads, n = head.x;
  if (n <= 1 || row >= head.w * G) return;                 // nothing to do, or written already
  const int h = (kTree ? item / p.n_blocks : item) % a.dims.n_kv_heads;
  const int64_t rec = static_cast<int64_t>(head.y) * p.record_rows + row, step = p.record_rows;
  float o[kAtOnce][E];
  auto load = [&](int s0) {
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) o[s][e] = s0 + s < n ? p.rec_o[(rec + (s0 + s) * step) * D + lane * E + e] : 0.0f;
  };
  load(0);
  // A record's sum in log2 units; what is merged are means, weighed by sums of at most 1.
  auto size_of = [](float2 x) -> float { return x.y == 0.0f ? -INFINITY : x.x + log2f(x.y); };
  float m = -INFINITY;
  bool nan = false;                                        // (a record of NaN logits alone has no maximum)
  for (int s = lane; s < n; s += 32) {
    const float2 x = p.rec_ml[rec + s * step];
    m = fmaxf(m, size_of(x));
    nan |= x.y != x.y;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.0f, acc[E] = {};
  if (m != -INFINITY || __any_sync(0xffffffffu, nan)) {
    for (int s0 = 0; s0 < n; s0 += kAtOnce) {
      float w = 0.0f;                         // lane s: weight of record s0 + s
      if (lane < kAtOnce && s0 + lane < n) {
        const float2 x = p.rec_ml[rec + (s0 + lane) * step];
        w = x.y == 0.0f ? 0.0f : x.y * exp2f(x.x - m);
      }
      if (s0 > 0) load(s0);
#pragma unroll
      for (int s = 0; s < kAtOnce; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        l += ws;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(o[s][e], ws, acc[e]);
      }
    }
  }
  const int64_t out_row = (static_cast<int64_t>(head.z) + row / G) * a.dims.n_q_heads + h * G + row % G;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t *to = reinterpret_cast<uint32_t *>(a.out + out_row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) to[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[out_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <bool kTree>
bs_status launch_rows(RowsArgs &a, void *workspace, size_t workspace_bytes, cudaStream_t cs) {
  const bs_dims &d = a.dims;
  HostPlan h = plan_rows(d, a.n_rows, a.max_new, kTree);
  if (h.items > INT32_MAX || h.items * h.p.splits > INT32_MAX) return BS_ERR_CAPACITY;
  h.p.items = static_cast<int>(h.items);
  if (h.p.splits > 1) {
    if (workspace == nullptr) return BS_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return BS_ERR_ALIGN;
    if (workspace_bytes < h.workspace_bytes) return BS_ERR_CAPACITY;
    h.p.rec_o = static_cast<float *>(workspace);
    h.p.rec_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + h.ml_at);
    h.p.heads = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + h.heads_at);
  }
  h.p.wait_ns = wait_limit_ns();
  const int G = d.n_q_heads / d.n_kv_heads;
  const uint64_t D = static_cast<uint64_t>(d.head_dim);
  RowsMaps maps{};
  const uint64_t q_size[3] = {D, static_cast<uint64_t>(d.n_q_heads), static_cast<uint64_t>(a.n_rows)};
  const uint64_t q_step[2] = {D * 2, static_cast<uint64_t>(a.q_stride) * 2};
  const uint32_t q_box[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(h.p.tokens)};
  bs_status s = make_bf16_map(&maps.q, a.q, 3, q_size, q_step, q_box);
  if (s == BS_OK && d.kv_dtype == BS_BF16) {
    s = make_kv_tensor_maps(d, a.kv, &maps.k, &maps.v);
    if (kTree) {
      const uint64_t size[2] = {D * d.n_kv_heads, static_cast<uint64_t>(a.drafts.n_rows)};
      const uint64_t step[1] = {static_cast<uint64_t>(a.drafts.row_stride) * 2};
      const uint32_t box[2] = {64, kPage};
      if (s == BS_OK) s = make_bf16_map(&maps.k_new, a.drafts.k_new, 2, size, step, box);
      if (s == BS_OK) s = make_bf16_map(&maps.v_new, a.drafts.v_new, 2, size, step, box);
    }
  }
  if (s != BS_OK) return s;
  s = d.kv_dtype == BS_BF16 ? launch_rows_bf16<kTree>(a, h.p, maps, h.rows, cs)
                            : launch_rows_quant<kTree>(a, h.p, maps, h.rows, cs);
  if (s != BS_OK || h.p.splits == 1) return s;
  auto merge = d.head_dim == 128 ? rows_merge_kernel<128, kTree> : rows_merge_kernel<64, kTree>;
  const dim3 grid(static_cast<unsigned>(h.items), static_cast<unsigned>((h.p.record_rows + kMergeWarps - 1) / kMergeWarps));
  return launch_ex(merge, grid, kMergeWarps * 32, 0, cs, 0, true, a, h.p) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

// Host checks that both calls share (after those of the dims). Arrays of no rows have no address.
bs_status check_rows(const bs_dims *dims, const void *q, int64_t q_stride, int64_t n_rows, const bs_kv *kv, const void *cfg,
                     const void *out, const void *dev_status) {
  if (dims->q_dtype != BS_BF16 || dims->kv_dtype == BS_FP32) return BS_ERR_INVALID_ARG;
  if (n_rows < 0 || (n_rows > 0 && (!q || !out))) return BS_ERR_INVALID_ARG;
  if (!kv || !kv->k_pool || !kv->v_pool || !kv->page_table || !kv->seq_lens || !cfg || !dev_status) return BS_ERR_INVALID_ARG;
  if (is_quant(dims->kv_dtype) && (!kv->k_scale || !kv->v_scale)) return BS_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(dims->n_q_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(kv->k_pool) || !aligned16(kv->v_pool) || q_stride % 8 != 0)
    return BS_ERR_ALIGN;
  return BS_OK;
}

}  // namespace
}  // namespace bsi

extern "C" size_t bs_prefill_workspace_size(const bs_dims *dims, int64_t n_rows, int32_t max_new_tokens) {
  using namespace bsi;
  if (check_dims(dims) != BS_OK || n_rows < 1 || n_rows > INT32_MAX || max_new_tokens < 1) return 0;
  return plan_rows(*dims, n_rows, max_new_tokens, false).workspace_bytes;
}

extern "C" size_t bs_tree_workspace_size(const bs_dims *dims, int32_t max_draft) {
  using namespace bsi;
  if (check_dims(dims) != BS_OK || max_draft < 1 || max_draft > BS_MAX_DRAFT) return 0;
  return plan_rows(*dims, 0, max_draft, true).workspace_bytes;
}

extern "C" bs_status bs_prefill_attn(const bs_dims *dims, const void *q, int64_t q_stride, int64_t n_rows,
                                     const bs_kv *kv, const bs_head_cfg *cfg, const int32_t *tok_begin,
                                     const int32_t *row_begin, int32_t max_new_tokens, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                     bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  s = check_rows(dims, q, q_stride, n_rows, kv, cfg, out, dev_status);
  if (s != BS_OK) return s;
  if (!cfg->cls || !cfg->sink_tokens || !cfg->local_tokens || !tok_begin || !row_begin) return BS_ERR_INVALID_ARG;
  if (max_new_tokens < 1) return BS_ERR_INVALID_ARG;
  if (n_rows > INT32_MAX) return BS_ERR_CAPACITY;
  if (n_rows == 0) return BS_OK;
  RowsArgs a{};
  a.dims = *dims;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.kv = kv_of(*dims, kv);
  a.row_begin = row_begin;
  a.cls = cfg->cls;
  a.sink_tokens = cfg->sink_tokens;
  a.local_tokens = cfg->local_tokens;
  a.tok_begin = tok_begin;
  a.max_new = max_new_tokens;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.st = dev_status;
  return launch_rows<false>(a, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" bs_status bs_tree_decode_attn(const bs_dims *dims, const void *q, int64_t q_stride, const bs_kv *kv,
                                         const bs_head_cfg *cfg, const int32_t *sel_idx, const int32_t *sel_cnt,
                                         const bs_drafts *drafts, void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (!drafts) return BS_ERR_INVALID_ARG;
  s = check_rows(dims, q, q_stride, drafts->n_rows, kv, cfg, out, dev_status);
  if (s != BS_OK) return s;
  if (!cfg->block_tokens || !sel_idx || !sel_cnt || !drafts->row_begin || !drafts->n_draft) return BS_ERR_INVALID_ARG;
  if (drafts->n_rows > 0 && (!drafts->k_new || !drafts->v_new || !drafts->visible)) return BS_ERR_INVALID_ARG;
  if (drafts->max_draft < 1 || drafts->max_draft > BS_MAX_DRAFT) return BS_ERR_INVALID_ARG;
  if (drafts->row_stride < static_cast<int64_t>(dims->n_kv_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(drafts->k_new) || !aligned16(drafts->v_new) || drafts->row_stride % 8 != 0 ||
      reinterpret_cast<uintptr_t>(drafts->visible) % 8 != 0)
    return BS_ERR_ALIGN;
  if (drafts->n_rows > INT32_MAX) return BS_ERR_CAPACITY;
  if (drafts->n_rows == 0) return BS_OK;
  RowsArgs a{};
  a.dims = *dims;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_stride;
  a.n_rows = drafts->n_rows;
  a.kv = kv_of(*dims, kv);
  a.row_begin = drafts->row_begin;
  a.block_tokens = cfg->block_tokens;
  a.sel_idx = sel_idx;
  a.sel_cnt = sel_cnt;
  a.drafts = *drafts;
  a.max_new = drafts->max_draft;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.st = dev_status;
  return launch_rows<true>(a, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}
