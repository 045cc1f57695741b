// Attention of new tokens over the paged cache: bs_prefill_attn and bs_tree_decode_attn.
#include "bs_attn_launch.cuh"
#include "bs_rows_attn.cuh"

namespace bsi {
namespace {

constexpr int kRowWarps = 4;

// A warp a row and query head.
template <int D, bool kTree>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const __grid_constant__ RowsArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");      // everything before this call has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int G = a.dims.n_q_heads / a.dims.n_kv_heads, lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t row = item / a.dims.n_q_heads;
  const int head = static_cast<int>(item % a.dims.n_q_heads), h = head / G;
  SeqRows r;
  int b = 0;
  for (; b < a.dims.batch; ++b) {
    const int bad = seq_rows<kTree>(a, b, r);
    if (bad != 0 && item == 0 && lane == 0) report(a.st, bad);
    if (r.n > 0 && row >= r.row0 && row < r.row0 + r.n) break;
  }
  if (b == a.dims.batch) return;
  const int i = static_cast<int>(row - r.row0);
  Keys k;
  const int bad = unit_keys<kTree>(a, r, b * a.dims.n_kv_heads + h, i, i + 1, k);
  if (bad != 0) {
    if (lane == 0) report(a.st, bad);
    return;
  }
  float m, l, o[D / 32];
  row_attend<D, kTree>(a, r, k, h, i, head % G, 0, k.n_groups, m, l, o);
  __nv_bfloat16 *out = a.out + (row * a.dims.n_q_heads + head) * D + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) out[e] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] / l);
  if (lane == 0 && a.lse != nullptr) a.lse[row * a.dims.n_q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <bool kTree>
bs_status launch_rows(const RowsArgs &a, cudaStream_t cs) {
  const int64_t warps = (kTree ? a.drafts.n_rows : a.n_rows) * a.dims.n_q_heads;
  const int64_t ctas = (warps + kRowWarps - 1) / kRowWarps;
  if (ctas > INT32_MAX) return BS_ERR_CAPACITY;
  auto kernel = a.dims.head_dim == 128 ? rows_kernel<128, kTree> : rows_kernel<64, kTree>;
  return launch_ex(kernel, dim3(static_cast<unsigned>(ctas)), kRowWarps * 32, 0, cs, 0, true, a) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

// Host checks that both calls share (after those of the dims).
bs_status check_rows(const bs_dims *dims, const void *q, int64_t q_stride, const bs_kv *kv, const void *cfg,
                     const void *out, const void *dev_status) {
  if (dims->q_dtype != BS_BF16 || dims->kv_dtype == BS_FP32) return BS_ERR_INVALID_ARG;
  if (!q || !kv || !kv->k_pool || !kv->v_pool || !kv->page_table || !kv->seq_lens || !cfg || !out || !dev_status)
    return BS_ERR_INVALID_ARG;
  if (is_quant(dims->kv_dtype) && (!kv->k_scale || !kv->v_scale)) return BS_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(dims->n_q_heads) * dims->head_dim) return BS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(kv->k_pool) || !aligned16(kv->v_pool) || q_stride % 8 != 0)
    return BS_ERR_ALIGN;
  return BS_OK;
}

}  // namespace
}  // namespace bsi

extern "C" size_t bs_prefill_workspace_size(const bs_dims *dims, int64_t n_rows, int32_t max_new_tokens) {
  return 0;
}

extern "C" size_t bs_tree_workspace_size(const bs_dims *dims, int32_t max_draft) { return 0; }

extern "C" bs_status bs_prefill_attn(const bs_dims *dims, const void *q, int64_t q_stride, int64_t n_rows,
                                     const bs_kv *kv, const bs_head_cfg *cfg, const int32_t *tok_begin,
                                     const int32_t *row_begin, int32_t max_new_tokens, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                     bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  s = check_rows(dims, q, q_stride, kv, cfg, out, dev_status);
  if (s != BS_OK) return s;
  if (!cfg->cls || !cfg->sink_tokens || !cfg->local_tokens || !tok_begin || !row_begin) return BS_ERR_INVALID_ARG;
  if (n_rows < 0 || max_new_tokens < 1) return BS_ERR_INVALID_ARG;
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
  return launch_rows<false>(a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" bs_status bs_tree_decode_attn(const bs_dims *dims, const void *q, int64_t q_stride, const bs_kv *kv,
                                         const bs_head_cfg *cfg, const int32_t *sel_idx, const int32_t *sel_cnt,
                                         const bs_drafts *drafts, void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  s = check_rows(dims, q, q_stride, kv, cfg, out, dev_status);
  if (s != BS_OK) return s;
  if (!cfg->block_tokens || !sel_idx || !sel_cnt || !drafts || !drafts->k_new || !drafts->v_new || !drafts->row_begin ||
      !drafts->n_draft || !drafts->visible)
    return BS_ERR_INVALID_ARG;
  if (drafts->max_draft < 1 || drafts->max_draft > BS_MAX_DRAFT || drafts->n_rows < 0) return BS_ERR_INVALID_ARG;
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
  return launch_rows<true>(a, reinterpret_cast<cudaStream_t>(stream));
}
