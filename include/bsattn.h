/*
 * bsattn.h - block-sparse decode attention over a paged KV cache (C ABI).
 *
 * One decode step of one attention layer, for every unit u = (sequence b, KV head
 * h_kv), u = b * n_kv_heads + h_kv:
 *
 *   bs_build_block_summaries  sub-block mean keys kept current as tokens are appended
 *   bs_score_blocks           block scores: mean-key dot products max-pooled over the
 *                             sub-blocks of a block and reduced over the GQA group
 *   bs_select_topk            per-unit block selection: forced sink/local blocks,
 *                             query-aware top-k, NOSA's eviction-driven dual selection
 *   bs_sparse_decode_attn     split-KV flash-decode over the selected blocks only
 *   bs_block_setdiff          blocks added to / removed from the selection since the
 *                             previous step
 *   bs_decode_step            all five for one layer in two launches
 *   bs_block_swap             moves the blocks that the set-difference adds from host
 *                             memory into a GPU block cache (the offload path)
 *   bs_cpu_sparse_attn,       attention of a block subset on the host cores, and the
 *   bs_lse_merge              GPU merge of two partial results (CPU/GPU split)
 *   bs_quant_append           new tokens' K and V quantised into the pages of an 8-bit
 *                             cache (BS_E4M3 or BS_INT8 codes, one scale per page)
 *   bs_pages_reserve, _fork,  pages of a cache handed out, shared between sequences,
 *   _free, _compact, _copy    taken back, and moved together, all on the device
 *   bs_rope_append            queries and keys normalised per head and rotated to their
 *                             positions; K and V written into the cache's pages
 *   bs_prefill_attn           attention of new prompt tokens (or of single tokens) over
 *                             the cache that holds them: dense, or sinks and a window
 *   bs_tree_decode_attn       attention of a tree of drafted tokens over the selected
 *                             blocks and their ancestors
 *   bs_tree_commit            the accepted drafts' K and V appended to the cache
 *
 * Method sources: "Technisches Resümee: NOSA: Native und Offloadable Sparse
 * Attention" (section Methodik: "1. Algorithmus: NOSA" and "2. System: NOSI") and
 * "Technische Samenvatting: Fluxion" (sections Probleemstelling, Kerninzichten,
 * Systeemcomponenten).
 *
 * Conventions shared by every call
 * --------------------------------
 * Ownership. The caller allocates and owns every buffer. The library allocates
 *   nothing and keeps no state between calls; the persistent state of a decode loop
 *   (summaries, alive mask, previous selection) lives in caller buffers.
 * Memory spaces. Struct arguments (bs_dims, bs_kv, bs_head_cfg) are HOST structs
 *   passed by pointer; every array they point to, and every array argument, is
 *   DEVICE memory unless the parameter says otherwise.
 * Asynchrony. Each call validates its host-visible arguments, enqueues kernels on
 *   `stream` and returns. Nothing waits for the GPU. The kernels run on the device that
 *   is current: `stream` must be one of its streams and every pointer valid there.
 * Errors. Host-detected problems (null pointers, bad shapes, misalignment, a too
 *   small workspace) return a non-zero bs_status before anything is enqueued.
 *   A failed launch returns BS_ERR_CUDA. Problems only the device can see (a page
 *   index outside the pool, a per-unit configuration that breaks a rule below, a
 *   capacity overflow, a bounded wait that ran out) store the first such code into
 *   `*dev_status` (an int32 device word the caller zeroes; atomicCAS from 0) and the
 *   offending unit's work is skipped, never performed out of bounds. Read it after
 *   synchronising.
 * Determinism. Results are bitwise reproducible run to run (no floating-point
 *   atomics; partials merge in a fixed order). Selections never depend on the other
 *   units of the batch; attention outputs depend on them only through the attention's
 *   plan (bs_sparse_decode_attn), in the last bits.
 *
 * Data layout (dims below are the fields of bs_dims)
 * ----------------------------------------------------
 *   K, V pools     [n_pages][page_size=16][head_dim], kv_dtype; 16-byte aligned base.
 *   K, V scales    float32 [n_pages], 8-bit caches only: a page belongs to one unit, so
 *                  this is a scale for each block of 16 tokens and KV head. The value of
 *                  a code c of page p is c * scale[p] (finite, >= 0).
 *   page_table     int32 [units][max_pages_per_unit]; entry p of unit u is the
 *                  physical page holding tokens [16p, 16p+16) of that unit.
 *   seq_lens       int32 [batch]; T = tokens in the cache including the current
 *                  decode token, which sits at position T-1.
 *   q              [batch][n_q_heads][head_dim], q_dtype; query heads
 *                  [h_kv*G, (h_kv+1)*G) share KV head h_kv (G = n_q_heads/n_kv_heads).
 *   summaries      float32; unit u's sub-block j occupies
 *                  summaries[sum_off[u] + j*head_dim ... + head_dim).
 *   scores         float32 [units][max_blocks_per_unit].
 *   evict_logits   float32 [units][max_blocks_per_unit] (dual units only).
 *   alive          uint8   [units][max_blocks_per_unit] (dual units only; start at 1).
 *   sel_idx        int32   [units][max_sel_per_unit], ascending, padded with -1.
 *   sel_cnt        int32   [units].
 *   out            float32 [batch][n_q_heads][head_dim];  lse float32 [batch][n_q_heads].
 */
#ifndef BSATTN_H_
#define BSATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t. NULL selects the legacy default stream. */
typedef struct CUstream_st *bs_stream_t;

typedef enum {
  BS_OK = 0,
  BS_ERR_INVALID_ARG = 1,   /* null pointer, value out of its documented range */
  BS_ERR_SHAPE = 2,         /* unsupported head_dim, group size or page size */
  BS_ERR_ALIGN = 3,         /* a pointer or offset breaks its alignment rule */
  BS_ERR_CAPACITY = 4,      /* a buffer or row is too small for the data */
  BS_ERR_CUDA = 5,          /* a CUDA launch failed */
  BS_ERR_DEVICE_BOUNDS = 6, /* (device) a page index outside the pool or table */
  BS_ERR_TIMEOUT = 7        /* (device) a bounded wait ran out */
} bs_status;

/* BS_E4M3 (float8 e4m3fn: 4 exponent bits, 3 mantissa bits, largest value 448, no
 * infinities) and BS_INT8 (signed, -127..127) are storage types of the K and V pools
 * only (bs_dims.kv_dtype), each with one scale per page; queries are BS_BF16 or BS_FP32. */
typedef enum { BS_BF16 = 0, BS_FP32 = 1, BS_E4M3 = 2, BS_INT8 = 3 } bs_dtype;

/* Head classes (Fluxion, Kerninzichten item 2: streaming vs retrieval heads;
 * NOSA, Dual-Selection-Mechanismus: query-aware plus query-agnostic selection). */
typedef enum { BS_STREAMING = 0, BS_RETRIEVAL = 1, BS_DUAL = 2 } bs_head_class;

/* How the G query heads of a group combine their max-pooled block scores
 * (Fluxion, Systeemcomponenten: GQA handled at group level). */
typedef enum { BS_GROUP_MAX = 0, BS_GROUP_MEAN = 1 } bs_group_reduce;

/* Shapes and capacities, host struct. Supported: head_dim 64 or 128, page_size 16,
 * G = n_q_heads / n_kv_heads in 1..8, max_blocks_per_unit <= 16384, and pools of at
 * most (2^31 - 1) / 16 pages (pool rows are signed 32-bit tensor-map coordinates);
 * larger values return BS_ERR_CAPACITY. */
typedef struct {
  int32_t batch, n_q_heads, n_kv_heads, head_dim, page_size;
  int32_t max_pages_per_unit;        /* page-table row length */
  int32_t max_blocks_per_unit;       /* row length of scores / evict_logits / alive */
  int32_t max_sel_per_unit;          /* row length of sel_idx and of setdiff outputs */
  int32_t max_subs_per_unit;         /* upper bound on ceil(T/s) over units (grid sizing) */
  int32_t max_gather_pages_per_unit; /* upper bound on pages covered by a selection */
  int64_t n_pages;                   /* pages in each of the K and V pools */
  bs_dtype kv_dtype, q_dtype;
} bs_dims;

/* Paged KV cache: device pointers. k_scale and v_scale are the page scales of an 8-bit
 * cache (kv_dtype BS_E4M3 or BS_INT8; required there, v_scale not by
 * bs_build_block_summaries) and not read otherwise: a caller built when the struct ended at
 * seq_lens may pass that. */
typedef struct {
  const void *k_pool, *v_pool;
  const int32_t *page_table;
  const int32_t *seq_lens;
  const float *k_scale, *v_scale;   /* [n_pages] */
} bs_kv;

/* Per-unit head properties, struct of arrays of length batch * n_kv_heads, device
 * memory (host memory for bs_check_head_cfg only). These are the outputs of the
 * pages' head-property predictor and granularity-budget selector, taken as inputs.
 * Rules (checked by bs_check_head_cfg on the host and by every kernel on the device):
 *   cls in {STREAMING, RETRIEVAL, DUAL};  g % 16 == 0;  g % s == 0 and g/s a power
 *   of two <= 64;  k >= 0;  0 <= k_e <= k (k_e used by DUAL units only);
 *   sink_tokens >= 0;  local_tokens >= 1 (the current token is always attended);
 *   sum_off % 4 == 0 (16-byte aligned summary rows); sum_rows >= ceil(T/s).
 * Selection: forced blocks F = [0, ceil(sink/g)) U [floor(max(0,T-local)/g), ceil(T/g));
 * candidates C = complete blocks outside F; streaming: S = F; retrieval: S = F plus
 * the k best of C; dual: S = F plus Gamma_e (k_e best alive blocks of C by eviction
 * logit) plus Gamma_q (k - k_e best of C minus Gamma_e by score). Ties go to the
 * lower block index. */
typedef struct {
  const int32_t *cls, *block_tokens, *sub_tokens, *k_total, *k_evict;
  const int32_t *sink_tokens, *local_tokens;
  const int64_t *sum_off;   /* float offset of unit u's first summary row */
  const int32_t *sum_rows;  /* summary rows reserved for unit u */
} bs_head_cfg;

/* Host-side check of a head configuration whose nine arrays are in HOST memory.
 * `seq_lens_host` (length batch) are the largest lengths the caller will use.
 * Returns BS_OK or the first rule broken (BS_ERR_INVALID_ARG, BS_ERR_ALIGN,
 * BS_ERR_CAPACITY). Launches nothing. */
bs_status bs_check_head_cfg(const bs_dims *dims, const bs_head_cfg *cfg_host,
                            const int32_t *seq_lens_host);

/* a1. Sub-block key summaries.
 * NOSA, "Blockweise Implementierung": mean pooling inside sub-blocks is the first
 * stage of the two-stage pooling; NOSI fuses the pooling with the KV write.
 * For each unit of sequence b, recomputes every sub-block j that holds a token of
 * [tok_begin[b], seq_lens[b]): kbar_j = (1/n_j) sum of K[t] over the n_j tokens of
 * [j*s, min((j+1)*s, T)), summed in token order in fp32. A decode step passes
 * tok_begin = T-1 (one sub-block per unit); a prefill passes 0. The result does not
 * depend on how the range was split across calls. 8-bit caches: K[t] is its code times
 * its page's scale, and because an append may round the codes of the page it starts in
 * again (bs_quant_append), every sub-block with a token of the page that holds
 * tok_begin[b] is recomputed too.
 * tok_begin: device int32 [batch]. max_new_tokens (host): an upper bound on
 * seq_lens[b] - tok_begin[b], used only to size the grid. */
bs_status bs_build_block_summaries(const bs_dims *dims, const bs_kv *kv, const bs_head_cfg *cfg,
                                   const int32_t *tok_begin, int32_t max_new_tokens,
                                   float *summaries, int32_t *dev_status, bs_stream_t stream);

/* a2. Block scores.
 * NOSA, "Blockweise Implementierung": max pooling at block level over the sub-block
 * means; Fluxion, "Granularity-Budget Selector": one selection per GQA group.
 * For every retrieval or dual unit and every candidate block c:
 *   S[c] = reduce_{h in group} max_{j in sub-blocks of c} (q_h . kbar_j) / sqrt(d),
 * reduce = max (BS_GROUP_MAX) or mean (BS_GROUP_MEAN). Entries of the row outside
 * the candidate range are written as -inf; rows of streaming units are not touched. */
bs_status bs_score_blocks(const bs_dims *dims, const void *q, const bs_head_cfg *cfg,
                          const int32_t *seq_lens, const float *summaries,
                          bs_group_reduce group_reduce, float *scores, int32_t *dev_status,
                          bs_stream_t stream);

/* a3. Block selection.
 * Fluxion, Kerninzichten item 2 (streaming vs retrieval heads, per-head budget and
 * granularity); NOSA, Dual-Selection-Mechanismus (Gamma_q, Gamma_e and the strict
 * eviction rule: a block of C that is not in Gamma_e is marked dead in `alive` and
 * never enters Gamma_e again) and ED-DMA (selection on pre-exponential logits).
 * Writes S of every unit, ascending, into sel_idx (padded with -1) and |S| into
 * sel_cnt. evict_logits and alive may be NULL when no unit is DUAL (a DUAL unit
 * with NULL arrays reports BS_ERR_INVALID_ARG on the device). Scores and logits are
 * compared exactly as float32 order keys. */
bs_status bs_select_topk(const bs_dims *dims, const bs_head_cfg *cfg, const int32_t *seq_lens,
                         const float *scores, const float *evict_logits, uint8_t *alive,
                         int32_t *sel_idx, int32_t *sel_cnt, int32_t *dev_status,
                         bs_stream_t stream);

/* a4. Sparse decode attention.
 * Fluxion, Probleemstelling item 1 (sparse attention over the selected KV blocks)
 * and Kerninzichten item 3 (bound by data movement). For each query head h of unit
 * u, over the tokens U of the selected blocks (each clipped to t < T):
 *   out_h = sum_t softmax_t(x_h(t)) V[t],  lse_h = log sum_t exp(x_h(t)),
 *   x_h(t) = q_h . K[t] / sqrt(d) + e[u][t / g]  (e = 0 when evict_bias is NULL).
 * evict_bias (device fp32 [units][max_blocks_per_unit], or NULL for plain softmax)
 * is the ED-DMA variant (NOSA, "ED-DMA": blocks are chosen on the eviction head's
 * pre-exponential logits and the exponential is applied only in the attention; here
 * read as each block's logit added to the attention logit of each of its tokens, so
 * exp(e) weights the block's tokens). Entries must be finite or -inf; a block at -inf
 * drops out, and a unit whose tokens all drop out gets a zero row and lse = -inf. Over
 * bf16 and fp32 caches an entry times log2(e) must be finite in fp32 too (magnitudes up
 * to 2.35e38; lower entries drop the block); over 8-bit caches every finite entry counts,
 * the type's lowest among them. Only the entries of selected blocks are read.
 * Split-KV: a unit's gathered pages are cut into contiguous pieces; each piece keeps an
 * fp32 online softmax and the partials are merged by log-sum-exp in a fixed order, so
 * the result does not depend on timing. Two plans, chosen from the dims:
 *   - cluster mode (max_gather_pages_per_unit <= 1024 with at most 19 units, at least
 *     304 units, or max_gather_pages_per_unit <= 256): every unit gets S splits, S the
 *     largest power of two <= 16 with units * S <= two CTAs per SM; the S CTAs of a
 *     unit form one thread-block cluster and merge through distributed shared memory;
 *     split j takes pages [j*p, (j+1)*p), p = ceil(pages / S);
 *   - workspace mode (the rest): each unit's splits are sized by its own page count,
 *     p = max(4 * ceil(pages / 128), m) pages per split (m = 24, or 4 when
 *     max_gather_pages_per_unit > 1024), so at most 32 splits; partials go through the
 *     workspace and the last split to finish merges them. In the fused step
 *     (bs_decode_step) only the splits that can hold pages take part: at most
 *     ceil(min(n_blk, |forced| + k_total) * block_tokens / 16 / m) when m = 24 (the
 *     others leave at once; the merge is the same, as their records were empty).
 * A unit's plan depends on its own sizes only, so a sub-batch launched with the same S
 * gives bitwise the same per-unit results as the full batch.
 * 8-bit caches: K[t] and V[t] are codes times their page's scale. Codes are exact in
 * fp16; queries and weights enter as fp16 parts hi + lo, a query element within 2^-22 of
 * itself or 2^-39 of its row's largest element, a weight within 2^-22 of itself or 2^-38
 * of its page's largest weight (a page whose largest is below 2^-112 of the unit's: 2^-150
 * of the unit's); sums and scales are fp32, whatever the scales. A
 * page whose block logit is -inf is not read; NaN codes in tokens past T do not count.
 * Their splits differ from the above: in cluster mode S is halved while a selection of
 * max_gather_pages_per_unit would leave a split fewer than 8 pages; in workspace mode up
 * to 1024 pages, m = max(8, units * max_gather_pages_per_unit / (2 CTAs per SM), up to a
 * multiple of 4), so that the splits fill one wave, and m = 40 in the fused step.
 * workspace: device scratch of at least bs_workspace_size(dims) bytes, 16-byte
 * aligned. It starts with four int32 words per unit (padded to 16 bytes): the fused
 * step's selection tickets, the attention's arrival tickets, the fused step's published
 * selections and the epochs of the last ones taken. These must be zero before the first
 * call: zero the workspace once after allocating it. Every call that completes leaves
 * the tickets zero again; after a call that reported BS_ERR_TIMEOUT, zero the workspace
 * again. Then, by mode: cluster mode the fused step's page lists (int32 [units]
 * [max_gather_pages_per_unit]); workspace mode 32 split records of G * (head_dim + 4)
 * floats per unit. The rest is overwritten per call.
 * Calls that share a workspace must not run concurrently. */
bs_status bs_sparse_decode_attn(const bs_dims *dims, const void *q, const bs_kv *kv,
                                const bs_head_cfg *cfg, const int32_t *sel_idx,
                                const int32_t *sel_cnt, const float *evict_bias, float *out, float *lse,
                                void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                bs_stream_t stream);

/* a4, without a workspace argument. The pages have no counterpart of this call; it
 * exists for callers that cannot allocate device memory for a workspace: a plugin
 * inside a host engine that owns every allocation and offers no allocator, or a
 * serving loop that may not call cudaMalloc once it runs (the call synchronises the
 * device and can fail under memory pressure). Same inputs, outputs and results as
 * bs_sparse_decode_attn, but the workspace it would take (arrival counters and, for
 * selections above 1024 pages per unit, split partials) lives in a fixed 8 MiB array
 * inside this library's device memory, which every GPU that loads the library keeps
 * until the process exits.
 * Limit: bs_workspace_size(dims) must not exceed 8 MiB; larger dims return
 * BS_ERR_CAPACITY before anything is enqueued. In workspace mode the split records
 * take 67.6 KB per unit at head_dim 128, G = 4: at most 124 units (62 at G = 8); in
 * cluster mode (counters and page lists, 16 + 4 * max_gather_pages_per_unit bytes per
 * unit) 2,040 units at 1024 pages per unit.
 * The first call on each device looks up the array's device address with that device
 * current and caches it; make that first call before any stream capture. The cached
 * address belongs to the device's context at that time: after cudaDeviceReset (or
 * anything else that destroys and re-creates the device's primary context) it is stale,
 * so do not call this entry point again in that process.
 * Every call clears the arrival counters on `stream` before its kernel. All calls
 * share the one array per device, so calls whose kernels overlap on the GPU (on
 * different streams, or from different threads) race and corrupt each other's
 * results; serialise them. Allocates nothing: no cudaMalloc, cudaFree or allocating
 * library routine. */
bs_status bs_sparse_decode_attn_noalloc(const bs_dims *dims, const void *q, const bs_kv *kv,
                                        const bs_head_cfg *cfg, const int32_t *sel_idx,
                                        const int32_t *sel_cnt, const float *evict_bias, float *out,
                                        float *lse, int32_t *dev_status, bs_stream_t stream);

/* a5. Set-difference of selections.
 * NOSA, "2. System: NOSI": set-difference kernels drive block swapping.
 * added = cur \ prev and removed = prev \ cur per unit, both ascending, padded with
 * -1 to max_sel_per_unit; counts in added_cnt / removed_cnt. prev_cnt[u] = 0 gives
 * added = cur (first step). Input lists must be ascending and duplicate-free. */
bs_status bs_block_setdiff(const bs_dims *dims, const int32_t *prev_idx, const int32_t *prev_cnt,
                           const int32_t *cur_idx, const int32_t *cur_cnt, int32_t *added,
                           int32_t *added_cnt, int32_t *removed, int32_t *removed_cnt,
                           int32_t *dev_status, bs_stream_t stream);

/* Buffers of one decode step of one layer for bs_decode_step (device pointers). */
typedef struct {
  const void *q;              /* [batch][n_q_heads][head_dim], q_dtype */
  float *summaries;           /* as for bs_build_block_summaries; the sub-block holding T-1 is rewritten */
  float *scores;              /* [units][max_blocks_per_unit] scratch: this step's candidate scores */
  const float *evict_logits;  /* [units][max_blocks_per_unit]; may be NULL when no unit is DUAL */
  uint8_t *alive;             /* [units][max_blocks_per_unit], in/out; may be NULL when no unit is DUAL */
  const float *evict_bias;    /* the attention's ED-DMA block logits, as for bs_sparse_decode_attn (NULL:
                                 plain softmax); may be evict_logits itself */
  const int32_t *prev_idx, *prev_cnt;  /* previous step's selection (prev_cnt 0 at the first step) */
  int32_t *cur_idx, *cur_cnt;          /* this step's selection (written); must not alias prev */
  int32_t *added, *added_cnt, *removed, *removed_cnt;  /* set-difference (written) */
  float *out, *lse;           /* attention output (written) */
  void *workspace;            /* as for bs_sparse_decode_attn: bs_workspace_size bytes, counters zeroed once */
  size_t workspace_bytes;
  int32_t *dev_status;
} bs_step_io;

/* One decode step of one layer: a1, a2, a3, a4 and a5 in two launches (three in the
 * attention's workspace mode when a unit can have more than 2048 candidate blocks;
 * bs_decode_step_launches says which).
 * The results are those of bs_score_blocks, bs_select_topk, bs_sparse_decode_attn and
 * bs_block_setdiff called in that order, plus the a1 update of the one sub-block that
 * holds token T-1 (call bs_build_block_summaries first if more than one token was
 * appended since the last step). Only the order of fp32 additions inside the
 * attention may differ from the separate calls (streaming units split their pages
 * differently), which stays within rounding.
 * Launch 1 scores every candidate tile (one or several 64-row tiles per CTA); the
 * unit's first CTA also updates a1 (that sub-block lies in the forced tail block,
 * which no score of this step reads); the unit's CTA that finishes last (an arrival
 * ticket) selects, publishes the selection (once the row and the page list are
 * written, cur_cnt receives the count and the unit's published word in the workspace
 * receives (epoch << 16) | count with a release store, the epoch one past the one the
 * attention last took, so a count left from an earlier step can never be taken for
 * this step's) and writes the set-difference. Launch 2 is the attention, launched as a
 * programmatic dependent: streaming units' pages need no selection and are attended
 * before launch 1 ends; the others wait, bounded, for their unit's published word.
 * With three launches: launch 1 scores the tiles of all units as one stream in equal
 * shares over a persistent grid; launch 2 runs one 1024-thread CTA per unit that
 * updates a1, waits for launch 1 (streaming units do not wait), selects, publishes and
 * writes the set-difference; launch 3 is the attention as above.
 * The launches may begin before the work ahead of them in `stream` has finished;
 * before waiting for it they read only the per-unit head configuration (cfg arrays),
 * so those must not be written by the kernel immediately before this call. Everything
 * else is read after that work has finished. Requires max_sel_per_unit <= 4096.
 * Errors as for the separate calls; after BS_ERR_TIMEOUT zero the workspace again. */
bs_status bs_decode_step(const bs_dims *dims, const bs_kv *kv, const bs_head_cfg *cfg, const bs_step_io *io,
                         bs_group_reduce group_reduce, bs_stream_t stream);

/* ------------------------------------------------------------------------------
 * Set-difference-driven block swap into a GPU block cache ("Technisches Resümee:
 * NOSA", Methodik / 2. System: NOSI: the KV cache in minimal block units, set-
 * difference kernels for block swapping, host-to-device transfer kernels over
 * Unified Virtual Addressing; Lokalitätsgarantie: blocks kept from one step to the
 * next stay in the GPU cache).
 *
 * The full KV lives in host memory; the GPU holds, per unit, `slots_per_unit` block
 * slots of `pages_per_slot` pages each (pages_per_slot >= g/16 of every unit). A
 * block is resident exactly while it is selected: after the swap of a step, the
 * cached blocks of unit u are that step's selection.
 * ------------------------------------------------------------------------------ */

/* Host-resident paged KV. The pools must be pinned host memory that the device can
 * read (under unified addressing the host pointer of cudaHostAlloc / cudaHostRegister
 * memory is that device pointer); `page_table` is DEVICE memory. */
typedef struct {
  const void *k_pool, *v_pool;   /* [n_pages][16][head_dim], kv_dtype, 16-byte aligned */
  const int32_t *page_table;     /* [units][max_pages_per_unit]: host page of each logical page */
  int64_t n_pages;
} bs_host_kv;

/* GPU block cache (all device memory). Slot s of unit u owns device pages
 * (u * slots_per_unit + s) * pages_per_slot + p, p < pages_per_slot, in `k_pool` and
 * `v_pool` ([units * slots_per_unit * pages_per_slot][16][head_dim]). `page_table`
 * ([units][max_pages_per_unit]) maps each logical page of a cached block to its
 * device page and every other entry to -1; with it and the cache pools, bs_kv
 * describes the cache for bs_sparse_decode_attn. slot_block / block_slot are the
 * cache state (in/out; start with all -1). */
typedef struct {
  void *k_pool, *v_pool;
  int32_t *page_table;          /* [units][max_pages_per_unit] */
  int32_t *slot_block;          /* [units][slots_per_unit]: block held by a slot, -1 free */
  int32_t *block_slot;          /* [units][max_blocks_per_unit]: slot of a block, -1 not cached */
  int32_t slots_per_unit;       /* 1..4096, at least the largest selection */
  int32_t pages_per_slot;       /* >= g/16 of every unit */
} bs_block_cache;

/* (Not for 8-bit caches: BS_ERR_INVALID_ARG.)
 * One step's swap for every unit: first every block of `removed` leaves the cache
 * (its slot is freed, its page-table entries become -1); then the blocks of `added`
 * (ascending) take the free slots in ascending slot order, their page-table entries
 * are set, and the pages of each added block that hold tokens (< T) are copied, K and
 * V, from the host pools into the block's slot (16-byte loads over the host link, no
 * staging copy). The page holding token T-1 (the token appended this step) is copied
 * and mapped too when its block was already cached, so the cache stays current as the
 * tail block grows. `added` / `removed` and their counts are bs_block_setdiff's output
 * (or bs_decode_step's); seq_lens (device, [batch]) give T. Two launches: the
 * bookkeeping (one CTA per unit), then the copies (one CTA per added block and one
 * per unit for the appended token's page).
 * Device-side errors: a block index outside [0, max_blocks_per_unit) or a host page
 * outside the host pool sets BS_ERR_DEVICE_BOUNDS (that block is skipped); more added
 * blocks than free slots sets BS_ERR_CAPACITY (the excess is not cached). */
bs_status bs_block_swap(const bs_dims *dims, const bs_head_cfg *cfg, const int32_t *seq_lens,
                        const bs_host_kv *host, const bs_block_cache *cache, const int32_t *added,
                        const int32_t *added_cnt, const int32_t *removed, const int32_t *removed_cnt,
                        int32_t *dev_status, bs_stream_t stream);

/* ------------------------------------------------------------------------------
 * CPU/GPU split attention ("Technische Samenvatting: Fluxion", Kerninzichten item 3:
 * sparse attention is bound by data movement; Systeemcomponenten: the CPU and the GPU
 * serve one step in parallel). A unit's selection may be split into two block subsets:
 * one attended on the GPU (bs_sparse_decode_attn, e.g. over the block cache), the
 * other on the host cores over host-resident KV (bs_cpu_sparse_attn); bs_lse_merge
 * combines the two partial results into the attention over the union.
 * ------------------------------------------------------------------------------ */

/* Host copies of the tables the CPU side reads (all HOST memory). */
typedef struct {
  const int32_t *page_table;    /* [units][max_pages_per_unit]: host page of each logical page */
  const int32_t *seq_lens;      /* [batch]: T */
  const int32_t *block_tokens;  /* [units]: g */
  const float *evict_bias;      /* NULL, or the ED-DMA block logits [units][max_blocks_per_unit] as for
                                   bs_sparse_decode_attn */
  int32_t max_blocks_per_unit;  /* row length of evict_bias (used only when it is set) */
} bs_host_tables;

/* (Not for 8-bit caches: BS_ERR_INVALID_ARG.)
 * Attention of each unit's listed blocks (tokens clipped to T) on the host cores,
 * fp32 arithmetic, units spread over n_threads threads; synchronous. Everything is
 * HOST memory: q ([batch][n_q_heads][head_dim], q_dtype), the pools of `kv` (its
 * page_table field is not used; `tables` gives the host page table), sel_idx
 * ([units][max_sel_per_unit], ascending), sel_cnt ([units]), out ([batch][n_q_heads]
 * [head_dim] fp32) and lse ([batch][n_q_heads] fp32, natural log; -inf and a zero row
 * for a unit with nothing to attend). Returns BS_ERR_DEVICE_BOUNDS (after finishing
 * the other units) if a block or page index is out of range. */
bs_status bs_cpu_sparse_attn(const bs_dims *dims, const void *q, const bs_host_kv *kv, const bs_host_tables *tables,
                             const int32_t *sel_idx, const int32_t *sel_cnt, float *out, float *lse,
                             int n_threads);

/* out, lse = the log-sum-exp merge of two partial attention results over disjoint
 * token sets of every query head (device memory, layout of out / lse above): with
 * M = max(lse_a, lse_b), w = exp(lse - M), out = (w_a o_a + w_b o_b) / (w_a + w_b) and
 * lse = M + log(w_a + w_b); a side with lse = -inf contributes nothing, and two
 * empty sides give a zero row and -inf. out / lse may be out_a / lse_a (in place). */
bs_status bs_lse_merge(const bs_dims *dims, const float *out_a, const float *lse_a, const float *out_b,
                       const float *lse_b, float *out, float *lse, bs_stream_t stream);

/* ------------------------------------------------------------------------------
 * Writing an 8-bit cache. ("Technisches Resümee: NOSA", 2. System: NOSI keeps the cache
 * in minimal block units and works on it as tokens are written; the storage type is not
 * the page's.)
 * ------------------------------------------------------------------------------ */

/* K and V pools that a call writes, with the page scales of an 8-bit cache (NULL and
 * unused otherwise). Device pointers. */
typedef struct {
  void *k_pool, *v_pool;        /* [n_pages][16][head_dim], kv_dtype, 16-byte aligned */
  float *k_scale, *v_scale;     /* [n_pages] */
} bs_pools;

/* Quantises new tokens into the pages of an 8-bit cache (kv_dtype BS_E4M3 or BS_INT8).
 * Token t of sequence b, tok_begin[b] <= t < seq_lens[b], is row row_begin[b] + t -
 * tok_begin[b] of k_new and v_new: n_rows rows of row_stride elements (q_dtype: BS_BF16
 * or BS_FP32), KV head h at [h * head_dim, (h + 1) * head_dim), so that K and V may be
 * columns of one fused projection's output. It goes to slot t % 16 of the page that
 * page_table names for t / 16; that page must be no other unit's (see bs_pages_fork).
 * For each page, K and V apart, with x the new values of the page:
 *   a = the largest |x| that is finite;  f(a) = 0 when a = 0, else
 *     BS_E4M3: the smallest power of two with a / f(a) <= 448,
 *     BS_INT8: a / 127 rounded to fp32;   both at least 2^-126;
 *   s = f(a) when the page held no token of the sequence before, else max(old scale, f(a));
 *   code of x = Q(x / s), the fp32 quotient rounded to the nearest code, ties to even,
 *     and cut to the largest magnitude (448, 127); NaN gives NaN (BS_E4M3) or 0 (BS_INT8);
 *     0 when s = 0;
 *   when s grew, the codes c already there become Q(c * old scale / s) (in fp32).
 * Slots of the page past seq_lens[b] keep what they hold. With BS_E4M3 the scales are
 * powers of two: rounding a page again changes only codes that become subnormal.
 * page_table int32 [units][max_pages_per_unit]; seq_lens, tok_begin, row_begin int32
 * [batch]; tok_begin[b] = seq_lens[b] appends nothing for b (row_begin[b] is not read).
 * max_new_tokens (host): an upper bound on seq_lens[b] - tok_begin[b]; sizes the grid
 * only. k_new and v_new 16-byte aligned, row_stride >= n_kv_heads * head_dim and a
 * multiple of 16 bytes. A sequence whose rows or lengths do not fit (tok_begin < 0 or
 * above seq_lens: BS_ERR_INVALID_ARG; more pages than a row: BS_ERR_CAPACITY; rows
 * outside [0, n_rows): BS_ERR_DEVICE_BOUNDS) is skipped, and so is a page outside the
 * pool (BS_ERR_DEVICE_BOUNDS). One launch; bitwise reproducible. */
bs_status bs_quant_append(const bs_dims *dims, const bs_pools *pools, const int32_t *page_table,
                          const int32_t *seq_lens, const int32_t *tok_begin, const int32_t *row_begin,
                          const void *k_new, const void *v_new, int64_t row_stride, int64_t n_rows,
                          int32_t max_new_tokens, int32_t *dev_status, bs_stream_t stream);

/* ------------------------------------------------------------------------------
 * Pages of a cache, handed out and taken back on the device. A page is free when no
 * page-table entry holds it (ref_count 0). Nothing waits for the GPU, so these calls
 * stand between decode steps, in a captured graph too. Calls on one map, and other
 * calls that read or write what it points to, must be ordered (one stream). The calls
 * work on the table only; bs_pages_copy then moves the data, once for each layer that
 * shares the table. They use batch, n_kv_heads, max_pages_per_unit and n_pages of the
 * dims (which must be valid as a whole); any kv_dtype.
 * Which free page is taken is fixed: the k-th page asked for (ascending unit, then
 * ascending logical page) gets the k-th lowest free page.
 * reserve and fork do all of their work or none: a call that reports an error leaves the
 * map as it was (and *count = 0).
 * ------------------------------------------------------------------------------ */

/* Device pointers; all in/out. A table entry is a page, or -1 for none; anything else lies
 * outside the pool (reserve, which writes every entry that holds no page, puts a page in place
 * of any below 0). */
typedef struct {
  int32_t *page_table;  /* [units][max_pages_per_unit]: page of each logical page, -1 none */
  int32_t *ref_count;   /* [n_pages]: page-table entries that hold the page, >= 0 */
  int32_t *seq_lens;    /* [batch]: tokens of each sequence (0: an empty slot) */
} bs_page_map;

/* Pages to copy (device memory, written by fork and compact): *count pairs (source page,
 * destination page). Within one list no page is a destination twice or a source and a
 * destination. */
typedef struct {
  int32_t *pairs;       /* [capacity][2], 8-byte aligned */
  int32_t *count;
  int32_t capacity;     /* host value: pairs that fit */
} bs_page_copies;

/* Scratch of reserve, fork and compact for these dims (0 on bad dims): 16-byte aligned,
 * overwritten by every call, needs no clearing. Calls that share it must be ordered. */
size_t bs_pages_workspace_size(const bs_dims *dims);

/* Every entry of a unit of sequence b below ceil(new_lens[b] / 16) that holds no page
 * gets a free one (ref_count 1). new_lens (device int32 [batch]) may be map->seq_lens;
 * <= 0 asks for nothing; the lengths themselves are not written. Too few free pages, or
 * a length beyond the row: BS_ERR_CAPACITY, nothing changes. Two launches. */
bs_status bs_pages_reserve(const bs_dims *dims, const bs_page_map *map, const int32_t *new_lens, void *workspace,
                           size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream);

/* Sequence slot dst[i] becomes a copy of sequence src[i], for i < n (device int32 [n]; a
 * negative src[i] or dst[i] skips i): its length is src's, its units share src's full
 * pages (their counts grow), and the partial last page, where tokens will be appended,
 * gets a free page of its own with a pair (src's page, the free page) in `copies`, in
 * order of i, then KV head. Logical pages of src past its length are not shared; an
 * entry of src that holds no page (-1) stays -1. A decode loop's other state of a unit
 * (summaries, alive mask, previous selection) is the caller's to copy.
 * One src may have many dst. Every dst must be an empty slot (no page in its rows), named
 * once, and be no src of the same call; both in [0, batch): else BS_ERR_INVALID_ARG.
 * BS_ERR_CAPACITY for too few free pages or a src length beyond its row (src length < 0:
 * BS_ERR_INVALID_ARG), BS_ERR_DEVICE_BOUNDS for a shared entry outside the pool or a
 * free page (count 0): nothing changes. copies->capacity >= n * n_kv_heads (checked on
 * the host: BS_ERR_CAPACITY); 1 <= n <= batch. Two launches. */
bs_status bs_pages_fork(const bs_dims *dims, const bs_page_map *map, const int32_t *src, const int32_t *dst, int32_t n,
                        const bs_page_copies *copies, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        bs_stream_t stream);

/* The sequences seqs[i], i < n (device int32 [n]), give up their pages: each entry of
 * their rows becomes -1 and its page's count falls by one; their lengths become 0. A
 * negative seqs[i] is skipped, a sequence named twice is freed once. (A decode call that
 * finds a length of 0 reports BS_ERR_INVALID_ARG for that sequence and does the others.)
 * An entry outside the pool, or whose page has count 0, is dropped with
 * BS_ERR_DEVICE_BOUNDS; a seqs[i] >= batch is skipped with BS_ERR_INVALID_ARG; the rest
 * is done. 1 <= n <= batch. One launch. */
bs_status bs_pages_free(const bs_dims *dims, const bs_page_map *map, const int32_t *seqs, int32_t n,
                        int32_t *dev_status, bs_stream_t stream);

/* Moves the pages in use together: with N pages in use (count > 0), the k-th lowest of
 * those at or above N moves to the k-th lowest free page below N. Table entries and
 * counts follow, the moves are listed in `copies`, and *n_live (device int32) = N: pages
 * [N, n_pages) are free. At most n_pages / 2 moves; more than copies->capacity:
 * BS_ERR_CAPACITY and nothing moves (*count = 0, *n_live is still written). An entry
 * outside the pool, or one at or above N on a free page, is left as it is with
 * BS_ERR_DEVICE_BOUNDS; the rest is done. Two launches. */
bs_status bs_pages_compact(const bs_dims *dims, const bs_page_map *map, const bs_page_copies *copies, int32_t *n_live,
                           void *workspace, size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream);

/* Copies the listed pages of one layer's K and V pools (any kv_dtype; 8-bit caches: and
 * their scales). copies->count is read on the device, at most copies->capacity pairs are
 * taken. A pair with a page outside the pool is skipped with BS_ERR_DEVICE_BOUNDS. One
 * launch. */
bs_status bs_pages_copy(const bs_dims *dims, const bs_pools *pools, const bs_page_copies *copies, int32_t *dev_status,
                        bs_stream_t stream);

/* ------------------------------------------------------------------------------
 * Prompts and drafted tokens. bs_rope_append turns a projection's rows into queries and
 * keys; bs_prefill_attn attends new tokens to the cache that holds them; a tree of drafts
 * is attended by bs_tree_decode_attn while its K and V stay outside the cache, and
 * bs_tree_commit appends those that were accepted. (A draft enters no page before it is
 * accepted: pages may be shared, and a page scale of an 8-bit cache only grows.)
 * Rows. New tokens of all sequences are packed rows; those of sequence b start at row
 * row_begin[b]. A row holds the heads of one token; row_stride (elements) lets q, k and v
 * be columns of one fused projection's output. Rows that belong to no sequence are
 * neither read for a result nor written. A call with n_rows = 0 does nothing (a commit reports
 * sequences that name rows all the same), and the arrays that have a place a row may be NULL (in
 * bs_quant_append too).
 * ------------------------------------------------------------------------------ */

/* Norm and rotation of queries and keys (host struct; device pointers). Pair i, i <
 * rot_dim / 2, of a head at position p turns by the angle p * inv_freq[i]; its elements are
 * i and i + rot_dim / 2, or 2i and 2i + 1 (interleaved). Elements from rot_dim on are not
 * rotated. */
typedef struct {
  const double *inv_freq;  /* [rot_dim / 2], radians a position, finite */
  int32_t rot_dim;         /* 16 .. head_dim, a multiple of 16 */
  int32_t interleaved;     /* 0 or 1 */
  float magnitude;         /* cosines and sines are multiplied by it (1: a plain rotation) */
  const float *q_weight, *k_weight;  /* norm weights [head_dim], or NULL: no norm of queries / keys */
  float eps;               /* >= 0, finite */
} bs_rope;

/* For each row r and each query or key head x of it, in fp32:
 *   x' = x * rsqrt(mean(x^2) + eps) * weight (x where the weight is NULL);
 *   (a, b) of each pair -> m (a cos - b sin), m (b cos + a sin), m = magnitude;
 * rounded once, to q_dtype in q_out and k_out, to kv_dtype in the cache. The angle keeps
 * its fraction of a turn to 2^-24 whatever the position (below 2^24) where |inv_freq| is at most 1,
 * to 2^-23 up to 32.
 * q rows: n_q_heads * head_dim elements at q + r * row_stride; k and v rows likewise with
 * n_kv_heads. positions int32 [n_rows], 0 .. 2^24 - 1. row_seq int32 [n_rows]: the row's
 * sequence, < 0 for a padding row, which is skipped; NULL (only without pools): no
 * padding. q_out [n_rows][n_q_heads][head_dim], k_out [n_rows][n_kv_heads][head_dim],
 * q_dtype, packed, 16-byte aligned, apart from the inputs.
 * With pools (kv_dtype BS_BF16 or BS_FP32; k_scale and v_scale not read) the rotated K and
 * the V of a row go to slot position % 16 of the page that page_table names for position /
 * 16 in the row's sequence; no two rows may name one slot. k_out may then be NULL. With
 * pools NULL, k_out takes the keys, and v and page_table are not read (8-bit caches: follow
 * with bs_quant_append; drafts: nothing is written to the cache yet). Those calls take K and V of one row
 * stride: where V is columns of a wider row, copy it to rows like k_out's.
 * A row whose position is outside the range is skipped (BS_ERR_INVALID_ARG), and so is one
 * whose row_seq >= batch (BS_ERR_DEVICE_BOUNDS) or whose position lies past the page table's
 * row (BS_ERR_CAPACITY); a page outside the pool: that head's K and V are not written
 * (BS_ERR_DEVICE_BOUNDS). One launch. */
bs_status bs_rope_append(const bs_dims *dims, const bs_rope *rope, const void *q, const void *k, const void *v,
                         int64_t row_stride, int64_t n_rows, const int32_t *positions, const int32_t *row_seq,
                         const bs_pools *pools, const int32_t *page_table, void *q_out, void *k_out,
                         int32_t *dev_status, bs_stream_t stream);

/* Attention of new tokens over the cache that already holds them. Token p of sequence b,
 * tok_begin[b] <= p < seq_lens[b] (kv->seq_lens), is row row_begin[b] + p - tok_begin[b] of
 * q, out and lse. Over the tokens t of its unit that it sees:
 *   out_h = sum_t softmax_t(x_h(t)) V[t],  lse_h = log sum_t exp(x_h(t)),  x_h(t) = q_h . K[t] / sqrt(d);
 * it sees every t <= p (retrieval and dual units), or the t <= p with t < sink_tokens or
 * t > p - local_tokens (streaming units: token for token, where selections cover both by
 * whole blocks). A chunk may be a whole prompt, a piece of one behind a cached prefix, or
 * one token; tok_begin[b] = seq_lens[b] has none for b.
 * q_dtype BS_BF16; kv_dtype BS_BF16, BS_E4M3 or BS_INT8 (BS_ERR_INVALID_ARG otherwise).
 * q: n_rows rows of q_stride elements, 16-byte aligned, q_stride a multiple of 8 and at least
 * n_q_heads * head_dim. out bf16 [n_rows][n_q_heads][head_dim], 16-byte aligned; lse fp32
 * [n_rows][n_q_heads], or NULL. Of cfg: cls, sink_tokens and local_tokens.
 * Weights (with an 8-bit cache times the mantissa of V's scale) are rounded to bf16, off by at most
 * 2^-8 of themselves each, before they meet V, and out is divided by their sum as rounded; lse has the
 * sum before. Logits, maxima, sums and outputs are fp32 until out's own rounding (values of V up to
 * 2^90, whose weighted sums stay finite on the way). An infinity or a NaN of a key that a row
 * does not see does not reach it: where some rows of a block of tokens see such a value and
 * others do not, the others are computed again without it, one by one. A row is not finite in
 * a column in which it sees a V that is not (a page's scale counts), and in any if one of its
 * logits is NaN or +inf; a key with a logit of -inf weighs nothing.
 * max_new_tokens (host): an upper bound on seq_lens[b] - tok_begin[b]. It and n_rows size the
 * grid and choose the splits of long rows, and so the order of sums; a row's result does not
 * depend on what other sequences hold.
 * workspace: bs_prefill_workspace_size bytes, 16-byte aligned, overwritten by every call,
 * needs no clearing (NULL when the size is 0). Calls that share one must not run
 * concurrently.
 * A sequence whose lengths or rows do not fit is skipped: tok_begin < 0 or above seq_lens
 * (BS_ERR_INVALID_ARG); more tokens than max_new_tokens or more pages than a row
 * (BS_ERR_CAPACITY); rows outside [0, n_rows) (BS_ERR_DEVICE_BOUNDS). A unit with a bad head
 * configuration is skipped (BS_ERR_INVALID_ARG); a page outside the pool is left out
 * (BS_ERR_DEVICE_BOUNDS). Sequences may not share rows. One launch, two where rows are
 * split. */
bs_status bs_prefill_attn(const bs_dims *dims, const void *q, int64_t q_stride, int64_t n_rows, const bs_kv *kv,
                          const bs_head_cfg *cfg, const int32_t *tok_begin, const int32_t *row_begin,
                          int32_t max_new_tokens, void *out, float *lse, void *workspace, size_t workspace_bytes,
                          int32_t *dev_status, bs_stream_t stream);

/* Bytes of workspace bs_prefill_attn needs on the current device (0 on bad arguments, or when it
 * needs none). Not monotonic: only calls whose rows leave CTAs without work split them, so that a
 * long prompt may need none where a single token needs some. A loop that keeps one workspace sizes it
 * for every shape that it calls with, each with its own n_rows and max_new_tokens, and takes the
 * largest; no call needs more than 66 MiB and 16 bytes for each KV head of a block of rows. */
size_t bs_prefill_workspace_size(const bs_dims *dims, int64_t n_rows, int32_t max_new_tokens);

/* Largest tree of drafts of one sequence. */
#define BS_MAX_DRAFT 64

/* Drafted tokens (device pointers but for the sizes). Draft i of sequence b, i < n_draft[b],
 * is row row_begin[b] + i of k_new, v_new (n_rows rows of row_stride elements, bf16, KV head
 * h at [h * head_dim, (h + 1) * head_dim)) and of visible, whose bit j says that draft i
 * attends draft j of the same sequence (its ancestors and itself; bits from n_draft[b] on do
 * not count). */
typedef struct {
  const void *k_new, *v_new;    /* 16-byte aligned */
  int64_t row_stride, n_rows;   /* row_stride: a multiple of 8, >= n_kv_heads * head_dim */
  const int32_t *row_begin;     /* [batch] */
  const int32_t *n_draft;       /* [batch], 0 .. max_draft */
  const uint64_t *visible;      /* [n_rows] */
  int32_t max_draft;            /* host value: 1 .. BS_MAX_DRAFT */
} bs_drafts;

/* Attention of a tree of drafted tokens: bs_sparse_decode_attn for every draft at once. Draft
 * i of sequence b attends, with each query head h of a unit, the tokens t < T of the unit's
 * selected blocks (sel_idx, sel_cnt; T = kv->seq_lens[b], which does not count the drafts) and
 * the drafts j that visible names; out_h and lse_h as there, without block logits. A row that
 * sees nothing gets zeros and lse = -inf. q, out, lse, types, rounding and non-finite keys as
 * for bs_prefill_attn; rows are the drafts'. Of cfg: block_tokens. T may be 0 (no cache yet).
 * Selections are those of bs_select_topk (for the root's query, say): ascending, at most
 * max_sel_per_unit blocks and max_gather_pages_per_unit pages (BS_ERR_CAPACITY).
 * workspace: bs_tree_workspace_size bytes, under the rules of bs_prefill_attn's.
 * Where key tiles are split, the points depend on what the whole batch has selected and drafted, and so
 * does the order of a row's sums: other sequences change its last bits (the same batch gives the same
 * bits), unlike bs_prefill_attn's.
 * Skipped: a sequence with n_draft outside 0 .. max_draft or T < 0 (BS_ERR_INVALID_ARG), rows outside
 * [0, n_rows) (BS_ERR_DEVICE_BOUNDS) or more pages than a row (BS_ERR_CAPACITY); a unit whose
 * block_tokens is not a positive multiple of 16 (BS_ERR_INVALID_ARG). A block or page out of
 * range is left out (BS_ERR_DEVICE_BOUNDS). One launch, two where rows are split. */
bs_status bs_tree_decode_attn(const bs_dims *dims, const void *q, int64_t q_stride, const bs_kv *kv,
                              const bs_head_cfg *cfg, const int32_t *sel_idx, const int32_t *sel_cnt,
                              const bs_drafts *drafts, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream);

/* Bytes of workspace bs_tree_decode_attn needs (0 on bad arguments, or when it needs none). */
size_t bs_tree_workspace_size(const bs_dims *dims, int32_t max_draft);

/* Appends the accepted drafts. Token t of sequence b, tok_begin[b] <= t < seq_lens[b], is row
 * row_begin[b] + path[b][t - tok_begin[b]] of k_new and v_new (layout and types as for
 * bs_quant_append); it goes to slot t % 16 of the page that page_table names for t / 16: by
 * the rule of bs_quant_append into an 8-bit cache, rounded to kv_dtype into a BS_BF16 or
 * BS_FP32 one. path int32 [batch][path_stride], 1 <= path_stride <= BS_MAX_DRAFT; entries past
 * the accepted ones are not read. tok_begin, seq_lens as for bs_quant_append: seq_lens counts
 * the accepted tokens already, so that one path and one pair of lengths serve every layer.
 * Errors as for bs_quant_append; a sequence with more tokens than path_stride
 * (BS_ERR_CAPACITY) or a path entry whose row is outside [0, n_rows) (BS_ERR_DEVICE_BOUNDS) is
 * skipped. Sub-block means are not touched: call bs_build_block_summaries with the same lengths
 * before the next step, which renews the one of its own token only. One launch; bitwise
 * reproducible. */
bs_status bs_tree_commit(const bs_dims *dims, const bs_pools *pools, const int32_t *page_table,
                         const int32_t *seq_lens, const int32_t *tok_begin, const int32_t *row_begin,
                         const int32_t *path, int32_t path_stride, const void *k_new, const void *v_new,
                         int64_t row_stride, int64_t n_rows, int32_t *dev_status, bs_stream_t stream);

/* Bytes of workspace bs_sparse_decode_attn needs for these dims (0 on bad dims). */
size_t bs_workspace_size(const bs_dims *dims);

/* Kernels one bs_decode_step call launches for these dims (each a programmatic
 * dependent of the one before), or 0 on bad dims. Host only; launches nothing. */
int bs_decode_step_launches(const bs_dims *dims);

/* Every wait inside a kernel (for a bulk copy to land, for the fused step's selection
 * to be published) gives up after a wall-clock limit, reports BS_ERR_TIMEOUT in the
 * status word and lets the kernel finish. This sets that limit, in nanoseconds, for the
 * kernels launched from now on (those already captured in a CUDA graph keep the limit
 * they were captured with); 1000 ns .. 60 s, default one second. Returns
 * BS_ERR_INVALID_ARG (and keeps the old limit) outside that range. Process-wide; host
 * only. */
bs_status bs_set_wait_limit_ns(uint64_t limit_ns);

/* The current limit of device-side waits, in nanoseconds. */
uint64_t bs_wait_limit_ns(void);

/* Static text for a status code. */
const char *bs_status_string(bs_status status);

#ifdef __cplusplus
}
#endif

#endif /* BSATTN_H_ */
