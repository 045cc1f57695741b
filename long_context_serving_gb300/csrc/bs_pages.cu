// Pages of a cache handed out, shared, taken back and moved together, on the device.
//
// A page is free when its reference count is 0. Which free page a call takes is fixed (the
// k-th page asked for gets the k-th lowest free one), so everything rests on ranks:
//   * a scan kernel reads the counts once: each tile (at most kMaxTiles of them) lists its free
//     pages in ascending order and counts them (and, for compact, keeps their bitmap with each
//     word's rank); beside it, other CTAs of the same launch count what each unit asks for and
//     check the arguments;
//   * the next kernel (its CTAs in place by the time the scan ends) sums tiles
//     and requests before its own (block scans over at most kMaxTiles and `units` ints) and
//     gives each request its page: a binary search over the tiles' ranks in shared memory, then
//     one load from the tile's list. (Binary searches over bitmap words instead, about fifteen
//     dependent loads a request, and one entry a thread: 25.6 us for a batch turnover of 21 of
//     64 sequences of 8 heads, 148K table entries, against 12.3.)
// The lists are a snapshot, so counts may be written while others still look pages up, and no
// floating-point or order-dependent atomics are involved: integer counts only.
// Bound by latency (a launch and a few dependent loads, about 2 us a kernel on small pools, 3 to
// 5 on large ones) except for the copies, which are bound by HBM.
#include <algorithm>

#include "bs_attn_launch.cuh"
#include "bs_quant.cuh"

namespace bsi {
namespace {

constexpr int kPgThreads = 256;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kMaxTiles = 1024;
constexpr int kMinTilePages = 4096;
constexpr int kApplyCtas = 304;     // two CTAs per SM
constexpr int kMaxCtas = 8 * kApplyCtas;   // one wave; each takes a contiguous share beyond
constexpr int kBatch = 4;           // row entries a thread has in flight at once
constexpr int kFreeBatch = 8;       // the same in free

__host__ __device__ inline int64_t tile_pages_for(int64_t n_pages) {
  int64_t t = kMinTilePages;
  while ((n_pages + t - 1) / t > kMaxTiles) t <<= 1;
  return t;
}

// Workspace (int32 words): tile_free [kMaxTiles] | need [units] | err [units] | bitmap [words] |
// word rank [words] | list [n_pages].
struct PgWs {
  int32_t *tile_free;
  int32_t *need, *err;
  uint32_t *bits;
  int32_t *rank;        // free pages of the word's tile before the word
  int32_t *list;        // tile t's free pages, ascending, from list[t * tile_pages]
  int32_t n_tiles;
  int64_t n_words, tile_pages;
};
__host__ inline size_t pg_ws_ints(const bs_dims &d) {
  const size_t units = static_cast<size_t>(d.batch) * d.n_kv_heads;
  const size_t words = (static_cast<size_t>(d.n_pages) + 31) / 32;
  return kMaxTiles + 2 * units + 2 * words + static_cast<size_t>(d.n_pages);
}
__host__ inline PgWs pg_ws(const bs_dims &d, void *workspace) {
  const size_t units = static_cast<size_t>(d.batch) * d.n_kv_heads;
  PgWs w;
  w.tile_pages = tile_pages_for(d.n_pages);
  w.n_tiles = static_cast<int32_t>((d.n_pages + w.tile_pages - 1) / w.tile_pages);
  w.n_words = (d.n_pages + 31) / 32;
  w.tile_free = static_cast<int32_t *>(workspace);
  w.need = w.tile_free + kMaxTiles;
  w.err = w.need + units;
  w.bits = reinterpret_cast<uint32_t *>(w.err + units);
  w.rank = reinterpret_cast<int32_t *>(w.bits + w.n_words);
  w.list = w.rank + w.n_words;
  return w;
}

// Every kernel here is a programmatic dependent of the work before it: its CTAs are in place
// when that ends, wait for it before they read anything, and only then let the next one's in.
__device__ __forceinline__ void pdl_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Exclusive prefix sum of one int per thread over the CTA; *total gets the sum. All threads.
__device__ __forceinline__ int cta_scan(int v, int *tmp, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < kPgWarps; ++w) {
    const int t = tmp[w];
    if (w < warp) before += t;
    tot += t;
  }
  __syncthreads();
  *total = tot;
  return before + x - v;
}
__device__ __forceinline__ long long cta_sum(long long v, long long *tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  long long s = 0;
#pragma unroll
  for (int w = 0; w < kPgWarps; ++w) s += tmp[w];
  __syncthreads();
  return s;
}
__device__ __forceinline__ int cta_max(int v, int *tmp) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  int m = 0;
#pragma unroll
  for (int w = 0; w < kPgWarps; ++w) m = max(m, tmp[w]);
  __syncthreads();
  return m;
}

// ---------------------------------------------------------------------------
// Tile t of the counts: the list of its free pages, their number and, with `words`, the
// bitmap's words and ranks.
// ---------------------------------------------------------------------------
__device__ void scan_tile(const bs_dims &dims, const int32_t *ref, const PgWs &ws, int t, bool words) {
  __shared__ int tmp[kPgWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ uint32_t wsm[kMinTilePages / 32];
  __shared__ int rsm[kMinTilePages / 32];
  const int64_t p0 = static_cast<int64_t>(t) * ws.tile_pages;
  const int64_t p1 = min(p0 + ws.tile_pages, dims.n_pages);
  int run = 0;
  for (int64_t q = p0; q < p1; q += kMinTilePages) {
    constexpr int kPer = kMinTilePages / 32 / kPgWarps;   // words a warp
    int v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t p = q + (warp * kPer + i) * 32 + lane;
      v[i] = p < p1 ? ref[p] : 1;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t w = __ballot_sync(0xffffffffu, v[i] == 0);
      if (lane == 0) wsm[warp * kPer + i] = w;
    }
    __syncthreads();
    const int n_words = static_cast<int>((min(p1 - q, static_cast<int64_t>(kMinTilePages)) + 31) / 32);
    const uint32_t mine = tid < n_words ? wsm[tid] : 0u;
    int total;
    const int before = cta_scan(__popc(mine), tmp, &total);
    if (tid < n_words) {
      rsm[tid] = run + before;
      if (words) {
        ws.bits[q / 32 + tid] = mine;
        ws.rank[q / 32 + tid] = run + before;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int w = warp * kPer + i;
      if (v[i] == 0) {   // (0 only for a page of the pool)
        const uint32_t below = wsm[w] & ((1u << lane) - 1u);
        ws.list[p0 + rsm[w] + __popc(below)] = static_cast<int32_t>(q + w * 32 + lane);
      }
    }
    run += total;
    __syncthreads();
  }
  if (tid == 0) ws.tile_free[t] = run;
}
static_assert(kMinTilePages / 32 <= kPgThreads, "one word a thread");

// Free pages below page p (0 <= p < n_pages).
__device__ __forceinline__ int free_rank(const PgWs &ws, const int *before, int64_t p) {
  const int64_t w = p >> 5;
  return before[p / ws.tile_pages] + ws.rank[w] + __popc(ws.bits[w] & ((1u << (p & 31)) - 1u));
}
// The k-th lowest free page (k below the number of free pages).
__device__ __forceinline__ int kth_free(const PgWs &ws, const int *before, int k) {
  int lo = 0, hi = ws.n_tiles - 1;
  while (lo < hi) {                       // the last tile that starts at rank <= k
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return ws.list[lo * ws.tile_pages + (k - before[lo])];
}

// What the scan found: free pages before each tile, [n_tiles + 1], into shared memory; what
// the requesters before `first` ask for, what all n ask for, and the worst error of any (0:
// none). All threads.
struct Requests {
  long long before, total;
  int err;
};
__device__ __forceinline__ Requests load_plan(const PgWs &ws, int n, int first, int *before) {
  __shared__ int w_free[kPgWarps], w_err[kPgWarps];
  __shared__ long long w_pre[kPgWarps], w_all[kPgWarps];
  constexpr int kPer = kMaxTiles / kPgThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = threadIdx.x * kPer + i;
    v[i] = t < ws.n_tiles ? ws.tile_free[t] : 0;
    sum += v[i];
  }
  long long pre = 0, all = 0;
  int err = 0;
  for (int i = threadIdx.x; i < n; i += kPgThreads) {
    const int k = ws.need[i];
    err = max(err, ws.err[i]);
    all += k;
    if (i < first) pre += k;
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  err = __reduce_max_sync(0xffffffffu, err);
  if (lane == 31) {
    w_free[warp] = x;
    w_pre[warp] = pre;
    w_all[warp] = all;
    w_err[warp] = err;
  }
  __syncthreads();
  Requests r = {0, 0, 0};
  int run = x - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kPgWarps; ++w) {
    if (w < warp) run += w_free[w];
    total += w_free[w];
    r.before += w_pre[w];
    r.total += w_all[w];
    r.err = max(r.err, w_err[w]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = threadIdx.x * kPer + i;
    if (t < ws.n_tiles) before[t] = run;
    run += v[i];
  }
  if (threadIdx.x == 0) before[ws.n_tiles] = total;
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------------------
// reserve: a CTA per unit. A thread takes four neighbouring entries, so that one scan ranks
// 1024 of them. With the free before it 12.3 us for 21 of 64 sequences of 8 heads, 148K entries
// in a pool of 383K pages (17.8 with the entries loaded after the scan's end), 6.0 us for one
// short sequence.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPgThreads) reserve_scan(bs_dims dims, bs_page_map map, const int32_t *new_lens, PgWs ws) {
  pdl_enter();
  if (static_cast<int>(blockIdx.x) < ws.n_tiles) {
    scan_tile(dims, map.ref_count, ws, blockIdx.x, false);
    return;
  }
  __shared__ long long tmp[kPgWarps];
  const int units = dims.batch * dims.n_kv_heads;
  for (int u = blockIdx.x - ws.n_tiles; u < units; u += gridDim.x - ws.n_tiles) {
    const int64_t len = max(new_lens[u / dims.n_kv_heads], 0);
    const int64_t np = (len + kPage - 1) / kPage;
    const int32_t *row = map.page_table + static_cast<size_t>(u) * dims.max_pages_per_unit;
    const int n = static_cast<int>(min(np, static_cast<int64_t>(dims.max_pages_per_unit)));
    int lacks = 0;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kPgThreads) lacks += row[i] < 0 ? 1 : 0;
    const long long sum = cta_sum(lacks, tmp);
    if (threadIdx.x == 0) {
      ws.need[u] = static_cast<int>(sum);
      ws.err[u] = np > dims.max_pages_per_unit ? BS_ERR_CAPACITY : BS_OK;
    }
  }
}

__global__ void __launch_bounds__(kPgThreads) reserve_apply(bs_dims dims, bs_page_map map, const int32_t *new_lens, PgWs ws,
                                                            int32_t *st) {
  __shared__ int before[kMaxTiles + 1];
  __shared__ int tmp[kPgWarps];
  const int units = dims.batch * dims.n_kv_heads;
  // A contiguous share of the units per CTA. The scan changes neither lengths nor rows, and was
  // let in after everything before it had finished: the first entries are loaded beside it.
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  const int MP = dims.max_pages_per_unit;
  auto unit_pages_wanted = [&](int u) {
    return (static_cast<int64_t>(max(__ldcg(new_lens + u / dims.n_kv_heads), 0)) + kPage - 1) / kPage;
  };
  int entry[kBatch];
  {
    const int64_t n0 = min(unit_pages_wanted(u0), static_cast<int64_t>(MP));
    const int32_t *row = map.page_table + static_cast<size_t>(u0) * MP;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int j = static_cast<int>(threadIdx.x) * kBatch + e;
      entry[e] = j < n0 ? __ldcg(row + j) : 0;
    }
  }
  pdl_enter();
  const Requests rq = load_plan(ws, units, u0, before);
  if (rq.err != BS_OK || rq.total > before[ws.n_tiles]) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(st, rq.err != BS_OK ? rq.err : BS_ERR_CAPACITY);
    return;
  }
  int k = static_cast<int>(rq.before);
  for (int u = u0; u < u1; ++u) {
    if (ws.need[u] == 0) continue;
    const int n = static_cast<int>(unit_pages_wanted(u));   // (within the row: else an error above)
    int32_t *row = map.page_table + static_cast<size_t>(u) * MP;
    for (int i0 = 0; i0 < n; i0 += kPgThreads * kBatch) {
      const int first = i0 + threadIdx.x * kBatch;   // a thread's entries are neighbours: ranks ascend
      bool lacks[kBatch];
      int mine = 0;
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (u > u0 || i0 > 0) entry[e] = first + e < n ? row[first + e] : 0;
        lacks[e] = first + e < n && entry[e] < 0;
        mine += lacks[e] ? 1 : 0;
      }
      int total;
      int r = k + cta_scan(mine, tmp, &total);
      int page[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (lacks[e]) page[e] = kth_free(ws, before, r++);
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (lacks[e]) {
          row[first + e] = page[e];
          map.ref_count[page[e]] = 1;
        }
      k += total;
    }
  }
}

// ---------------------------------------------------------------------------
// fork: item (i, h) = fork i, KV head h. The scan reads what apply will write (dst's row) and
// share (src's entries and their counts), so that apply need not check. With the free before
// and the copy after it 12.0 us for 16 beams of 8 heads over 8K tokens, 8.2 us for three short
// ones.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPgThreads) fork_scan(bs_dims dims, bs_page_map map, const int32_t *src, const int32_t *dst,
                                                        int n, PgWs ws) {
  pdl_enter();
  if (static_cast<int>(blockIdx.x) < ws.n_tiles) {
    scan_tile(dims, map.ref_count, ws, blockIdx.x, false);
    return;
  }
  __shared__ int tmp[kPgWarps];
  const int MP = dims.max_pages_per_unit;
  for (int it = blockIdx.x - ws.n_tiles; it < n * dims.n_kv_heads; it += gridDim.x - ws.n_tiles) {
    const int i = it / dims.n_kv_heads, h = it % dims.n_kv_heads;
    const int s = src[i], d = dst[i];
    int need = 0, err = 0;
    if (s >= 0 && d >= 0) {
      if (s >= dims.batch || d >= dims.batch || s == d) {
        err = BS_ERR_INVALID_ARG;
      } else {
        for (int j = threadIdx.x; j < n; j += kPgThreads) {
          const int sj = src[j], dj = dst[j];
          if (sj < 0 || dj < 0) continue;
          if ((j != i && dj == d) || sj == d) err = BS_ERR_INVALID_ARG;
        }
        const int32_t *from = map.page_table + (static_cast<size_t>(s) * dims.n_kv_heads + h) * MP;
        const int32_t *to = map.page_table + (static_cast<size_t>(d) * dims.n_kv_heads + h) * MP;
#pragma unroll 4
        for (int j = threadIdx.x; j < MP; j += kPgThreads)
          if (to[j] >= 0) err = BS_ERR_INVALID_ARG;
        const int T = map.seq_lens[s];
        const int64_t np = (static_cast<int64_t>(T) + kPage - 1) / kPage;
        if (T < 0) {
          err = BS_ERR_INVALID_ARG;
        } else if (np > MP) {
          err = max(err, static_cast<int>(BS_ERR_CAPACITY));
        } else {
          for (int j0 = threadIdx.x; j0 < np; j0 += kPgThreads * kBatch) {
            int p[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) p[e] = j0 + e * kPgThreads < np ? from[j0 + e * kPgThreads] : -1;
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              if (p[e] < -1 || (p[e] >= 0 && (p[e] >= dims.n_pages || map.ref_count[p[e]] <= 0)))
                err = max(err, static_cast<int>(BS_ERR_DEVICE_BOUNDS));
          }
          if (T % kPage != 0 && from[T / kPage] >= 0) need = 1;
        }
      }
    }
    err = cta_max(err, tmp);
    if (threadIdx.x == 0) {
      ws.need[it] = need;
      ws.err[it] = err;
    }
  }
}

__global__ void __launch_bounds__(kPgThreads) fork_apply(bs_dims dims, bs_page_map map, const int32_t *src, const int32_t *dst,
                                                         int n, bs_page_copies copies, PgWs ws, int32_t *st) {
  __shared__ int before[kMaxTiles + 1];
  const int items = n * dims.n_kv_heads, MP = dims.max_pages_per_unit;
  const int i0 = static_cast<int>(static_cast<int64_t>(items) * blockIdx.x / gridDim.x);
  const int i1 = static_cast<int>(static_cast<int64_t>(items) * (blockIdx.x + 1) / gridDim.x);
  // As in reserve_apply: the first item's entries are loaded beside the scan (which has not
  // checked them yet, so nothing is taken for granted).
  int entry[kBatch];
  {
    const int s0 = __ldcg(src + i0 / dims.n_kv_heads);
    const bool in = s0 >= 0 && s0 < dims.batch;
    const int full0 = in ? min(max(__ldcg(map.seq_lens + s0), 0) / kPage, MP) : 0;
    const int32_t *from = map.page_table + (static_cast<size_t>(in ? s0 : 0) * dims.n_kv_heads + i0 % dims.n_kv_heads) * MP;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int j = static_cast<int>(threadIdx.x) + e * kPgThreads;
      entry[e] = j < full0 ? __ldcg(from + j) : -1;
    }
  }
  pdl_enter();
  const Requests rq = load_plan(ws, items, i0, before);
  const bool bad = rq.err != BS_OK || rq.total > before[ws.n_tiles];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *copies.count = bad ? 0 : static_cast<int>(rq.total);
    if (bad) report(st, rq.err != BS_OK ? rq.err : BS_ERR_CAPACITY);
  }
  if (bad) return;
  int k = static_cast<int>(rq.before);
  for (int it = i0; it < i1; ++it) {
    const int i = it / dims.n_kv_heads, h = it % dims.n_kv_heads;
    const int s = src[i], d = dst[i];
    if (s < 0 || d < 0) continue;
    const int T = map.seq_lens[s], full = T / kPage;
    const int32_t *from = map.page_table + (static_cast<size_t>(s) * dims.n_kv_heads + h) * MP;
    int32_t *to = map.page_table + (static_cast<size_t>(d) * dims.n_kv_heads + h) * MP;
    for (int j0 = threadIdx.x; j0 < full; j0 += kPgThreads * kBatch) {
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (it > i0 || j0 >= kPgThreads * kBatch) entry[e] = j0 + e * kPgThreads < full ? from[j0 + e * kPgThreads] : -1;
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = j0 + e * kPgThreads, p = entry[e];
        if (j >= full) continue;
        to[j] = p < 0 ? -1 : p;
        if (p >= 0) atomicAdd(map.ref_count + p, 1);
      }
    }
    if (threadIdx.x == 0) {
      if (ws.need[it]) {
        const int p = kth_free(ws, before, k);
        to[full] = p;
        map.ref_count[p] = 1;
        copies.pairs[2 * k] = from[full];
        copies.pairs[2 * k + 1] = p;
      }
      if (h == 0) map.seq_lens[d] = T;
    }
    k += ws.need[it];
  }
}

// ---------------------------------------------------------------------------
// free: CTA (i, h). Eight entries a thread in flight: rows of 2048 pages in one round of loads
// and one of counts.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPgThreads) free_kernel(bs_dims dims, bs_page_map map, const int32_t *seqs, int n, int32_t *st) {
  __shared__ int tmp[kPgWarps];
  pdl_enter();
  for (int it = blockIdx.x; it < n * dims.n_kv_heads; it += gridDim.x) {
    const int i = it / dims.n_kv_heads, h = it % dims.n_kv_heads;
    const int s = seqs[i];
    if (s < 0) continue;
    if (s >= dims.batch) {
      if (h == 0 && threadIdx.x == 0) report(st, BS_ERR_INVALID_ARG);
      continue;
    }
    int again = 0;   // named before: done there
    for (int j = threadIdx.x; j < i; j += kPgThreads) again |= seqs[j] == s ? 1 : 0;
    const int MP = dims.max_pages_per_unit;
    int32_t *row = map.page_table + (static_cast<size_t>(s) * dims.n_kv_heads + h) * MP;
    int p[kFreeBatch];   // (the first entries are loaded beside the check)
#pragma unroll
    for (int e = 0; e < kFreeBatch; ++e) {
      const int j = threadIdx.x + e * kPgThreads;
      p[e] = j < MP ? row[j] : -1;
    }
    if (cta_max(again, tmp)) continue;
    for (int j0 = threadIdx.x; j0 < MP; j0 += kPgThreads * kFreeBatch) {
      int had[kFreeBatch];
      if (j0 >= kPgThreads * kFreeBatch) {
#pragma unroll
        for (int e = 0; e < kFreeBatch; ++e) p[e] = j0 + e * kPgThreads < MP ? row[j0 + e * kPgThreads] : -1;
      }
#pragma unroll
      for (int e = 0; e < kFreeBatch; ++e) {
        had[e] = 1;
        if (p[e] != -1) row[j0 + e * kPgThreads] = -1;
        if (p[e] >= 0) had[e] = p[e] < dims.n_pages ? atomicSub(map.ref_count + p[e], 1) : -1;
      }
#pragma unroll
      for (int e = 0; e < kFreeBatch; ++e)
        if (had[e] <= 0 || p[e] < -1) {
          if (p[e] >= 0 && p[e] < dims.n_pages) atomicAdd(map.ref_count + p[e], 1);
          report(st, BS_ERR_DEVICE_BOUNDS);
        }
    }
    if (h == 0 && threadIdx.x == 0) map.seq_lens[s] = 0;
  }
}

// ---------------------------------------------------------------------------
// compact: pages and table entries look their ranks up in the same launch (a remap table in
// between cost a third one: 9.5 us a small cache with its copy, against 7.7).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPgThreads) compact_scan(bs_dims dims, bs_page_map map, PgWs ws) {
  pdl_enter();
  scan_tile(dims, map.ref_count, ws, blockIdx.x, true);
}

// The first `move_ctas` CTAs: one thread per page, a page in use at or above N moves. The
// others: one thread per table entry, which finds where its page goes from the same ranks.
__global__ void __launch_bounds__(kPgThreads) compact_apply(bs_dims dims, bs_page_map map, bs_page_copies copies, int32_t *n_live,
                                                            PgWs ws, int move_ctas, int32_t *st) {
  __shared__ int before[kMaxTiles + 1];
  pdl_enter();
  load_plan(ws, 0, 0, before);
  const int n_pages = static_cast<int>(dims.n_pages);
  const int N = n_pages - before[ws.n_tiles];
  // Pages in use below N: N - (free pages below N); the others move.
  const int moves = N < n_pages ? free_rank(ws, before, N) : 0;
  const bool fits = moves <= copies.capacity;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *n_live = N;
    *copies.count = fits ? moves : 0;
    if (!fits) report(st, BS_ERR_CAPACITY);
  }
  if (!fits) return;
  const int live_below_n = N - moves;
  auto is_free = [&](int64_t p) { return (ws.bits[p >> 5] >> (p & 31) & 1u) != 0; };
  auto move_of = [&](int64_t p) { return static_cast<int>(p) - free_rank(ws, before, p) - live_below_n; };
  if (static_cast<int>(blockIdx.x) < move_ctas) {
    for (int64_t p = N + static_cast<int64_t>(blockIdx.x) * kPgThreads + threadIdx.x; p < n_pages;
         p += static_cast<int64_t>(move_ctas) * kPgThreads) {
      if (is_free(p)) continue;
      const int k = move_of(p), to = kth_free(ws, before, k);
      copies.pairs[2 * k] = static_cast<int>(p);
      copies.pairs[2 * k + 1] = to;
      map.ref_count[to] = map.ref_count[p];
      map.ref_count[p] = 0;
    }
    return;
  }
  const int64_t total = static_cast<int64_t>(dims.batch) * dims.n_kv_heads * dims.max_pages_per_unit;
  for (int64_t i = static_cast<int64_t>(blockIdx.x - move_ctas) * kPgThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x - move_ctas) * kPgThreads) {
    const int p = map.page_table[i];
    if (p >= -1 && p < N) continue;
    if (p < 0 || p >= n_pages || is_free(p)) {
      report(st, BS_ERR_DEVICE_BOUNDS);
      continue;
    }
    map.page_table[i] = kth_free(ws, before, move_of(p));
  }
}

// ---------------------------------------------------------------------------
// copy: a CTA per pair, K and V in flight together; 23K pages of 2 + 2 KB: 30.5 us, 6.1 TB/s.
// ---------------------------------------------------------------------------
constexpr int kCopyPageThreads = 128;

__global__ void __launch_bounds__(kCopyPageThreads) copy_kernel(bs_dims dims, bs_pools pools, bs_page_copies copies, int page_bytes,
                                                                bool scales, int32_t *st) {
  pdl_enter();
  const int n = min(max(*copies.count, 0), copies.capacity);
  const int vecs = page_bytes / 16;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int2 pr = reinterpret_cast<const int2 *>(copies.pairs)[i];
    if (pr.x < 0 || pr.y < 0 || pr.x >= dims.n_pages || pr.y >= dims.n_pages) {
      if (threadIdx.x == 0) report(st, BS_ERR_DEVICE_BOUNDS);
      continue;
    }
    const uint4 *ks = reinterpret_cast<const uint4 *>(static_cast<const char *>(pools.k_pool) + static_cast<size_t>(pr.x) * page_bytes);
    const uint4 *vs = reinterpret_cast<const uint4 *>(static_cast<const char *>(pools.v_pool) + static_cast<size_t>(pr.x) * page_bytes);
    uint4 *kd = reinterpret_cast<uint4 *>(static_cast<char *>(pools.k_pool) + static_cast<size_t>(pr.y) * page_bytes);
    uint4 *vd = reinterpret_cast<uint4 *>(static_cast<char *>(pools.v_pool) + static_cast<size_t>(pr.y) * page_bytes);
    for (int j = threadIdx.x; j < vecs; j += kCopyPageThreads) {
      const uint4 a = ks[j], b = vs[j];
      kd[j] = a;
      vd[j] = b;
    }
    if (scales && threadIdx.x == 0) {
      pools.k_scale[pr.y] = pools.k_scale[pr.x];
      pools.v_scale[pr.y] = pools.v_scale[pr.x];
    }
  }
}

template <int NT = kPgThreads, typename K, typename... Args>
bs_status launch_pg(K kernel, int ctas, cudaStream_t cs, Args... args) {
  return launch_ex(kernel, dim3(ctas), NT, 0, cs, 0, true, args...) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

bs_status check_map(const bs_dims *dims, const bs_page_map *map, const int32_t *dev_status) {
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (!map || !map->page_table || !map->ref_count || !map->seq_lens || !dev_status) return BS_ERR_INVALID_ARG;
  return BS_OK;
}
bs_status check_copies(const bs_page_copies *c) {
  if (!c || !c->pairs || !c->count || c->capacity < 1) return BS_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(c->pairs) & 7u) ? BS_ERR_ALIGN : BS_OK;
}
bs_status check_ws(const bs_dims &d, const void *ws, size_t bytes) {
  if (!ws) return BS_ERR_INVALID_ARG;
  if (!aligned16(ws)) return BS_ERR_ALIGN;
  return bytes < bs_pages_workspace_size(&d) ? BS_ERR_CAPACITY : BS_OK;
}

}  // namespace
}  // namespace bsi

extern "C" {

size_t bs_pages_workspace_size(const bs_dims *dims) {
  if (bsi::check_dims(dims) != BS_OK) return 0;
  return (bsi::pg_ws_ints(*dims) * 4 + 15) / 16 * 16;
}

bs_status bs_pages_reserve(const bs_dims *dims, const bs_page_map *map, const int32_t *new_lens, void *workspace,
                           size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_map(dims, map, dev_status);
  if (s != BS_OK) return s;
  if (!new_lens) return BS_ERR_INVALID_ARG;
  s = check_ws(*dims, workspace, workspace_bytes);
  if (s != BS_OK) return s;
  const PgWs ws = pg_ws(*dims, workspace);
  const int units = dims->batch * dims->n_kv_heads;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = launch_pg(reserve_scan, ws.n_tiles + std::min(units, kMaxCtas), cs, *dims, *map, new_lens, ws);
  if (s != BS_OK) return s;
  return launch_pg(reserve_apply, std::min(units, kMaxCtas), cs, *dims, *map, new_lens, ws, dev_status);
}

bs_status bs_pages_fork(const bs_dims *dims, const bs_page_map *map, const int32_t *src, const int32_t *dst, int32_t n,
                        const bs_page_copies *copies, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_map(dims, map, dev_status);
  if (s != BS_OK) return s;
  if (!src || !dst || n < 1 || n > dims->batch) return BS_ERR_INVALID_ARG;
  s = check_copies(copies);
  if (s != BS_OK) return s;
  const int items = n * dims->n_kv_heads;
  if (copies->capacity < items) return BS_ERR_CAPACITY;
  s = check_ws(*dims, workspace, workspace_bytes);
  if (s != BS_OK) return s;
  const PgWs ws = pg_ws(*dims, workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = launch_pg(fork_scan, ws.n_tiles + std::min(items, kMaxCtas), cs, *dims, *map, src, dst, n, ws);
  if (s != BS_OK) return s;
  return launch_pg(fork_apply, std::min(items, kMaxCtas), cs, *dims, *map, src, dst, n, *copies, ws, dev_status);
}

bs_status bs_pages_free(const bs_dims *dims, const bs_page_map *map, const int32_t *seqs, int32_t n,
                        int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_map(dims, map, dev_status);
  if (s != BS_OK) return s;
  if (!seqs || n < 1 || n > dims->batch) return BS_ERR_INVALID_ARG;
  return launch_pg(free_kernel, std::min(n * dims->n_kv_heads, kMaxCtas), reinterpret_cast<cudaStream_t>(stream), *dims, *map,
                   seqs, n, dev_status);
}

bs_status bs_pages_compact(const bs_dims *dims, const bs_page_map *map, const bs_page_copies *copies, int32_t *n_live,
                           void *workspace, size_t workspace_bytes, int32_t *dev_status, bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_map(dims, map, dev_status);
  if (s != BS_OK) return s;
  if (!n_live) return BS_ERR_INVALID_ARG;
  s = check_copies(copies);
  if (s != BS_OK) return s;
  s = check_ws(*dims, workspace, workspace_bytes);
  if (s != BS_OK) return s;
  const PgWs ws = pg_ws(*dims, workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = launch_pg(compact_scan, ws.n_tiles, cs, *dims, *map, ws);
  if (s != BS_OK) return s;
  const int64_t entries = static_cast<int64_t>(dims->batch) * dims->n_kv_heads * dims->max_pages_per_unit;
  const int move_ctas = static_cast<int>(std::min<int64_t>((dims->n_pages + kPgThreads - 1) / kPgThreads, 2 * kApplyCtas));
  const int table_ctas = static_cast<int>(std::min<int64_t>((entries + kPgThreads - 1) / kPgThreads, 2 * kApplyCtas));
  return launch_pg(compact_apply, move_ctas + table_ctas, cs, *dims, *map, *copies, n_live, ws, move_ctas, dev_status);
}

bs_status bs_pages_copy(const bs_dims *dims, const bs_pools *pools, const bs_page_copies *copies, int32_t *dev_status,
                        bs_stream_t stream) {
  using namespace bsi;
  bs_status s = check_dims(dims);
  if (s != BS_OK) return s;
  if (!pools || !pools->k_pool || !pools->v_pool || !dev_status) return BS_ERR_INVALID_ARG;
  const bool quant = is_quant(dims->kv_dtype);
  if (quant && (!pools->k_scale || !pools->v_scale)) return BS_ERR_INVALID_ARG;
  s = check_copies(copies);
  if (s != BS_OK) return s;
  if (!aligned16(pools->k_pool) || !aligned16(pools->v_pool)) return BS_ERR_ALIGN;
  const int esz = quant ? 1 : dims->kv_dtype == BS_BF16 ? 2 : 4;
  return launch_pg<kCopyPageThreads>(copy_kernel, std::min(copies->capacity, 16 * kApplyCtas),
                                     reinterpret_cast<cudaStream_t>(stream), *dims, *pools, *copies, kPage * dims->head_dim * esz,
                                     quant, dev_status);
}

}  // extern "C"
