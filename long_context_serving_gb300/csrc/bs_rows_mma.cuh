// Rows of new tokens against tiles of 128 keys on the fifth-generation tensor cores.
//
// One CTA takes one KV head's rows of a block of tokens (all query heads of the group: a K or V
// tile is fetched once for all of them), packed as 128-row tiles of whole tokens, kTiles of them
// (1 or 2), against a contiguous piece of the block's key groups:
//   copy warps     fetch K and V tiles, 128 keys each, into a ring of shared-memory slots: bf16
//                  pages by tiled copies (a warp for K, one for V); 8-bit pages as codes by plain
//                  loads, written as the bf16 values they stand for (four warps);
//   product warp   S = Q K^T into tensor memory (one thread issues); O += P V with P from tensor
//                  memory, page by page, so that a page that is not there takes no part;
//   row warps      four a tile, a thread a row: logits from tensor memory, the running maximum and
//                  sum in registers, weights back to tensor memory as bf16, over the logits.
// S of the next key tile is issued behind O's update, so with two tiles one's products run beside
// the other's softmax; weights are handed over 64 keys at a time, so that O's update starts while
// the second half's are made. O is brought to a new maximum only when that has grown by more than 2^8
// (weights of at most 256 in between; the final division takes it back), at the start of a
// tile, when the products in flight are done: O's rescaling through registers is rare and needs no
// warps of its own. What the second half's maximum adds waits for the next tile (a weight too large
// for its type meanwhile makes the row one of those that are computed again).
// Precision: products of bf16 in fp32; weights enter as bf16 (2^-9 of themselves), which is the
// operand type of V; their sum is taken before that rounding. Page scales: K's multiplies logits
// in fp32; V's is m * 2^e, 2^e goes into the bf16 values (exact), m into the weights, so that
// neither a tiny nor a large scale leaves the type's range on its own.
// A key that no row may see has no place in a product: 0 times an infinity is a NaN. Slots past
// the cache's end are zeroed, pages that are not there are left out, and a row whose sums are not
// finite is computed again by row_attend.
#pragma once

#include "bs_attn_launch.cuh"
#include "bs_rows_attn.cuh"
#include "bs_umma.cuh"

namespace bsi {

constexpr int kKeyTile = 128;                 // keys of a tile
constexpr int kTileGroups = kKeyTile / kPage; // groups of a tile
constexpr int kInfos = 8;                     // tiles whose description is kept

struct RowsPlan {
  int tokens;         // tokens of a row tile: 128 / G
  int block_tokens;   // of a CTA
  int n_blocks;       // prefill: blocks of all sequences, at most; tree: of a sequence
  int splits;         // CTAs a block's keys are split over, at most
  int record_rows;    // rows of a block, at most
  float *rec_o;       // [item][split][record_rows][D], when splits > 1
  float2 *rec_ml;     // [item][split][record_rows]: maximum (log2 units), sum
  uint64_t wait_ns;
};

struct RowsMaps {
  CUtensorMap q, k, v, k_new, v_new;
};

// What a CTA works on.
struct RowsItem {
  SeqRows r;
  Keys k;
  int b, h, i0, i1;       // tokens [i0, i1) of the sequence
  int64_t index;          // item (for the records)
  int t_lo, t_hi;         // key tiles of this split; empty: nothing to do
  int n_splits;           // splits that have work
};

// Key tiles of split s of an item.
__device__ __forceinline__ void split_tiles(const RowsPlan &p, int n_groups, int s, RowsItem &it) {
  const int n = (n_groups + kTileGroups - 1) / kTileGroups;
  const int per = max(1, (n + p.splits - 1) / p.splits);
  it.n_splits = (n + per - 1) / per;
  it.t_lo = min(s * per, n);
  it.t_hi = min(it.t_lo + per, n);
}

// Item of a CTA index, by a whole warp (every lane gets it). Errors are reported once.
template <bool kTree>
__device__ __forceinline__ void find_item(const RowsArgs &a, const RowsPlan &p, int64_t index, int split, RowsItem &it) {
  const int lane = threadIdx.x & 31;
  it.index = index;
  it.t_lo = it.t_hi = it.n_splits = 0;
  it.i0 = it.i1 = 0;
  int block;
  if constexpr (kTree) {
    const int64_t u = index / p.n_blocks;
    block = static_cast<int>(index - u * p.n_blocks);
    it.b = static_cast<int>(u / a.dims.n_kv_heads);
    it.h = static_cast<int>(u % a.dims.n_kv_heads);
    const int bad = seq_rows<kTree>(a, it.b, it.r);
    if (bad != 0 && lane == 0 && block == 0 && split == 0 && it.h == 0) report(a.st, bad);
    if (it.r.n <= block * p.block_tokens) return;
  } else {
    it.h = static_cast<int>(index % a.dims.n_kv_heads);
    int at = static_cast<int>(index / a.dims.n_kv_heads);   // blocks before this one
    const bool first = index == 0 && split == 0;            // looks at every sequence, and reports
    it.b = -1;
    block = 0;
    int total = 0;
    for (int b0 = 0; b0 < a.dims.batch && (it.b < 0 || first); b0 += 32) {
      SeqRows r;
      r.n = 0;
      r.p0 = r.T = 0;
      r.row0 = 0;
      const int b = b0 + lane;
      const int bad = b < a.dims.batch ? seq_rows<kTree>(a, b, r) : 0;
      if (bad != 0 && first) report(a.st, bad);
      const int mine = (r.n + p.block_tokens - 1) / p.block_tokens;
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const unsigned here = __ballot_sync(0xffffffffu, sum > at);
      if (it.b < 0 && here != 0) {
        const int src = __ffs(here) - 1;
        it.b = b0 + src;
        // (a sequence's last block first: it has the most keys)
        block = __shfl_sync(0xffffffffu, sum, src) - 1 - at;
        it.r.n = __shfl_sync(0xffffffffu, r.n, src);
        it.r.p0 = __shfl_sync(0xffffffffu, r.p0, src);
        it.r.T = __shfl_sync(0xffffffffu, r.T, src);
        it.r.row0 = __shfl_sync(0xffffffffu, r.row0, src);
      }
      const int all = __shfl_sync(0xffffffffu, sum, 31);
      at -= all;
      total += all;
    }
    if (first && lane == 0 && total > p.n_blocks) report(a.st, BS_ERR_CAPACITY);   // sequences that share rows
    if (it.b < 0) return;
  }
  it.i0 = block * p.block_tokens;
  it.i1 = min(it.i0 + p.block_tokens, it.r.n);
  const int bad = unit_keys<kTree>(a, it.r, it.b * a.dims.n_kv_heads + it.h, it.i0, it.i1, it.k);
  if (bad != 0) {
    if (lane == 0 && split == 0) report(a.st, bad);
    return;
  }
  split_tiles(p, it.k.n_groups, split, it);
}

// Description of a key tile, written by the copy warps.
struct TileInfo {
  int base[kTileGroups];      // first key of each group
  uint32_t flags;             // bits 0..7: rows differ in what they see of the group, or its end is
                              // past the cache's; 8..15: it is not there; 16..23: it is of drafts
  float ks[kTileGroups], vs[kTileGroups];   // 8-bit caches: K's scale, mantissa of V's
};

struct RowsShared {
  RowsItem item;
  TileInfo info[kInfos];
  uint64_t full[12], empty[12];
  uint64_t q_full, s_full[2], p_full[2][2], o_full[2], drained;   // (p_full: [row tile][half of the keys])
  uint32_t tmem;
};

template <int D, int kKv, int kTiles>
struct RowsTraits {
  static constexpr bool kQuant = kKv != 0;              // 1: E4M3, 2: INT8
  static constexpr int kHalves = D / 64;                // 128-byte columns of a row
  static constexpr int kSlotBytes = kKeyTile * D * 2;
  static constexpr int kHalfBytes = kKeyTile * 128;
  static constexpr int kQBytes = kTiles * 128 * D * 2;
  static constexpr int kControl = 2048;                 // RowsShared
  static constexpr int kMaxDyn = 232448;                // shared memory of a CTA, at most
  static constexpr int kRoom = (kMaxDyn - 1024 - kControl - kQBytes) / kSlotBytes;
  static constexpr int kSlots = kRoom < 12 ? kRoom : 12;
  static constexpr int kRowWarps = 4 * kTiles;
  static constexpr int kCopyWarps = kQuant ? 4 : 2;
  static constexpr int kThreads = 32 * (kRowWarps + 1 + kCopyWarps);
  static constexpr int kColumns = kTiles == 1 ? 256 : 512;
  static constexpr int kSmem = 1024 + kQBytes + kSlots * kSlotBytes + kControl;
  static_assert(sizeof(RowsShared) <= kControl, "control block");
  static_assert(kSlots >= 3 && kSmem <= kMaxDyn, "ring");
};

// Flags of a group for the rows of tokens [i0, i1).
template <bool kTree>
__device__ __forceinline__ uint32_t group_flags(const Keys &k, const Group &g, int i0, int i1) {
  if (g.page == -2) return 0x100u;
  if constexpr (kTree) {
    if (g.page == -1) return 0x10001u;
    return g.base + kPage > k.T ? 1u : 0u;
  } else {
    const int pa = k.p0 + i0, pb = k.p0 + i1 - 1;
    const bool all = g.base + kPage - 1 <= pa && (!k.windowed || g.base + kPage <= k.sink || g.base > pb - k.local);
    return all ? 0u : 1u;
  }
}

// Four codes as four bf16 (exact: E4M3 times 2^120 from the bits in place, INT8 by adding in the
// low mantissa bits); with `scaled`, times 2^e.
template <bool I8>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, bool scaled, __nv_bfloat162 two_e, uint32_t &lo, uint32_t &hi) {
  __nv_bfloat162 v[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (I8) {
      const uint32_t x = __byte_perm(w, 0, j == 0 ? 0x4140 : 0x4342);
      const uint32_t p = (x & 0x007f007fu) | 0x43004300u, n = (x & 0x00800080u) | 0x43004300u;
      v[j] = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&p), *reinterpret_cast<const __nv_bfloat162 *>(&n));
    } else {
      const uint32_t x = __byte_perm(w, 0, j == 0 ? 0x1404 : 0x3424);
      const uint32_t y = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
      const uint32_t up = 0x7b807b80u;   // 2^120
      v[j] = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), *reinterpret_cast<const __nv_bfloat162 *>(&up));
    }
    if (scaled) v[j] = __hmul2(v[j], two_e);
  }
  lo = *reinterpret_cast<const uint32_t *>(&v[0]);
  hi = *reinterpret_cast<const uint32_t *>(&v[1]);
  if constexpr (!I8) {
    // 0x7f and 0xff are NaN
    if ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0) {
      if ((w & 0x7fu) == 0x7fu) lo |= 0x00007fffu;
      if ((w & 0x7f00u) == 0x7f00u) lo |= 0x7fff0000u;
      if ((w & 0x7f0000u) == 0x7f0000u) hi |= 0x00007fffu;
      if ((w & 0x7f000000u) == 0x7f000000u) hi |= 0x7fff0000u;
    }
  }
}

// A scale as m * 2^e, 2^e a normal bf16 (returned twice in a word); m in [1, 2), smaller for a
// subnormal scale, and what there is for 0, infinity and NaN.
__device__ __forceinline__ uint32_t split_scale(float s, float &m) {
  const uint32_t bits = __float_as_uint(s), e = (bits >> 23) & 0xffu;
  if (e == 0xffu || s == 0.0f) {
    m = s;
    return 0x3f803f80u;
  }
  const uint32_t ee = e == 0 ? 1u : e;   // subnormal: 2^-126
  m = e == 0 ? s * 8.507059173023462e37f : __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);   // (2^126)
  return ee << 7 | ee << 23;
}

template <int D, int kKv, int kTiles, bool kTree>
__global__ void __launch_bounds__(RowsTraits<D, kKv, kTiles>::kThreads, 1)
    rows_mma_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ RowsPlan p, const __grid_constant__ RowsMaps maps) {
  using Tr = RowsTraits<D, kKv, kTiles>;
  constexpr int kSlots = Tr::kSlots;
  extern __shared__ unsigned char raw_smem[];
  unsigned char *smem = align_smem_1024(raw_smem);
  unsigned char *q_smem = smem, *ring = smem + Tr::kQBytes;
  RowsShared &sh = *reinterpret_cast<RowsShared *>(ring + kSlots * Tr::kSlotBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.dims.n_q_heads / a.dims.n_kv_heads;

  if (warp == Tr::kRowWarps) {
    tmem_alloc(&sh.tmem, Tr::kColumns);
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(&sh.full[i], Tr::kQuant ? Tr::kCopyWarps : 1);
        mbar_init(&sh.empty[i], 1);
      }
      mbar_init(&sh.q_full, 1);
      for (int t = 0; t < kTiles; ++t) {
        mbar_init(&sh.s_full[t], 1);
        mbar_init(&sh.p_full[t][0], 4);
        mbar_init(&sh.p_full[t][1], 4);
        mbar_init(&sh.o_full[t], 1);
      }
      mbar_init(&sh.drained, 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    tmem_fence_before();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // everything before this call has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    RowsItem it;
    const int64_t index = blockIdx.x / p.splits;
    find_item<kTree>(a, p, index, static_cast<int>(blockIdx.x - index * p.splits), it);
    if (lane == 0) sh.item = it;
  }
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  const RowsItem &it = sh.item;
  const int t_lo = it.t_lo, t_hi = it.t_hi;
  const uint32_t s_col[2] = {tmem, tmem + 128}, o_col[2] = {tmem + 128 * kTiles, tmem + 128 * kTiles + 128};
  // Tiles that hold rows (a last block may have one only).
  const int live_tiles = kTiles == 1 || it.i1 - it.i0 <= p.tokens ? 1 : 2;
  // A whole warp waits; false (for every lane) when a wait ran out. Each role then leaves its loop.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.st, p.wait_ns));
  };

  if (t_lo < t_hi) {
    if (warp > Tr::kRowWarps) {
      // ---- copy warps ----------------------------------------------------------------------
      const Keys k = it.k;
      const int64_t row0 = it.r.row0;
      const int h = it.h;
      auto group_of = [&](int j) -> Group {     // lanes 0..7: a tile's groups
        const int i = j * kTileGroups + lane;
        if (lane < kTileGroups && j < t_hi && i < k.n_groups) return key_group<kTree>(a, k, i);
        return Group{0, -2};
      };
      auto flags_of = [&](const Group &g) -> uint32_t {
        const uint32_t f = lane < kTileGroups ? group_flags<kTree>(k, g, it.i0, it.i1) : 0u;
        return __ballot_sync(0xffffffffu, f & 1u) | __ballot_sync(0xffffffffu, f & 0x100u) << 8 |
               __ballot_sync(0xffffffffu, f & 0x10000u) << 16;
      };
      int item = 0;
      if constexpr (!Tr::kQuant) {
        // q rows of the block, tile by tile: [token][head of the group], 64 columns at a time
        const int kv = warp - Tr::kRowWarps - 1;       // 0: K, 1: V
        if (kv == 0 && lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, static_cast<uint32_t>(live_tiles * Tr::kHalves * p.tokens * G * 128));
          for (int t = 0; t < live_tiles; ++t)
            for (int x = 0; x < Tr::kHalves; ++x)
              tma_3d(q_smem + t * (128 * D * 2) + x * 16384, &maps.q, x * 64, h * G, static_cast<int>(row0) + it.i0 + t * p.tokens, &sh.q_full);
        }
        const CUtensorMap *map = kv == 0 ? &maps.k : &maps.v, *map_new = kv == 0 ? &maps.k_new : &maps.v_new;
        const int box_page = lane / Tr::kHalves % kTileGroups, half = lane % Tr::kHalves;
        Group g = group_of(t_lo);
        bool ok = true;
        item = kv;
        for (int j = t_lo; j < t_hi; ++j, item += 2) {
          const uint32_t flags = flags_of(g);
          const int boxes = __popc(~(flags >> 8) & 0xffu) * Tr::kHalves;
          const int page = __shfl_sync(0xffffffffu, g.page, box_page), base = __shfl_sync(0xffffffffu, g.base, box_page);
          const int my_base = g.base;
          g = group_of(j + 1);     // (its loads fly beside this tile's copies)
          const int slot = item % kSlots;
          ok = wait(&sh.empty[slot], (item / kSlots & 1) ^ 1);
          if (!ok) break;
          if (kv == 0) {
            TileInfo &info = sh.info[(j - t_lo) % kInfos];
            if (lane < kTileGroups) info.base[lane] = my_base;
            if (lane == 0) info.flags = flags;
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], static_cast<uint32_t>(boxes * kPage * 128));
          __syncwarp();
          if (lane < kTileGroups * Tr::kHalves && page != -2) {
            unsigned char *dst = ring + slot * Tr::kSlotBytes + half * Tr::kHalfBytes + box_page * (kPage * 128);
            if (kTree && page == -1) tma_2d(dst, map_new, h * D + half * 64, static_cast<int>(row0) + base, &sh.full[slot]);
            else tma_2d(dst, map, half * 64, page * kPage, &sh.full[slot]);
          }
        }
        // (after a wait that ran out: the copies in flight land before the CTA leaves)
        if (!ok)
          for (int i = item - 2; i >= 0 && i > item - kSlots; i -= 2) mbar_wait_bounded(&sh.full[i % kSlots], i / kSlots & 1, a.st, p.wait_ns);
      } else {
        constexpr int kChunks = kPage * D / 16 / 32;     // 16-code loads of a lane and page
        constexpr int kPerRow = D / 16;
        const int cw = warp - Tr::kRowWarps - 1;         // takes groups 2 cw, 2 cw + 1 of a tile
        if (cw == 0 && lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, static_cast<uint32_t>(live_tiles * Tr::kHalves * p.tokens * G * 128));
          for (int t = 0; t < live_tiles; ++t)
            for (int x = 0; x < Tr::kHalves; ++x)
              tma_3d(q_smem + t * (128 * D * 2) + x * 16384, &maps.q, x * 64, h * G, static_cast<int>(row0) + it.i0 + t * p.tokens, &sh.q_full);
        }
        struct Pages {
          int page[2], base[2];
        };
        auto my_pages = [&](const Group &g) {
          Pages x;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x.page[i] = __shfl_sync(0xffffffffu, g.page, 2 * cw + i);
            x.base[i] = __shfl_sync(0xffffffffu, g.base, 2 * cw + i);
          }
          return x;
        };
        auto chunk_of = [&](int page, bool is_v, int c) -> uint4 {
          const uint8_t *pool = static_cast<const uint8_t *>(is_v ? a.kv.v_pool : a.kv.k_pool);
          return page >= 0 ? ld_stream16(pool + static_cast<int64_t>(page) * (kPage * D) + (c * 32 + lane) * 16) : make_uint4(0u, 0u, 0u, 0u);
        };
        // two bf16 chunks of 16 bytes at the place of a row's 16 elements from col on
        auto put = [&](unsigned char *slot, int row, int col, uint4 lo, uint4 hi) {
          unsigned char *at = slot + (col / 64) * Tr::kHalfBytes + row * 128;
          const int c = col % 64 / 8;
          *reinterpret_cast<uint4 *>(at + ((c ^ (row & 7)) * 16)) = lo;
          *reinterpret_cast<uint4 *>(at + (((c + 1) ^ (row & 7)) * 16)) = hi;
        };
        // Writes an item (K or V of a tile) from the codes in raw, and loads the next one's behind them.
        auto store = [&](const Pages &x, bool is_v, uint4 (&raw)[2][kChunks], const uint32_t (&two_e)[2], unsigned char *slot, const Pages &then) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int g_row = (2 * cw + i) * kPage;
            if (kTree && x.page[i] == -1) {              // drafts are bf16 already
              const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(is_v ? a.drafts.v_new : a.drafts.k_new) + static_cast<int64_t>(h) * D;
#pragma unroll 1
              for (int c = lane; c < kPage * kPerRow; c += 32) {
                const int row = c / kPerRow, col = c % kPerRow * 16;
                uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                if (x.base[i] + row < k.n_draft) {
                  const __nv_bfloat16 *at = src + (row0 + x.base[i] + row) * a.drafts.row_stride + col;
                  lo = ld_stream16(at);
                  hi = ld_stream16(at + 8);
                }
                put(slot, g_row + row, col, lo, hi);
              }
            }
            const __nv_bfloat162 e = *reinterpret_cast<const __nv_bfloat162 *>(&two_e[i]);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const uint4 w = raw[i][c];
              raw[i][c] = chunk_of(then.page[i], !is_v, c);
              if (x.page[i] >= 0) {
                const int chunk = c * 32 + lane, row = chunk / kPerRow, col = chunk % kPerRow * 16;
                uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                if (x.base[i] + row < k.T) {
                  codes_to_bf16<kKv == 2>(w.x, is_v, e, lo.x, lo.y);
                  codes_to_bf16<kKv == 2>(w.y, is_v, e, lo.z, lo.w);
                  codes_to_bf16<kKv == 2>(w.z, is_v, e, hi.x, hi.y);
                  codes_to_bf16<kKv == 2>(w.w, is_v, e, hi.z, hi.w);
                }
                put(slot, g_row + row, col, lo, hi);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        };
        // (pages and their scales one tile ahead, codes one item ahead)
        struct Scales {
          float k, v;
        };
        auto scales_of = [&](const Group &g) -> Scales {
          return g.page >= 0 ? Scales{a.kv.k_scale[g.page], a.kv.v_scale[g.page]} : Scales{1.0f, 1.0f};
        };
        Group g = group_of(t_lo);
        Scales sc = scales_of(g);
        Pages now = my_pages(g);
        uint4 raw[2][kChunks];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) raw[i][c] = chunk_of(now.page[i], false, c);
        for (int j = t_lo; j < t_hi; ++j) {
          const uint32_t flags = flags_of(g);
          float vm = 1.0f;
          const uint32_t ve = split_scale(sc.v, vm);
          const uint32_t two_e[2] = {__shfl_sync(0xffffffffu, ve, 2 * cw), __shfl_sync(0xffffffffu, ve, 2 * cw + 1)};
          const int my_base = g.base;
          const float ks = sc.k;
          g = group_of(j + 1);
          const Pages next = my_pages(g);
          int slot = item % kSlots;
          if (!wait(&sh.empty[slot], (item / kSlots & 1) ^ 1)) break;
          if (cw == 0) {
            TileInfo &info = sh.info[(j - t_lo) % kInfos];
            if (lane < kTileGroups) {
              info.base[lane] = my_base;
              info.ks[lane] = ks;
              info.vs[lane] = vm;
            }
            if (lane == 0) info.flags = flags;
          }
          store(now, false, raw, two_e, ring + slot * Tr::kSlotBytes, now);
          if (lane == 0) mbar_arrive(&sh.full[slot]);
          ++item;
          sc = scales_of(g);
          slot = item % kSlots;
          if (!wait(&sh.empty[slot], (item / kSlots & 1) ^ 1)) break;
          store(now, true, raw, two_e, ring + slot * Tr::kSlotBytes, next);
          if (lane == 0) mbar_arrive(&sh.full[slot]);
          ++item;
          now = next;
        }
      }
    } else if (warp == Tr::kRowWarps) {
      // ---- product warp ------------------------------------------------------------------------
      constexpr uint32_t kShapeS = umma_shape(kKeyTile, false), kShapeO = umma_shape(D, true);
      const int n = t_hi - t_lo, T = it.k.T;
      const uint32_t lead = elect_lane();
      // Operands of the first slot and the first row tile; others lie at whole steps of the address field.
      const uint64_t q_op = umma_operand(smem_u32(q_smem), 16, 1024), k_op = umma_operand(smem_u32(ring), 16, 1024);
      const uint64_t v_op = umma_operand(smem_u32(ring), Tr::kHalfBytes, 1024);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t s_tm[2] = {tm, tm + 128}, o_tm[2] = {tm + 128 * kTiles, tm + 128 * kTiles + 128};
      auto logits = [&](int t, int slot) {      // S of row tile t
        const uint64_t kd = k_op + static_cast<uint32_t>(slot * (Tr::kSlotBytes / 16)), qd = q_op + static_cast<uint32_t>(t * (128 * D * 2 / 16));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * (16384 / 16) + (kk % 4) * (32 / 16);
          umma_ss(lead, s_tm[t], qd + off, kd + off, kShapeS, kk > 0);
        }
      };
      uint32_t started = 0;      // bit t: O of row tile t has been written
      bool ok = wait(&sh.q_full, 0) && wait(&sh.full[0], 0);
      if (ok) {
        tmem_fence_after();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t >= live_tiles) break;
          logits(t, 0);
          umma_commit(lead, &sh.s_full[t]);
        }
        umma_commit(lead, &sh.empty[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int v_item = 2 * j + 1, v_slot = v_item % kSlots;
        const int k_item = 2 * j + 2, k_slot = k_item % kSlots;
        const TileInfo &info = sh.info[j % kInfos];
        ok = wait(&sh.full[v_slot], v_item / kSlots & 1);
        if (!ok) break;
        const uint32_t flags = info.flags;
        if constexpr (!Tr::kQuant) {
          // rows of V past the cache's end or the drafts' are not zero by themselves
          uint32_t marked = flags & ~(flags >> 8) & 0xffu;
          bool wrote = false;
          while (marked != 0) {
            const int i = __ffs(marked) - 1;
            marked &= marked - 1;
            const int end = (kTree && (flags >> (16 + i) & 1u)) ? it.k.n_draft : T;
            const int kept = end - info.base[i];
            if (kept >= kPage) continue;
            wrote = true;
            unsigned char *at = ring + v_slot * Tr::kSlotBytes + i * (kPage * 128);
            for (int c = lane; c < (kPage - kept) * 8 * Tr::kHalves; c += 32)
              *reinterpret_cast<uint4 *>(at + (c % Tr::kHalves) * Tr::kHalfBytes + kept * 128 + c / Tr::kHalves * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          if (wrote) fence_proxy_async_smem();
          __syncwarp();
        }
        if (j + 1 < n) ok = wait(&sh.full[k_slot], k_item / kSlots & 1);
        const uint64_t vd = v_op + static_cast<uint32_t>(v_slot * (Tr::kSlotBytes / 16));
        const uint32_t there = __reduce_or_sync(0xffffffffu, ~(flags >> 8) & 0xffu);     // pages of the tile
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t >= live_tiles || !ok) break;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            ok = wait(&sh.p_full[t][part], j & 1);
            if (!ok) break;
            tmem_fence_after();
            const uint32_t here = there >> (4 * part) & 0xfu;
            if (here == 0xfu) {
#pragma unroll
              for (int i = 4 * part; i < 4 * part + 4; ++i)
                umma_ts(lead, o_tm[t], s_tm[t] + i * 8, vd + static_cast<uint32_t>(i * (kPage * 128 / 16)), kShapeO,
                        i > 4 * part || (started >> t & 1u));
              started |= 1u << t;
            } else {
#pragma unroll 1
              for (uint32_t left = here; left != 0; left &= left - 1) {
                const int i = 4 * part + __ffs(left) - 1;
                umma_ts(lead, o_tm[t], s_tm[t] + i * 8, vd + static_cast<uint32_t>(i * (kPage * 128 / 16)), kShapeO,
                        (started >> t & 1u) != 0);
                started |= 1u << t;
              }
            }
          }
          if (!ok) break;
          if (t == live_tiles - 1) umma_commit(lead, &sh.empty[v_slot]);
          if (j + 1 < n) {
            logits(t, k_slot);
            umma_commit(lead, &sh.s_full[t]);
            if (t == live_tiles - 1) umma_commit(lead, &sh.empty[k_slot]);
          } else {
            umma_commit(lead, &sh.o_full[t]);
          }
        }
      }
      if (!ok) {     // products in flight end before the tensor memory is given back
        umma_commit(lead, &sh.drained);
        wait(&sh.drained, 0);
      }
    } else {
      // ---- row warps -----------------------------------------------------------------------------
      const int t = warp / 4;
      if (t < live_tiles) {
        const int row = (warp % 4) * 32 + lane;
        const int i = it.i0 + t * p.tokens + row / G, gq = row % G;
        const bool valid = row < p.tokens * G && i < it.i1;
        const bool any = __any_sync(0xffffffffu, valid);
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const uint32_t s_at = s_col[t] + lanes, o_at = o_col[t] + lanes;
        const Keys &k = it.k;
        const int pos = k.p0 + i;
        const float sc = kLog2e * rsqrtf(static_cast<float>(D));
        uint64_t mask = 0;
        if (kTree && valid) {
          mask = a.drafts.visible[it.r.row0 + i];
          if (k.n_draft < 64) mask &= (1ull << k.n_draft) - 1;
        }
        float m = -INFINITY, l = 0.0f;       // reference in the logits' units (times sc: log2), sum
        float pend = -INFINITY;              // maximum of the last second half
        const int n = t_hi - t_lo;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
          ok = wait(&sh.s_full[t], j & 1);
          if (!ok) break;
          tmem_fence_after();
          if (any) {
            const TileInfo &info = sh.info[j % kInfos];
            const uint32_t flags = info.flags;
            // bf16: the tile's logits stay in registers. 8-bit (whose copy warps need registers too):
            // they are read twice, 32 at a time, for the maximum and for the weights.
            constexpr bool kKeep = !Tr::kQuant;
            float s[kKeep ? 128 : 32];
            auto fetch = [&](int c32) {
              tmem_ld32(s_at + c32 * 32, s);
              tmem_wait_ld();
            };
            if constexpr (kKeep) {
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, s + c * 32);
            }
            // What the row sees, a bit a key.
            uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            const bool masked = (flags & 0xffffu) != 0;
            if (masked) {
#pragma unroll
              for (int gi = 0; gi < kTileGroups; ++gi) {
                if ((flags >> gi | flags >> (8 + gi)) & 1u) {
                  const int base = info.base[gi];
                  uint32_t bits;
                  if (flags >> (8 + gi) & 1u) {
                    bits = 0;
                  } else if constexpr (kTree) {
                    if (flags >> (16 + gi) & 1u) {
                      bits = static_cast<uint32_t>(mask >> base) & 0xffffu;
                    } else {
                      bits = (1u << min(k.T - base, kPage)) - 1u;
                    }
                  } else {
                    // t <= p: keys [0, p - base]; t > p - local or t < sink: all but [sink - base, p - local - base]
                    auto below = [](int x) -> uint32_t { return x <= 0 ? 0u : x >= 16 ? 0xffffu : (1u << x) - 1u; };
                    bits = below(pos - base + 1);
                    if (k.windowed) bits &= below(k.sink - base) | ~below(pos - k.local - base + 1);
                  }
                  seen[gi / 2] &= gi % 2 == 0 ? 0xffff0000u | bits : 0xffffu | bits << 16;
                }
              }
            }
            auto largest = [&](const float *x) -> float {      // of 16
              float top[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) top[c] = fmaxf(fmaxf(x[c], x[4 + c]), fmaxf(x[8 + c], x[12 + c]));
              return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            if constexpr (kKeep) tmem_wait_ld();
            auto half_max = [&](int half) -> float {
              float mx = -INFINITY;
#pragma unroll
              for (int c32 = 2 * half; c32 < 2 * half + 2; ++c32) {
                if constexpr (!kKeep) fetch(c32);
                float *x = kKeep ? s + c32 * 32 : s;
                if (masked) {
#pragma unroll
                  for (int c = 0; c < 32; ++c)
                    if (!(seen[c32] >> c & 1u)) x[c] = -INFINITY;
                }
#pragma unroll
                for (int gi = 0; gi < 2; ++gi) {
                  float of = largest(x + gi * 16);
                  if (Tr::kQuant && of != -INFINITY) of *= info.ks[c32 * 2 + gi];
                  mx = fmaxf(mx, of);
                }
              }
              return mx;
            };
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            auto half_weights = [&](int half) {
              const float base_m = m == -INFINITY ? 0.0f : -m * sc;
              const float2 m2 = make_float2(base_m, base_m);
#pragma unroll
              for (int c32 = 2 * half; c32 < 2 * half + 2; ++c32) {
                if constexpr (!kKeep) fetch(c32);
                const float *from = kKeep ? s + c32 * 32 : s;
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const int gi = c32 * 2 + x / 8;
                  const float to_log2 = Tr::kQuant ? info.ks[gi] * sc : sc;
                  float2 y = __ffma2_rn(make_float2(from[2 * x], from[2 * x + 1]), make_float2(to_log2, to_log2), m2);
                  if (!kKeep && masked) {
                    if (!(seen[c32] >> (2 * x) & 1u)) y.x = -INFINITY;
                    if (!(seen[c32] >> (2 * x + 1) & 1u)) y.y = -INFINITY;
                  }
                  float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                  sum[x & 1] = __fadd2_rn(sum[x & 1], e);
                  if constexpr (Tr::kQuant) {
                    const float vs = info.vs[gi];
                    e = __fmul2_rn(e, make_float2(vs, vs));
                  }
                  w[x] = pack_bf16(e.x, e.y);
                }
                tmem_st16(s_at + c32 * 16, w);
              }
              tmem_wait_st();
              tmem_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.p_full[t][half]);
            };
            const float mx = fmaxf(half_max(0), pend);
            if (m == -INFINITY) m = mx;      // (nothing seen before: O's row is zero)
            const bool grow = valid && (mx - m) * sc > 8.0f;
            if (__any_sync(0xffffffffu, grow)) {
              const float to = grow ? mx : m;
              const float f = grow ? exp2_approx((m - to) * sc) : 1.0f;
              m = to;
              l *= f;
              if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  float o[16];
                  tmem_ld16(o_at + c * 16, o);
                  tmem_wait_ld();
                  uint32_t w[16];
#pragma unroll
                  for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * f);
                  tmem_st16(o_at + c * 16, w);
                }
              }
            }
            half_weights(0);
            pend = half_max(1);
            if (m == -INFINITY) m = pend;    // (its row of O is still zero, its first half's weights too)
            half_weights(1);
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          } else if (lane == 0) {
            mbar_arrive(&sh.p_full[t][0]);
            mbar_arrive(&sh.p_full[t][1]);
          }
        }
        if (ok) ok = wait(&sh.o_full[t], 0);
        if (ok && any) {
          tmem_fence_after();
          const float m_log2 = m == -INFINITY ? -INFINITY : m * sc;
          const bool last = it.n_splits == 1;
          const int64_t out_row = (it.r.row0 + i) * a.dims.n_q_heads + it.h * G + gq;
          const int64_t rec = static_cast<int64_t>(blockIdx.x) * p.record_rows + (t * p.tokens * G + row);
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          float odd = fabsf(l);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(o_at + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              if (l == 0.0f) o[x] = 0.0f;      // (a row that has seen nothing: no product may have written its O)
              odd = odd + 0.0f * o[x];         // NaN when one is not finite
            }
            if (valid) {
              if (last) {
                uint4 *to = reinterpret_cast<uint4 *>(a.out + out_row * D + c * 32);
#pragma unroll
                for (int x = 0; x < 32; x += 8)
                  to[x / 8] = make_uint4(pack_bf16(o[x] * inv, o[x + 1] * inv), pack_bf16(o[x + 2] * inv, o[x + 3] * inv),
                                         pack_bf16(o[x + 4] * inv, o[x + 5] * inv), pack_bf16(o[x + 6] * inv, o[x + 7] * inv));
              } else {
                float4 *to = reinterpret_cast<float4 *>(p.rec_o + rec * D + c * 32);
#pragma unroll
                for (int x = 0; x < 32; x += 4) to[x / 4] = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
              }
            }
          }
          if (valid) {
            if (!last) p.rec_ml[rec] = make_float2(m_log2, l);
            else if (a.lse != nullptr) a.lse[out_row] = l == 0.0f ? -INFINITY : (m_log2 + log2f(l)) * kLn2;
          }
          // Rows that are not finite are computed again, one after the other, by the whole warp.
          unsigned again = __ballot_sync(0xffffffffu, valid && !(odd < INFINITY));
          while (again != 0) {
            const int src = __ffs(again) - 1;
            again &= again - 1;
            const int ri = __shfl_sync(0xffffffffu, i, src), rg = __shfl_sync(0xffffffffu, gq, src);
            const int64_t r_out = __shfl_sync(0xffffffffu, out_row, src), r_rec = __shfl_sync(0xffffffffu, rec, src);
            float rm, rl, ro[D / 32];
            row_attend<D, kTree>(a, it.r, k, it.h, ri, rg, t_lo * kTileGroups, min(t_hi * kTileGroups, k.n_groups), rm, rl, ro);
            __syncwarp();                      // (after what the row's own lane has written)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
              if (last) a.out[r_out * D + lane * (D / 32) + e] = __float2bfloat16_rn(rl == 0.0f ? 0.0f : ro[e] / rl);
              else p.rec_o[r_rec * D + lane * (D / 32) + e] = ro[e];
            }
            if (lane == 0) {
              if (!last) p.rec_ml[r_rec] = make_float2(rm, rl);
              else if (a.lse != nullptr) a.lse[r_out] = rl == 0.0f ? -INFINITY : (rm + log2f(rl)) * kLn2;
            }
          }
        }
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == Tr::kRowWarps) {
    tmem_fence_after();
    tmem_free(tmem, Tr::kColumns);
  }
}

template <int D, int kKv, int kTiles, bool kTree>
bs_status launch_rows_mma(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int64_t items, cudaStream_t cs) {
  using Tr = RowsTraits<D, kKv, kTiles>;
  auto kernel = rows_mma_kernel<D, kKv, kTiles, kTree>;
  static OncePerDevice attrs;
  if (!attrs([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Tr::kSmem) == cudaSuccess; }))
    return BS_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(items * p.splits));
  return launch_ex(kernel, grid, Tr::kThreads, Tr::kSmem, cs, 0, true, a, p, maps) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

// By the row tiles of a CTA (1 or 2) and the cache's type; each in a file of its own.
template <bool kTree>
bs_status launch_rows_bf16(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int64_t items, int tiles, cudaStream_t cs);
template <bool kTree>
bs_status launch_rows_quant(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int64_t items, int tiles, cudaStream_t cs);

template <int kKv, bool kTree>
bs_status dispatch_rows(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int64_t items, int tiles, cudaStream_t cs) {
  if (a.dims.head_dim == 128)
    return tiles == 1 ? launch_rows_mma<128, kKv, 1, kTree>(a, p, maps, items, cs) : launch_rows_mma<128, kKv, 2, kTree>(a, p, maps, items, cs);
  return tiles == 1 ? launch_rows_mma<64, kKv, 1, kTree>(a, p, maps, items, cs) : launch_rows_mma<64, kKv, 2, kTree>(a, p, maps, items, cs);
}

}  // namespace bsi
