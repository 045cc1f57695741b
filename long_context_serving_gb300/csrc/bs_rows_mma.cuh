// Rows of new tokens against tiles of 128 keys on the fifth-generation tensor cores.
//
// One CTA takes one KV head's rows of a block of tokens (all query heads of the group: a K or V
// tile is fetched once for all of them), packed as 128-row tiles of whole tokens, kTiles of them
// (1 or 2), against a contiguous piece of the block's key groups:
//   copy warps     one for K, one for V: fetch tiles of 128 keys into a ring of shared-memory slots,
//                  bf16 pages by tiled copies; 8-bit pages by bulk copies into a ring of their own,
//   (8-bit) eight warps write the bf16 values that the codes stand for into the ring's slots;
//   product warp   S = Q K^T into tensor memory (one thread issues); O += P V with P from tensor
//                  memory, page by page, so that a page that is not there takes no part;
//   row warps      four a tile, a thread a row: logits from tensor memory, the running maximum and
//                  sum in registers, weights back to tensor memory as bf16, over the logits.
// S of the next key tile is issued behind O's update, so with two tiles one's products run beside
// the other's softmax; weights are handed over in two parts, 96 keys and 32, so that O's update
// starts while the last are made and the rest of it and S do not wait for much. O is brought to a
// new maximum only when that has grown by more than 2^8 (the final division takes it back), at the
// start of a tile, when the products in flight are done: O's rescaling through registers is rare and
// needs no warps of its own. The second half of a tile is measured against the same reference, and
// only where it passes that by 2^30 is everything brought to its maximum at once. So 64 weights are
// 2^30 at most, until the next tile's start brings them to 2^8 too: with V up to 2^90 sums stay below
// 2^127. Records of split rows are divided by their own sums, so that as many as there are can be added.
// Tiles are 128 rows for the tensor cores' full rate and 128 keys because a product of 128 x 128 takes
// from shared memory just what that delivers meanwhile (128 bytes a cycle); two row tiles are what
// tensor memory holds (512 columns: S and O of each, weights over S).
// Bounds, measured: with two row tiles, S's and O's products (2,048 cycles a key tile) against a
// tile's chain of 330 (S ready) + 1,640 to 1,800 (softmax) + 900 cycles, by clock stamps in an
// instrumented copy of an earlier step: half of a 16K prompt, 8 heads of 4 queries, half of them
// streaming, 670 to 702 us over several machines, 1.38 to 1.45 PFLOP/s. 8-bit caches
// wait for conversion and shared memory (windows of four ragged chunks 190 us, bf16 128 to 135). With few
// rows HBM: 32 sequences' single tokens over 2K to 16K tokens 165 us, 5.9 TB/s; E4M3 225 us, conversion.
// Small trees: launch, lookup, copy, products, records and merge one after another, 10.9 us for eight
// drafts over 32K tokens.
// Precision: products of bf16 in fp32; weights enter as bf16 (off by up to 2^-8 of themselves), which is the
// operand type of V. A row is divided by the sum of its weights as they entered, so that the rounding of
// one that dominates falls out (against a plain form in fp32 with bf16 outputs trees are 1.9e-3 apart for 2.5e-3
// when divided by the sum before rounding, single tokens 1.7 for 2.3e-3); the other sum is lse's. It costs 4 to 5 %
// of prompts (half a 16K prompt 671 for 640 us, E4M3 1066 for 1016), 0 to 6 % of trees, 0 to 2 % of single tokens. (Weights
// in two parts, twice the products of P and V, took 5 to 17 % more of trees, 7 and 28 % of single tokens over bf16 and E4M3.)
// Page scales: K's multiplies logits in fp32; V's is m * 2^e, 2^e goes into the bf16 values (exact), m
// into the weights, by their exponent, so that neither a tiny nor a large scale leaves the type's range on its own.
// A key that a row does not see still stands in its products, with a weight of 0, and 0 times an
// infinity is a NaN. Slots past the cache's end are zeroed and pages that are not there left out; where
// a group that rows see differently holds a value that is not finite, the block is marked, and its
// rows' columns that are not finite are computed again without unseen keys (row_columns).
#pragma once

#include "bs_attn_launch.cuh"
#include "bs_rows_attn.cuh"
#include "bs_umma.cuh"

namespace bsi {

constexpr int kKeyTile = 128;                 // keys of a tile
constexpr int kTileGroups = kKeyTile / kPage; // groups of a tile
constexpr int kFirstKeys = 96;                // keys whose weights are handed over first
constexpr int kShareItems = 64;               // tree: items whose key tiles a wave of CTAs shares
constexpr uint64_t kInFlightNs = 10000000;    // longer than any copy or product takes
constexpr int kInfos = 8;                     // tiles whose description is kept

struct RowsPlan {
  int tokens;         // tokens of a row tile: its rows / G
  int block_tokens;   // of a CTA
  int n_blocks;       // tree: blocks of a sequence; prefill: of all sequences, at most, or 0: one of each
  int items;          // blocks of all units, at most
  int splits;         // CTAs a block's keys are split over, at most (1: records unused)
  int even;           // > 0: that many CTAs share all items' key tiles (tree_share)
  int record_rows;    // rows of a block, at most
  float *rec_o;       // [CTA][record_rows][D]: outputs over the CTA's keys
  float2 *rec_ml;     // [CTA][record_rows]: reference (log2 units), sum of the weights relative to it
  int4 *heads;        // [item]: CTAs that took part, the first of them, first row, rows
  uint64_t wait_ns;
};

struct RowsMaps {
  CUtensorMap q, k, v, k_new, v_new;
};

// 32 bytes, in one instruction where the address allows (a lane's row is far from the next lane's:
// each store then fills the sectors it touches).
__device__ __forceinline__ void store_sector(void *to, const uint32_t *w, bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// sum + the two bf16 of w, by additions of mixed types (with shifts and masks instead, half a 16K prompt took
// 723 us for 671). Volatile, so that they stay behind the store of what they add.
__device__ __forceinline__ void add_bf16x2(float2 &sum, uint32_t w) {
  asm volatile("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(sum.x), "+f"(sum.y)
      : "r"(w));
}

// Is one of eight bf16 infinite or NaN?
__device__ __forceinline__ bool any_odd_bf16(uint4 w) {
  auto top = [](uint32_t x) { return __vcmpgeu2(x & 0x7fff7fffu, 0x7f807f80u); };
  return (top(w.x) | top(w.y) | top(w.z) | top(w.w)) != 0;
}

// What a CTA works on.
struct RowsItem {
  SeqRows r;
  Keys k;
  int b, h, i0, i1;       // tokens [i0, i1) of the sequence
  int item;
  int t_lo, t_hi;         // key tiles of this CTA; empty: nothing to do
  int n_splits, first;    // CTAs that share the item, the first of them
};

__device__ __forceinline__ int key_tiles(const Keys &k) { return (k.n_groups + kTileGroups - 1) / kTileGroups; }

// Rows and keys of a tree's item from what is told of it: 0, or the status of a sequence or unit
// that does not fit (no tokens then).
struct ItemWords {
  SeqWords seq;
  UnitWords unit;
};
__device__ __forceinline__ ItemWords tree_words(const RowsArgs &a, const RowsPlan &p, int item) {
  const int u = p.n_blocks == 1 ? item : item / p.n_blocks;
  return ItemWords{seq_words<true>(a, u / a.dims.n_kv_heads), unit_words<true>(a, u)};
}
__device__ __forceinline__ int tree_item(const RowsArgs &a, const RowsPlan &p, int item, const ItemWords &w, RowsItem &it) {
  const int u = p.n_blocks == 1 ? item : item / p.n_blocks, block = item - u * p.n_blocks;
  it.b = u / a.dims.n_kv_heads;
  it.h = u - it.b * a.dims.n_kv_heads;
  it.i0 = it.i1 = 0;
  int bad = seq_rows<true>(a, w.seq, it.r);
  if (bad != 0) return bad;
  if (it.r.n <= block * p.block_tokens) return 0;
  const int i0 = block * p.block_tokens, i1 = min(i0 + p.block_tokens, it.r.n);
  bad = unit_keys<true>(a, it.r, w.unit, u, i0, i1, it.k);
  if (bad != 0) return bad;
  it.i0 = i0;
  it.i1 = i1;
  return 0;
}

// The tree's few items (at most kShareItems) over p.even CTAs: pieces of `per` tiles, about the
// smallest number that does not ask for more CTAs, whatever the units' own sizes; a key tile against
// two row tiles counts twice. Every CTA works this out by itself: a warp, a lane to every 32nd item,
// one round of loads.
constexpr int kLaneItems = kShareItems / 32;
__device__ __forceinline__ void tree_share(const RowsArgs &a, const RowsPlan &p, int cta, RowsItem &it) {
  const int lane = threadIdx.x & 31, used = (p.items + 31) / 32;
  ItemWords w[kLaneItems];
#pragma unroll
  for (int q = 0; q < kLaneItems; ++q)
    if (q < used) w[q] = tree_words(a, p, min(q * 32 + lane, p.items - 1));
  int n[kLaneItems], total = 0;
#pragma unroll
  for (int q = 0; q < kLaneItems; ++q) {
    const int item = q * 32 + lane;
    n[q] = 0;
    if (item < p.items) {
      RowsItem x;
      const int bad = tree_item(a, p, item, w[q], x);
      if (bad != 0 && cta == 0) report(a.st, bad);
      n[q] = x.i1 > x.i0 ? key_tiles(x.k) * (x.i1 - x.i0 > p.tokens ? 2 : 1) : 0;
      if (n[q] == 0 && cta == 0) p.heads[item] = make_int4(0, 0, 0, 0);
    }
    total += n[q];
  }
  total = __reduce_add_sync(0xffffffffu, total);
  int per = max(1, (total + p.even - 1) / p.even), pieces[kLaneItems];
  for (;; per += max(1, per / 16)) {
    const float inv = __frcp_rn(static_cast<float>(per));
    int ctas = 0;
#pragma unroll
    for (int q = 0; q < kLaneItems; ++q) {
      // (the quotient is at least 1 / (2 per) from an integer, its error below that for n < 2^21)
      pieces[q] = __float2int_rz((static_cast<float>(n[q] + per - 1) + 0.5f) * inv);
      ctas += pieces[q];
    }
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, ctas)) <= p.even) break;   // (items are no more than CTAs)
  }
  int before = 0;
  it.item = -1;
#pragma unroll
  for (int q = 0; q < kLaneItems; ++q) {
    if (q >= used) break;
    const int mine = pieces[q];
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned here = __ballot_sync(0xffffffffu, before + sum > cta);
    if (it.item < 0 && here != 0) {
      const int src = __ffs(here) - 1;
      it.item = q * 32 + src;
      it.n_splits = __shfl_sync(0xffffffffu, mine, src);
      it.first = before + __shfl_sync(0xffffffffu, sum, src) - it.n_splits;
      ItemWords x;
      x.seq.T = __shfl_sync(0xffffffffu, w[q].seq.T, src);
      x.seq.x = __shfl_sync(0xffffffffu, w[q].seq.x, src);
      x.seq.row0 = __shfl_sync(0xffffffffu, w[q].seq.row0, src);
      x.unit.x = __shfl_sync(0xffffffffu, w[q].unit.x, src);
      x.unit.y = __shfl_sync(0xffffffffu, w[q].unit.y, src);
      x.unit.z = 0;
      tree_item(a, p, it.item, x, it);
      const int tiles = key_tiles(it.k), s = cta - it.first;
      it.n_splits = min(it.n_splits, tiles);
      const int even = (tiles + it.n_splits - 1) / it.n_splits;      // (pieces of a unit alike)
      it.n_splits = (tiles + even - 1) / even;
      it.t_lo = min(s * even, tiles);
      it.t_hi = min(it.t_lo + even, tiles);
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
}

// Item of a CTA, by a whole warp (every lane gets it). Errors are reported once.
template <bool kTree>
__device__ __forceinline__ void find_item(const RowsArgs &a, const RowsPlan &p, int cta, RowsItem &it) {
  const int lane = threadIdx.x & 31;
  it.t_lo = it.t_hi = it.n_splits = 0;
  it.i0 = it.i1 = 0;
  if (kTree && p.even > 0) {
    tree_share(a, p, cta, it);
    return;
  }
  it.item = cta / p.splits;
  it.first = it.item * p.splits;
  const int split = cta - it.first;
  if constexpr (kTree) {
    const int bad = tree_item(a, p, it.item, tree_words(a, p, it.item), it);
    if (bad != 0 && lane == 0 && split == 0) report(a.st, bad);
  } else {
    it.h = it.item % a.dims.n_kv_heads;
    int block = 0;
    if (p.n_blocks == 0) {
      it.b = it.item / a.dims.n_kv_heads;
      const int bad = seq_rows<kTree>(a, seq_words<kTree>(a, it.b), it.r);
      if (bad != 0 && lane == 0 && split == 0 && it.h == 0) report(a.st, bad);
      if (it.r.n == 0) it.b = -1;
    } else {
      // Blocks are numbered sequence by sequence, each sequence's last block (which has the most keys)
      // first: 128 sequences at a time, a lane to four of them.
      constexpr int kEach = 4;
      int at = it.item / a.dims.n_kv_heads;                 // blocks before this one
      const bool first = cta == 0;                          // looks at every sequence, and reports
      int total = 0;
      it.b = -1;
      for (int b0 = 0; b0 < a.dims.batch && (it.b < 0 || first); b0 += 32 * kEach) {
        SeqWords w[kEach];
        int mine[kEach], sum = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) w[i] = seq_words<kTree>(a, min(b0 + lane * kEach + i, a.dims.batch - 1));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          SeqRows r;
          r.n = 0;
          const int bad = b0 + lane * kEach + i < a.dims.batch ? seq_rows<kTree>(a, w[i], r) : 0;
          if (bad != 0 && first) report(a.st, bad);
          mine[i] = (r.n + p.block_tokens - 1) / p.block_tokens;
          sum += mine[i];
        }
        int end = sum;                                      // blocks of this lane's sequences and those before
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += x;
        }
        const unsigned here = __ballot_sync(0xffffffffu, end > at);
        if (it.b < 0 && here != 0) {
          const int src = __ffs(here) - 1;
          int i = 0, before = end - sum;                    // (meant for lane src)
#pragma unroll
          for (int x = 0; x < kEach - 1; ++x)
            if (i == x && before + mine[x] <= at) {
              before += mine[x];
              ++i;
            }
          i = __shfl_sync(0xffffffffu, i, src);
          before = __shfl_sync(0xffffffffu, before, src);
          it.b = b0 + src * kEach + i;
          seq_rows<kTree>(a, seq_words<kTree>(a, it.b), it.r);
          block = before + (it.r.n + p.block_tokens - 1) / p.block_tokens - 1 - at;
        }
        const int all = __shfl_sync(0xffffffffu, end, 31);
        at -= all;
        total += all;
      }
      if (first && lane == 0 && total > p.n_blocks) report(a.st, BS_ERR_CAPACITY);   // sequences that share rows
    }
    if (it.b >= 0) {
      it.i0 = block * p.block_tokens;
      it.i1 = min(it.i0 + p.block_tokens, it.r.n);
      const int u = it.b * a.dims.n_kv_heads + it.h;
      const int bad = unit_keys<kTree>(a, it.r, unit_words<kTree>(a, u), u, it.i0, it.i1, it.k);
      if (bad != 0) {
        if (lane == 0 && split == 0) report(a.st, bad);
        it.i1 = it.i0;
      }
    }
  }
  if (it.i1 > it.i0) {
    const int n = key_tiles(it.k), per = max(1, (n + p.splits - 1) / p.splits);
    it.n_splits = (n + per - 1) / per;
    it.t_lo = min(split * per, n);
    it.t_hi = min(it.t_lo + per, n);
  }
  if (p.splits > 1 && split == 0 && it.n_splits == 0 && lane == 0) p.heads[it.item] = make_int4(0, 0, 0, 0);
}

// Description of a key tile, written by the copy warps.
struct TileInfo {
  int base[kTileGroups];      // first key of each group
  uint32_t flags;             // bits 0..7: rows differ in what they see of the group, or its end is
                              // past the cache's; 8..15: it is not there; 16..23: it is of drafts
  float2 ks[kTileGroups];     // 8-bit caches: K's scale; log2 of the mantissa of V's, in the logits' units
  float inv_vs[kTileGroups];  // 1 / that mantissa
  float ve[kTileGroups];      // its power of two
};

struct RowsShared {
  RowsItem item;
  TileInfo info[kInfos];
  uint64_t empty[12];         // a slot's products are done
  uint64_t raw_full[8], raw_empty[8];
  uint64_t k0_full, full[kInfos];   // K of the first tile; V of a tile and K of the next one, have landed
  uint64_t q_full, s_full[2], p_full[2][2], o_full[2], looked, never;   // (p_full: [row tile][part])
  uint32_t tmem;
  int failed;                 // a wait ran out
  int marked;                 // a group that rows see differently has a V that is not finite
};

// kRows: rows of a CTA, 256 (two row tiles), 128 or 32. With 32 (single tokens, small trees) one row
// warp and the first quarter of a tile do; the products' other rows are whatever lies behind the
// queries, in rows of S and O that nobody reads. Two such CTAs an SM: one's start and softmax beside the
// other's keys (32 sequences' single tokens, bf16: 164 us, with one 200).
template <int D, int kKv, int kRows>
struct RowsTraits {
  static constexpr bool kQuant = kKv != 0;              // 1: E4M3, 2: INT8
  static constexpr int kTiles = kRows == 256 ? 2 : 1;
  static constexpr int kPerSm = kRows == 32 ? 2 : 1;
  static constexpr int kHalves = D / 64;                // 128-byte columns of a row
  static constexpr int kSlotBytes = kKeyTile * D * 2;
  static constexpr int kHalfBytes = kKeyTile * 128;
  static constexpr int kQHalf = (kRows == 32 ? 32 : 128) * 128;   // 64 columns of a row tile's queries
  static constexpr int kQTile = kQHalf * kHalves;
  static constexpr int kQBytes = kTiles * kQTile;
  static constexpr int kControl = 2048;                 // RowsShared
  static constexpr int kMaxDyn = kPerSm == 2 ? 233472 / 2 - 1024 : 232448;   // shared memory of a CTA, at most
  // K or V tiles in codes. (Two row tiles, d = 128: four slots and two of these rather than three and
  // four, with which K's conversion waited for the products of the V before it.)
  static constexpr int kRaw = !kQuant ? 0 : kRows == 128 ? 4 : 2;
  static constexpr int kRawBytes = kQuant ? kKeyTile * D : 0;
  static constexpr int kRoom = (kMaxDyn - 1024 - kControl - kQBytes - kRaw * kRawBytes) / kSlotBytes;
  static constexpr int kSlots = kRoom < 12 ? kRoom : 12;
  static constexpr int kTileWarps = kRows == 32 ? 1 : 4;          // row warps of a tile
  static constexpr int kRowWarps = kTileWarps * kTiles;
  static constexpr int kWriters = !kQuant ? 1 : kRows == 32 ? 4 : 8;       // warps that fill a slot
  // Product warp, two copy warps, (8-bit) conversion warps, one on each scheduler, row warps from a
  // multiple of four.
  // (bf16, 128 and 256 rows: the warp that is left over looks for values that are not finite.)
  static constexpr bool kLooker = !kQuant && kRows != 32;
  static constexpr int kProduct = kRows == 32 ? 1 : 0, kCopy = kProduct + 1, kConvert = 4;
  static constexpr int kFirstRow = kRows == 32 ? 0 : kQuant ? 4 + kWriters : 4;
  static constexpr int kThreads = 32 * (kRows == 32 ? (kQuant ? 8 : 4) : kFirstRow + kRowWarps);
  static constexpr int kColumns = kTiles == 1 ? 256 : 512;
  static constexpr int kSmem = 1024 + kQBytes + kSlots * kSlotBytes + kRaw * kRawBytes + kControl;
  static_assert(sizeof(RowsShared) <= kControl, "control block");
  static_assert(kSlots >= 2 && kRaw <= 8 && kSmem <= kMaxDyn, "ring");
  static_assert(kQBytes + kSlots * kSlotBytes >= kQTile - kQHalf + 16384, "products read 128 rows");
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

// Four codes, with `scaled` times a power of two, as four bf16: exact short of bf16's range. (Through fp16 and fp32:
// 8 x 16 codes a lane 190 cycles more than their copy; placing the bits and multiplying by 2^120
// took 400, and 1500 with a look for NaN codes, which come through here by themselves.)
template <bool I8>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, bool scaled, float two_e, uint32_t &lo, uint32_t &hi) {
  float f[4];
  codes_to_f32<I8>(w, f);
  float2 a = make_float2(f[0], f[1]), b = make_float2(f[2], f[3]);
  if (scaled) {
    a = __fmul2_rn(a, make_float2(two_e, two_e));
    b = __fmul2_rn(b, make_float2(two_e, two_e));
  }
  lo = pack_bf16(a.x, a.y);
  hi = pack_bf16(b.x, b.y);
}

// A scale as m * 2^e, 2^e with its sign returned; m in [1, 2), smaller for a subnormal scale. 0, infinity
// and NaN are returned as they are, with m = 1.
__device__ __forceinline__ float split_scale(float s, float &m) {
  const uint32_t bits = __float_as_uint(s), e = (bits >> 23) & 0xffu;
  if (e == 0xffu || s == 0.0f) {
    m = 1.0f;
    return s;
  }
  m = e == 0 ? fabsf(s) * 8.507059173023462e37f : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);   // (2^126)
  return __uint_as_float((bits & 0x80000000u) | (e == 0 ? 1u : e) << 23);
}

template <int D, int kKv, int kRows, bool kTree>
__global__ void __launch_bounds__(RowsTraits<D, kKv, kRows>::kThreads, RowsTraits<D, kKv, kRows>::kPerSm)
    rows_mma_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ RowsPlan p, const __grid_constant__ RowsMaps maps) {
  using Tr = RowsTraits<D, kKv, kRows>;
  constexpr int kTiles = Tr::kTiles, kSlots = Tr::kSlots, kRaw = Tr::kQuant ? Tr::kRaw : 1;
  extern __shared__ unsigned char raw_smem[];
  unsigned char *smem = align_smem_1024(raw_smem);
  unsigned char *q_smem = smem, *ring = smem + Tr::kQBytes;
  unsigned char *raw_ring = ring + kSlots * Tr::kSlotBytes;
  RowsShared &sh = *reinterpret_cast<RowsShared *>(raw_ring + Tr::kRaw * Tr::kRawBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.dims.n_q_heads / a.dims.n_kv_heads;

  if (warp == Tr::kProduct) {
    tmem_alloc(&sh.tmem, Tr::kColumns);
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(&sh.empty[i], Tr::kLooker ? 2 : 1);
      }
      mbar_init(&sh.k0_full, Tr::kWriters);
      for (int i = 0; i < kInfos; ++i) mbar_init(&sh.full[i], 2 * Tr::kWriters);
      for (int i = 0; i < kRaw; ++i) {
        mbar_init(&sh.raw_full[i], 1);
        mbar_init(&sh.raw_empty[i], Tr::kWriters);
      }
      mbar_init(&sh.q_full, 1);
      for (int t = 0; t < kTiles; ++t) {
        mbar_init(&sh.s_full[t], 1);
        mbar_init(&sh.p_full[t][0], Tr::kTileWarps);
        mbar_init(&sh.p_full[t][1], Tr::kTileWarps);
        mbar_init(&sh.o_full[t], 1);
      }
      mbar_init(&sh.looked, 1);
      mbar_init(&sh.never, 1);
      sh.failed = 0;
      sh.marked = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    tmem_fence_before();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // everything before this call has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == Tr::kFirstRow) {
    RowsItem it;
    find_item<kTree>(a, p, static_cast<int>(blockIdx.x), it);
    if (lane == 0) {
      sh.item = it;
      if (it.n_splits > 0 && it.first == static_cast<int>(blockIdx.x) && p.splits > 1)
        p.heads[it.item] = make_int4(it.n_splits, it.first, static_cast<int>(it.r.row0) + it.i0, it.i1 - it.i0);
    }
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
  // Barrier on which an item (K or V of key tile j) lands: K of a tile goes with V of the one before.
  auto full_of = [&](int j, int kv) -> uint64_t * {
    const int pair = j - t_lo - (kv == 0);
    return pair < 0 ? &sh.k0_full : &sh.full[pair % kInfos];
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.st, p.wait_ns))) return true;
    *const_cast<volatile int *>(&sh.failed) = 1;
    return false;
  };

  // Rows of group i of a tile that are tokens or drafts (bf16).
  auto kept_rows = [&](const TileInfo &info, int i) -> int {
    const int end = (kTree && (info.flags >> (16 + i) & 1u)) ? it.k.n_draft : it.k.T;
    return min(end - info.base[i], kPage);
  };
  // Marks the block if a V of a group that rows see differently is not finite (bf16; a whole warp).
  auto look = [&](const TileInfo &info, int slot) {
    bool odd = false;
    for (uint32_t left = info.flags & ~(info.flags >> 8) & 0xffu; left != 0; left &= left - 1) {
      const int i = __ffs(left) - 1, kept = kept_rows(info, i);
      const unsigned char *at = ring + slot * Tr::kSlotBytes + i * (kPage * 128);
#pragma unroll 2
      for (int c = lane; c < kept * 8 * Tr::kHalves; c += 32)
        odd |= any_odd_bf16(*reinterpret_cast<const uint4 *>(at + (c % Tr::kHalves) * Tr::kHalfBytes + c / Tr::kHalves * 16));
    }
    if (__any_sync(0xffffffffu, odd)) {
      *const_cast<volatile int *>(&sh.marked) = 1;
      __threadfence_block();
    }
  };

  if (t_lo < t_hi) {
    if (warp == Tr::kCopy || warp == Tr::kCopy + 1) {
      // ---- copy warps: K, V -----------------------------------------------------------------
      const Keys k = it.k;
      const int64_t row0 = it.r.row0;
      const int h = it.h, kv = warp - Tr::kCopy;
      // Pages (and scales) are looked up for four tiles at once, a lane each, four tiles ahead: two or
      // three loads one behind another, mostly from memory.
      struct Lookup {
        Group g;
        float ks, inv_vs, ve, lv;            // as in TileInfo
        uint32_t differ, absent, drafts;     // of the 32 groups, as in TileInfo::flags
      };
      auto look_up = [&](int j) -> Group {
        const int i = j * kTileGroups + lane;
        return i < min(k.n_groups, t_hi * kTileGroups) ? key_group<kTree>(a, k, i) : Group{0, -2};
      };
      auto complete = [&](const Group &g) -> Lookup {
        Lookup x{g, 1.0f, 1.0f, 1.0f, 0.0f, 0u, 0u, 0u};
        if (Tr::kQuant && kv == 0 && g.page >= 0) {
          x.ks = a.kv.k_scale[g.page];
          float vs;
          x.ve = split_scale(a.kv.v_scale[g.page], vs);
          // (an error of the logarithm, 2^-21 of the weights, is one of V's scale)
          constexpr float kUnits = (D == 128 ? 11.3137085f : 8.0f) * kLn2;
          x.lv = __log2f(vs) * kUnits;
          x.inv_vs = __fdividef(1.0f, vs);
        }
        uint32_t f = group_flags<kTree>(k, g, it.i0, it.i1);
        if (Tr::kQuant && x.ks != x.ks) f |= 1u;     // (a NaN scale of K: the row warps put it into the logits)
        x.differ = __ballot_sync(0xffffffffu, f & 1u);
        x.absent = __ballot_sync(0xffffffffu, f & 0x100u);
        x.drafts = __ballot_sync(0xffffffffu, f & 0x10000u);
        return x;
      };
      // q rows of the block, tile by tile: [token][head of the group], 64 columns at a time
      if (kv == 0 && lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full, static_cast<uint32_t>(live_tiles * Tr::kHalves * p.tokens * G * 128));
        for (int t = 0; t < live_tiles; ++t)
          for (int x = 0; x < Tr::kHalves; ++x)
            tma_3d(q_smem + t * Tr::kQTile + x * Tr::kQHalf, &maps.q, x * 64, h * G, static_cast<int>(row0) + it.i0 + t * p.tokens, &sh.q_full);
      }
      const CUtensorMap *map = kv == 0 ? &maps.k : &maps.v, *map_new = kv == 0 ? &maps.k_new : &maps.v_new;
      const int box_page = Tr::kQuant ? lane % kTileGroups : lane / Tr::kHalves % kTileGroups, half = lane % Tr::kHalves;
      Lookup now = complete(look_up(t_lo)), then{};
      Group ahead{0, -2};
      bool ok = true;
      int item = kv;
      for (int j = t_lo; j < t_hi; ++j, item += 2) {
        const int s = (j - t_lo) % 4 * kTileGroups;          // the tile's lanes
        if (s == 0 && j > t_lo) now = then;
        const uint32_t flags = (now.differ >> s & 0xffu) | (now.absent >> s & 0xffu) << 8 | (now.drafts >> s & 0xffu) << 16;
        const int page = __shfl_sync(0xffffffffu, now.g.page, s + box_page), base = __shfl_sync(0xffffffffu, now.g.base, s + box_page);
        const int slot = item % (Tr::kQuant ? kRaw : kSlots), turn = item / (Tr::kQuant ? kRaw : kSlots);
        ok = wait(Tr::kQuant ? &sh.raw_empty[slot] : &sh.empty[slot], (turn & 1) ^ 1);
        if (!ok) break;
        if (kv == 0) {
          TileInfo &info = sh.info[(j - t_lo) % kInfos];
          if (lane >= s && lane < s + kTileGroups) {
            info.base[lane - s] = now.g.base;
            if constexpr (Tr::kQuant) {
              info.ve[lane - s] = now.ve;
              info.ks[lane - s] = make_float2(now.ks, now.lv);
              info.inv_vs[lane - s] = now.inv_vs;
            }
          }
          if (lane == 0) info.flags = flags;
          __syncwarp();
        }
        if constexpr (Tr::kQuant) {
          const int pages = __popc(~((flags >> 8) | (flags >> 16)) & 0xffu);
          if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[slot], static_cast<uint32_t>(pages * kPage * D));
          __syncwarp();
          if (lane < kTileGroups && page >= 0)
            bulk_g2s(raw_ring + slot * Tr::kRawBytes + lane * (kPage * D),
                     static_cast<const uint8_t *>(kv == 0 ? a.kv.k_pool : a.kv.v_pool) + static_cast<int64_t>(page) * (kPage * D), kPage * D,
                     &sh.raw_full[slot]);
        } else {
          uint64_t *bar = full_of(j, kv);
          const int boxes = __popc(~(flags >> 8) & 0xffu) * Tr::kHalves;
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * kPage * 128));
          if (kv == 1 && j == t_hi - 1 && lane == 0) mbar_arrive(bar);     // (there is no next K)
          __syncwarp();
          if (lane < kTileGroups * Tr::kHalves && page != -2) {
            unsigned char *dst = ring + slot * Tr::kSlotBytes + half * Tr::kHalfBytes + box_page * (kPage * 128);
            if (kTree && page == -1) tma_2d(dst, map_new, h * D + half * 64, static_cast<int>(row0) + base, bar);
            else tma_2d(dst, map, half * 64, page * kPage, bar);
          }
        }
        if (s == 0 && j + 4 < t_hi) ahead = look_up(j + 4);
        if (s == 3 * kTileGroups && j + 1 < t_hi) then = complete(ahead);
      }
    } else if (Tr::kQuant && warp >= Tr::kConvert && warp < Tr::kConvert + Tr::kWriters) {
      // ---- conversion warps: one group of every tile each -----------------------------------------------
      constexpr int kPieces = kPage * D / 16 / 32;       // 16-code pieces of a lane and page
      constexpr int kRowStep = kPage / kPieces;          // a lane's pieces lie this many rows apart
      constexpr int kMine = kTileGroups / Tr::kWriters;   // groups of a tile for each warp
      const int cw = warp - Tr::kConvert;
      const Keys &k = it.k;
      const int64_t row0 = it.r.row0;
      // A piece is two of a slot row's 16-byte chunks, so four lanes have 64 columns of one parity of
      // chunks; the other four of a group of eight take the next row, whose swizzle has the other
      // parity (and for d = 128 the other 64 columns, whose codes lie on the other banks).
      const int sub = lane % 8, up = sub / 4;
      const int row = Tr::kHalves == 2 ? lane / 16 * 2 + up : lane / 4;
      const int column = Tr::kHalves == 2 ? (up ^ (lane / 8 & 1)) * 64 : 0, col = column + sub % 4 * 16;
      const uint32_t at0 = (column / 64) * Tr::kHalfBytes + row * 128 + ((sub % 4 * 2) ^ (row & 7)) * 16;
      // Piece c of the lane into the group whose rows begin at `rows` in the slot.
      auto put = [&](unsigned char *rows, int c, uint4 lo, uint4 hi) {
        const uint32_t at = (at0 ^ (c * kRowStep & 7) * 16) + c * (kRowStep * 128);
        *reinterpret_cast<uint4 *>(rows + at) = lo;
        *reinterpret_cast<uint4 *>(rows + (at ^ 16)) = hi;
      };
      int item = 0;
      bool ok = true;
      for (int j = t_lo; j < t_hi && ok; ++j) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++item) {
          const int slot = item % kSlots, raw = item % kRaw;
          ok = wait(&sh.raw_full[raw], item / kRaw & 1) && wait(&sh.empty[slot], (item / kSlots & 1) ^ 1);
          if (!ok) break;
          const TileInfo &info = sh.info[(j - t_lo) % kInfos];
          bool odd = false;
          uint4 codes[kMine][kPieces];                       // (all on their way before the first store)
#pragma unroll
          for (int i = 0; i < kMine; ++i)
#pragma unroll
            for (int c = 0; c < kPieces; ++c)
              codes[i][c] = *reinterpret_cast<const uint4 *>(raw_ring + raw * Tr::kRawBytes + (kMine * cw + i) * (kPage * D) + (c * kRowStep + row) * D + col);
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int gi = kMine * cw + i, base = info.base[gi];
            const uint32_t flags = info.flags >> gi;
            unsigned char *rows = ring + slot * Tr::kSlotBytes + gi * (kPage * 128);
            if (flags & 0x100u) continue;
            if (kTree && (flags & 0x10000u)) {           // drafts are bf16 already
              const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(kv == 0 ? a.drafts.k_new : a.drafts.v_new) + static_cast<int64_t>(it.h) * D + col;
#pragma unroll 1
              for (int c = 0; c < kPieces; ++c) {
                const int draft = base + c * kRowStep + row;
                uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                if (draft < k.n_draft) {
                  const __nv_bfloat16 *at = src + (row0 + draft) * a.drafts.row_stride;
                  lo = ld_stream16(at);
                  hi = ld_stream16(at + 8);
                }
                odd |= kv == 1 && (any_odd_bf16(lo) || any_odd_bf16(hi));
                put(rows, c, lo, hi);
              }
              continue;
            }
            const float two_e = info.ve[gi];
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
              const uint4 w = codes[i][c];
              uint4 lo, hi;
              codes_to_bf16<kKv == 2>(w.x, kv == 1, two_e, lo.x, lo.y);
              codes_to_bf16<kKv == 2>(w.y, kv == 1, two_e, lo.z, lo.w);
              codes_to_bf16<kKv == 2>(w.z, kv == 1, two_e, hi.x, hi.y);
              codes_to_bf16<kKv == 2>(w.w, kv == 1, two_e, hi.z, hi.w);
              put(rows, c, lo, hi);
            }
            if ((flags & 1u) && kv == 1) odd |= !(fabsf(info.ve[gi]) < INFINITY);
            if (flags & 1u)                              // a group that rows see differently
#pragma unroll 1
              for (int c = 0; c < kPieces; ++c) {
                if (base + c * kRowStep + row >= k.T) {
                  put(rows, c, make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u));   // (zeros behind the last token)
                } else if (kKv == 1 && kv == 1) {        // E4M3's NaN: all seven bits
                  const uint4 w = *reinterpret_cast<const uint4 *>(raw_ring + raw * Tr::kRawBytes + gi * (kPage * D) + (c * kRowStep + row) * D + col);
                  auto nan = [](uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                  odd |= (nan(w.x) | nan(w.y) | nan(w.z) | nan(w.w)) != 0;
                }
              }
          }
          if (__any_sync(0xffffffffu, odd)) *const_cast<volatile int *>(&sh.marked) = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.raw_empty[raw]);
            mbar_arrive(full_of(j, kv));
            if (kv == 1 && j == t_hi - 1) mbar_arrive(full_of(j, kv));     // (there is no next K)
          }
        }
      }
    } else if (warp == Tr::kProduct) {
      // ---- product warp ------------------------------------------------------------------------
      constexpr uint32_t kShapeS = umma_shape(kKeyTile, false), kShapeO = umma_shape(D, true);
      const int n = t_hi - t_lo;
      const uint32_t lead = elect_lane();
      // Operands of the first slot and the first row tile; others lie at whole steps of the address field.
      const uint64_t q_op = umma_operand(smem_u32(q_smem), 16, 1024), k_op = umma_operand(smem_u32(ring), 16, 1024);
      const uint64_t v_op = umma_operand(smem_u32(ring), Tr::kHalfBytes, 1024);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t s_tm[2] = {tm, tm + 128}, o_tm[2] = {tm + 128 * kTiles, tm + 128 * kTiles + 128};
      auto logits = [&](int t, int slot) {      // S of row tile t
        const uint64_t kd = k_op + static_cast<uint32_t>(slot * (Tr::kSlotBytes / 16)), qd = q_op + static_cast<uint32_t>(t * (Tr::kQTile / 16));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk % 4) * (32 / 16);
          umma_ss(lead, s_tm[t], qd + (kk / 4) * (Tr::kQHalf / 16) + in, kd + (kk / 4) * (Tr::kHalfBytes / 16) + in, kShapeS, kk > 0);
        }
      };
      uint32_t started = 0;      // bit t: O of row tile t has been written
      bool ok = wait(&sh.q_full, 0) && wait(&sh.k0_full, 0);
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
        const int v_slot = (2 * j + 1) % kSlots, k_slot = (2 * j + 2) % kSlots;
        const uint64_t vd = v_op + static_cast<uint32_t>(v_slot * (Tr::kSlotBytes / 16));
        const TileInfo &info = sh.info[j % kInfos];     // (it came with the tile's K)
        const uint32_t flags = info.flags;
        const uint32_t pages = __reduce_or_sync(0xffffffffu, ~(flags >> 8) & 0xffu);
        ok = wait(&sh.full[j % kInfos], j / kInfos & 1);      // V, and K of the next tile
        if (!ok) break;
        if constexpr (!Tr::kQuant) {
          // rows of V past the cache's end or the drafts' hold anything: they become zero
          uint32_t differ = flags & ~(flags >> 8) & 0xffu;
          if (differ != 0) {
            for (uint32_t left = differ; left != 0; left &= left - 1) {
              const int i = __ffs(left) - 1, kept = kept_rows(info, i);
              unsigned char *at = ring + v_slot * Tr::kSlotBytes + i * (kPage * 128);
              for (int c = kept * 8 * Tr::kHalves + lane; c < kPage * 8 * Tr::kHalves; c += 32)
                *reinterpret_cast<uint4 *>(at + (c % Tr::kHalves) * Tr::kHalfBytes + c / Tr::kHalves * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            if constexpr (!Tr::kLooker) look(info, v_slot);
            __syncwarp();
          }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t >= live_tiles || !ok) break;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            ok = wait(&sh.p_full[t][part], j & 1);
            if (!ok) break;
            tmem_fence_after();
            constexpr int kFirst = kFirstKeys / kPage;
            const int lo = part * kFirst, hi = part == 0 ? kFirst : kTileGroups;
            const uint32_t all = (1u << hi) - (1u << lo), here = pages & all;
            if (here == all) {
#pragma unroll
              for (int i = lo; i < hi; ++i)
                umma_ts(lead, o_tm[t], s_tm[t] + i * 8, vd + static_cast<uint32_t>(i * (kPage * 128 / 16)), kShapeO,
                        i > lo || (started >> t & 1u));
              started |= 1u << t;
            } else {
#pragma unroll 1
              for (uint32_t left = here; left != 0; left &= left - 1) {
                const int i = __ffs(left) - 1;
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
    } else if (Tr::kLooker && warp == 3) {
      // ---- looks at V tiles beside the products; a slot is free when both are done with it ---------
      const int n = t_hi - t_lo;
      bool ok = wait(&sh.k0_full, 0);
      if (ok && lane == 0) mbar_arrive(&sh.empty[0]);
      for (int j = 0; j < n && ok; ++j) {
        ok = wait(&sh.full[j % kInfos], j / kInfos & 1);
        if (!ok) break;
        const int v_slot = (2 * j + 1) % kSlots;
        const TileInfo &info = sh.info[j % kInfos];
        if ((info.flags & ~(info.flags >> 8) & 0xffu) != 0) look(info, v_slot);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.empty[v_slot]);
          if (j + 1 < n) mbar_arrive(&sh.empty[(2 * j + 2) % kSlots]);
        }
      }
      if (ok && lane == 0) mbar_arrive(&sh.looked);
    } else if (warp >= Tr::kFirstRow && warp < Tr::kFirstRow + Tr::kRowWarps) {
      // ---- row warps -----------------------------------------------------------------------------
      const int t = (warp - Tr::kFirstRow) / Tr::kTileWarps;
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
        float used = 0.0f;                   // sum of the weights as they enter the products
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
            // Half a tile's logits are in registers at a time; the other half flies ahead of its use
            // where the registers are there (bf16: fewer warps, more of them each).
            constexpr bool kAhead = !Tr::kQuant;
            auto largest = [&](const float *x) -> float {      // of 16
              float top[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) top[c] = fmaxf(fmaxf(x[c], x[4 + c]), fmaxf(x[8 + c], x[12 + c]));
              return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)}, rounded = make_float2(0.0f, 0.0f);   // this tile's l, used
            if ((flags & 0xffffu) != 0) {
              // Logits of keys that the row does not see become -inf, in tensor memory: most tiles have
              // none, and their code keeps its registers.
#pragma unroll 1
              for (int c32 = 0; c32 < 4; ++c32) {
                float x[32];
                tmem_ld32(s_at + c32 * 32, x);
                uint32_t seen = 0;             // a bit a key
                float nan_or_1[2] = {1.0f, 1.0f};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int gi = c32 * 2 + y;
                  uint32_t bits = 0xffffu;
                  if ((flags >> gi | flags >> (8 + gi)) & 1u) {
                    const int base = info.base[gi];
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
                  }
                  seen |= (bits & 0xffffu) << (16 * y);
                  if (Tr::kQuant && info.ks[gi].x != info.ks[gi].x) nan_or_1[y] = info.ks[gi].x;   // (the weights' bound below drops it)
                }
                tmem_wait_ld<32>(x);
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) w[c] = seen >> c & 1u ? __float_as_uint(Tr::kQuant ? x[c] * nan_or_1[c / 16] : x[c]) : 0xff800000u;
                tmem_st16(s_at + c32 * 32, w);
                tmem_st16(s_at + c32 * 32 + 16, w + 16);
              }
              tmem_wait_st();
            }
            float first[64], ahead[kAhead ? 64 : 1];
            float *const second = kAhead ? ahead : first;
            auto read = [&](int half, float *to) {
              tmem_ld32(s_at + half * 64, to);
              tmem_ld32(s_at + half * 64 + 32, to + 32);
            };
            read(0, first);
            auto max_of = [&](int half, const float *x) -> float {
              float mx = -INFINITY;
#pragma unroll
              for (int gi = 0; gi < 4; ++gi) {
                float of = largest(x + gi * 16);
                // (8-bit: of weight times V's mantissa, which is what is rounded to bf16. A reference that is
                // the row's maximum then makes the largest of them 1, which rounds to itself: in a model rows
                // of 3 to 200 keys are 1.8 to 2.0e-3 off for 1.8 to 2.2e-3 with the logits' maximum. Costs 0.2 to 0.7 %.)
                if (Tr::kQuant && of != -INFINITY) of = fmaf(of, info.ks[half * 4 + gi].x, info.ks[half * 4 + gi].y);
                mx = fmaxf(mx, of);
              }
              return mx;
            };
            // Weights of keys [32 c32, + 32), over the first logits (8-bit: times V's mantissa, through
            // the exponent; both sums are of weights without it).
            auto weigh = [&](int c32, const float *x32) {
              const float base_m = m == -INFINITY ? 0.0f : -m * sc;
              uint32_t w[16];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int gi = c32 * 2 + y;
                // (a K scale of 0 must not make a NaN of -inf)
                const float to_log2 = Tr::kQuant ? fmaxf(info.ks[gi].x * sc, 1.17549435e-38f) : sc;
                const float from = Tr::kQuant ? fmaf(info.ks[gi].y, sc, base_m) : base_m;
                float2 exact = make_float2(0.0f, 0.0f);                // of the group (8-bit)
#pragma unroll
                for (int x = 8 * y; x < 8 * y + 8; ++x) {
                  const float2 z = __ffma2_rn(make_float2(x32[2 * x], x32[2 * x + 1]), make_float2(to_log2, to_log2), make_float2(from, from));
                  const float2 e = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                  if constexpr (Tr::kQuant) exact = __fadd2_rn(exact, e);
                  else sum[x & 1] = __fadd2_rn(sum[x & 1], e);
                  w[x] = pack_bf16(e.x, e.y);
                }
                if constexpr (Tr::kQuant) sum[0] = __ffma2_rn(exact, make_float2(info.inv_vs[gi], info.inv_vs[gi]), sum[0]);
              }
              tmem_st16(s_at + c32 * 16, w);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float2 taken = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int x = 8 * y; x < 8 * y + 8; ++x) {
                  if constexpr (Tr::kQuant) add_bf16x2(taken, w[x]);
                  else add_bf16x2(rounded, w[x]);
                }
                if constexpr (Tr::kQuant) rounded = __ffma2_rn(taken, make_float2(info.inv_vs[c32 * 2 + y], info.inv_vs[c32 * 2 + y]), rounded);
              }
            };
            auto hand_over = [&](int part) {
              tmem_wait_st();
              tmem_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.p_full[t][part]);
            };
            tmem_wait_ld<64>(first);
            if constexpr (kAhead) read(1, ahead);
            const float mx = fmaxf(max_of(0, first), pend);
            if (m == -INFINITY) m = mx;      // (nothing seen before: O's row is zero)
            // O's row, and l with it, relative to a new reference.
            auto rescale = [&](float to) {
              const float f = to == m ? 1.0f : exp2_approx((m - to) * sc);
              m = to;
              l *= f;
              used *= f;
              if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  float o[16];
                  tmem_ld16(o_at + c * 16, o);
                  tmem_wait_ld<16>(o);
                  uint32_t w[16];
#pragma unroll
                  for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * f);
                  tmem_st16(o_at + c * 16, w);
                }
              }
              return f;
            };
            const bool grow = valid && (mx - m) * sc > 8.0f;
            if (__any_sync(0xffffffffu, grow)) rescale(grow ? mx : m);
            weigh(0, first);
            weigh(1, first + 32);
            if constexpr (!kAhead) read(1, first);
            tmem_wait_ld<64>(second);
            pend = max_of(1, second);
            if (m == -INFINITY) m = pend;    // (the first half's weights are zero too)
            const bool far = valid && (pend - m) * sc > 30.0f;
            if (__any_sync(0xffffffffu, far)) {
              // the first half's weights are in tensor memory already
              const float f = rescale(far ? pend : m);
              sum[0] = __fmul2_rn(sum[0], make_float2(f, f));
              sum[1] = __fmul2_rn(sum[1], make_float2(f, f));
              rounded = __fmul2_rn(rounded, make_float2(f, f));
              tmem_wait_st();
#pragma unroll 1
              for (int c = 0; c < 2; ++c) {
                float p16[16];
                tmem_ld16(s_at + c * 16, p16);
                tmem_wait_ld<16>(p16);
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const uint32_t u = __float_as_uint(p16[x]);
                  w[x] = pack_bf16(bf16lo(u) * f, bf16hi(u) * f);
                }
                tmem_st16(s_at + c * 16, w);
              }
            }
            weigh(2, second);
            hand_over(0);
            weigh(3, second + 32);
            hand_over(1);
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            used += rounded.x + rounded.y;
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
          const float inv = l == 0.0f ? 0.0f : 1.0f / used;
          float odd[4] = {fabsf(l), 0.0f, 0.0f, 0.0f};     // NaN or infinite when the row's sums are
          const bool aligned = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0, rec_aligned = (reinterpret_cast<uintptr_t>(p.rec_o) & 31) == 0;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(o_at + c * 32, o);
            tmem_wait_ld<32>(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              if (l == 0.0f) o[x] = 0.0f;      // (a row that has seen nothing: no product may have written its O)
              odd[x % 4] = fmaf(0.0f, o[x], odd[x % 4]);
              o[x] *= inv;
            }
            if (valid) {
              if (last) {
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) w[x] = pack_bf16(o[2 * x], o[2 * x + 1]);
                __nv_bfloat16 *to = a.out + out_row * D + c * 32;
                store_sector(to, w, aligned);
                store_sector(to + 16, w + 8, aligned);
              } else {
                uint32_t w[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) w[x] = __float_as_uint(o[x]);
#pragma unroll
                for (int x = 0; x < 32; x += 8) store_sector(p.rec_o + rec * D + c * 32 + x, w + x, rec_aligned);
              }
            }
          }
          if (valid) {
            if (!last) p.rec_ml[rec] = make_float2(m_log2, l);
            else if (a.lse != nullptr) a.lse[out_row] = l == 0.0f ? -INFINITY : (m_log2 + log2f(l)) * kLn2;
          }
          // A marked block: columns that are not finite, row by row, by the whole warp. (Sums of weights
          // have no unseen key in them: where they are not finite, neither is the row.)
          if ((!Tr::kLooker || wait(&sh.looked, 0)) && *const_cast<volatile int *>(&sh.marked) != 0) {
            const bool sums = fabsf(l) < INFINITY;
            unsigned again = __ballot_sync(0xffffffffu, valid && sums && !((odd[0] + odd[1]) + (odd[2] + odd[3]) < INFINITY));
            __syncwarp();                      // (the lanes' rows are written)
            while (again != 0) {
              const int src = __ffs(again) - 1;
              again &= again - 1;
              const int ri = __shfl_sync(0xffffffffu, i, src), rg = __shfl_sync(0xffffffffu, gq, src);
              const int64_t r_out = __shfl_sync(0xffffffffu, out_row, src), r_rec = __shfl_sync(0xffffffffu, rec, src);
              const float r_m = __shfl_sync(0xffffffffu, m_log2, src), r_inv = __shfl_sync(0xffffffffu, inv, src);
              __nv_bfloat16 *to = a.out + r_out * D + lane * (D / 32);
              float *to_rec = p.rec_o + r_rec * D + lane * (D / 32);
              uint32_t bad = 0;
#pragma unroll
              for (int e = 0; e < D / 32; ++e)
                if (!(fabsf(last ? __bfloat162float(to[e]) : to_rec[e]) < INFINITY)) bad |= 1u << e;
              float rm, ro[D / 32];
              row_columns<D, kTree>(a, it.r, k, it.h, ri, rg, t_lo * kTileGroups, min(t_hi * kTileGroups, k.n_groups), bad, rm, ro);
#pragma unroll
              for (int e = 0; e < D / 32; ++e)
                if (bad >> e & 1u) {
                  const float x = ro[e] * exp2f(rm - r_m) * r_inv;
                  if (last) to[e] = __float2bfloat16_rn(x);
                  else to_rec[e] = x;
                }
            }
          }
        }
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == Tr::kProduct) {
    // (After a wait that ran out, copies and products in flight, which take microseconds, end before
    // the CTA gives its memory back.)
    if (sh.failed != 0) mbar_wait_bounded(&sh.never, 0, a.st, kInFlightNs);
    tmem_fence_after();
    tmem_free(tmem, Tr::kColumns);
  }
}

template <int D, int kKv, int kRows, bool kTree>
bs_status launch_rows_mma(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, cudaStream_t cs) {
  using Tr = RowsTraits<D, kKv, kRows>;
  auto kernel = rows_mma_kernel<D, kKv, kRows, kTree>;
  static OncePerDevice attrs;
  if (!attrs([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Tr::kSmem) == cudaSuccess; }))
    return BS_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(p.even > 0 ? p.even : p.items * p.splits));
  return launch_ex(kernel, grid, Tr::kThreads, Tr::kSmem, cs, 0, true, a, p, maps) == cudaSuccess ? BS_OK : BS_ERR_CUDA;
}

// By the rows of a CTA (32, 128 or 256) and the cache's type; each in a file of its own.
template <bool kTree>
bs_status launch_rows_bf16(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs);
template <bool kTree>
bs_status launch_rows_quant(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs);

template <int D, int kKv, bool kTree>
bs_status dispatch_rows(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs) {
  switch (rows) {
    case 32: return launch_rows_mma<D, kKv, 32, kTree>(a, p, maps, cs);
    case 128: return launch_rows_mma<D, kKv, 128, kTree>(a, p, maps, cs);
    default: return launch_rows_mma<D, kKv, 256, kTree>(a, p, maps, cs);
  }
}
template <int kKv, bool kTree>
bs_status dispatch_rows(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs) {
  return a.dims.head_dim == 128 ? dispatch_rows<128, kKv, kTree>(a, p, maps, rows, cs) : dispatch_rows<64, kKv, kTree>(a, p, maps, rows, cs);
}

}  // namespace bsi
