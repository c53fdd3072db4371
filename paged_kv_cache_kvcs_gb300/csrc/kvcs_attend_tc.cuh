// kvcs_attend_tc.cuh -- attention of a chunk of new tokens over a paged cache
// on the tensor-memory tensor cores (heads of 64 or 128; 16-bit caches, in extended
// views 8-bit ones as well).
//
// Mathematics as in kvcs_attend.cuh.  Bound: 4 * head_dim operations per
// visible (row, token) pair, far above the bytes, so the tensor cores are the
// floor, and next to them the exponentials (one per pair).
//
// A unit is 256 query rows (new tokens x the KV head's query group, so that
// the group shares every K and V tile) in two tiles of 128, against tiles of
// 128 tokens.  Roles of the CTA's warps:
//   warps 9, 11  load K and V tiles page by page with TMA (boxes of as many
//              slots as a page holds in a row, 128-byte swizzle) into a ring;
//   warps 8, 10  issue the products of one query tile each: S_i = Q_i K^T into
//              tensor memory, then O_i += P_i V with P_i from tensor memory;
//   warps 0-3, warps 4-7   the softmax of one query tile each, a thread per
//              row: S from tensor memory, weights back over S as 16-bit P.
// The two tiles take turns: while one tile's weights are made, the other
// tile's products run.  One warp's products run in issue order, so P_i is read
// before S_i of the next token tile overwrites it, and the signal that S_i is
// ready also says that O_i's last addition is done.
//
// The running maximum is only raised when a row's scores pass it by more than
// 2^8: weights then stay below 2^8 (2^15 in fp16, which starts 2^7 higher) and
// nothing has to be rescaled for most tiles; when a row does pass, its thread
// rescales its row of O in tensor memory itself (the additions to it are done
// by then).
//
// A weight of 0 times a NaN or infinite V value would be NaN.  V rows of slots
// that hold no token are therefore zeroed in shared memory, and in tiles that
// some row sees only in part, rows with a non-finite value are zeroed and
// noted; the rows that do see them add them at the end.
//
// Measured (4 requests of 2048 new tokens over 8192, 32 query heads to 8 KV
// heads of 128, bf16): 669 us, 1437 TFLOP/s, 77% of the measured burst rate of
// a library product and 86% of its sustained rate.  With the weights left out
// the products and loads alone take 510 us.  What it grew from and what was
// left again, for the same call: mma.sync 6300; one issuing thread for both
// query tiles 1027; loads of 64-element halves, one warp for K and V 918 with
// no weights at all; an issuing thread per tile, without turns, 863; four
// softmax warps a scheduler with 16 rows a warp (two threads of a quad sharing
// 64 columns) 926; a maximum found in the same pass as both halves' weights 706.
//
// Extended views.  A unit's tiles are the sinks', then the window's; which tokens a
// row sees comes from its RowSight, a word of 32 tokens at a time, in the tiles that
// some row sees only in part: of a tree those of its new tokens and of the windows'
// ends.  The trees' masks are made by the kernel before, which this one overlaps
// until it reads them.  4 requests of 2048 new tokens over 8192 under a window of
// 2048, 64 first tokens kept (the same heads): 279 us, 1016 TFLOP/s, 54% of the
// measured burst rate; what it leaves are 10 us from a unit's last product to the next
// one's first, of 17 tiles and 1.8 us each.  Trees of 16 tokens of 64 requests over
// 512 to 4096: 176 us, 3.5 TB/s: units of one query tile, so that neither tile's
// products hide the other's weights (1.4 us a tile where the bytes would take 0.75).
// Tried for those and not kept: two streams of 128 rows a CTA, with rings of their own
// and runs of one line, 157 (of 64 rows, joined in place, 165), but one of 32,768
// tokens 73 instead of 48, 7 drafted tokens over 709 29 instead of 21; the line of
// tiles cut into equal runs of one query tile pair 195.
//
// Caches of bytes, with or without scales.  The tensor cores multiply the values that
// are stored, as bfloat16, which holds each of them exactly: four warps read the
// bytes, and write the K and V tiles that TMA brings of 16-bit caches.  A token's score
// is multiplied by its K scale, its weight by its V scale before it is rounded to
// bfloat16, which has the range for it; l counts the weights without it.  Rows of S are
// taken 64 tokens at a time, once for their maximum and once for the weights, so that
// four warpgroups have registers enough.  A token with a scale or value that is not
// finite, where some row may not see it, is taken out and noted, as above.
// Chunks of 2048 of 4 requests over 8192: int8 1643 us, e4m3 1827 (585 and 527 TFLOP/s
// over the (row, token) pairs that are seen; 16-bit values 621 us beside them, 1550;
// kvcs_attend_cols.cuh's kernel 6319 and 6361 us).
// What bounds it is the conversion, 32,768 values a tile with some five instructions
// for two of them (without it 1165), then the weights (without both 527).  As four
// warps for K and four for V over copies in shared memory, which leave room for three
// tiles of 16 bits instead of four, 1856 and 2012; NaN bytes looked at where values are
// written, 2127; with everything unrolled the instructions no longer fit their cache.
#pragma once

#include "kvcs_attend_cols.cuh"
#include "kvcs_tcgen.cuh"

namespace kvcs {

// Three warpgroups (the third: loads and products).  Launched
// with 168 registers a thread, 64512 in all; the softmax warpgroups take 208
// (a row of S is 128 of them), the third keeps 88: 2 * 208 + 88 = 3 * 168.
constexpr int kTcThreads = 384;
constexpr int kTcRegsSoftmax = 208;
constexpr int kTcRegsOther = 88;
// Caches of bytes: a fourth one makes 16-bit tiles of them.  512 threads of 128: the
// softmax takes 144, the products' keep 64 and the converting one takes 160:
// 2 * 144 + 64 + 160 = 4 * 128.
constexpr int kTcBytesThreads = 512;
constexpr int kTcBytesRegsSoftmax = 144, kTcBytesRegsProducts = 64, kTcBytesRegsConvert = 160;
template <int kType>
constexpr int kTcThreadsOf = kIs8Bit<kType> ? kTcBytesThreads : kTcThreads;
constexpr int kTcRows = 256;      // query rows of a unit
constexpr int kTcKeys = 128;      // tokens of a tile
constexpr int kTcMaxSplits = 16;  // parts of a unit's token range, at most
constexpr float kTcSlack = 8.0f;  // log2 of what scores pass the running maximum by, unscaled
// As kLift: with the slack the largest weight is 2^15, and weights vanish below
// 2^-32 of the row's largest.
template <bool kBf16>
constexpr float kTcLift = kBf16 ? 0.0f : 7.0f;
// Partly seen tiles of a unit, at most: those of 256 tokens' own and windows'
// ends, or a tree's 1024 and the window's ends of their depths, and the sinks'.
constexpr int kTcDirty = 24;

template <int kDim, bool kBytes = false>
struct TcShape {
  static constexpr int kHalves = kDim / 64;               // 128-byte column halves
  // Q tile: [half][128 rows][128 bytes]; K and V tiles, as their boxes arrive:
  // [8 rows][half][128 bytes each], the groups of 8 rows one after another
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // Q, K or V tile
  static constexpr int kStages = (kBytes ? 4 : 5) * (128 / kDim);
  // caches of bytes: the scales of some tiles, K's and V's
  static constexpr int kScaleTiles = kBytes ? kStages : 0;
  static_assert(kScaleTiles <= 8, "TcShared has as many barriers");
  static constexpr int kScaleBytes = kScaleTiles * 2 * kTcKeys * 4;
  static constexpr int kSmemBytes = (2 + kStages) * kTileBytes + kScaleBytes + 1024;
  static constexpr int kPartFloats = kDim + 4;   // o, m, l of a row, on 16-byte boundaries
};

struct TcParams {
  AttnParams a;
  int box;        // slots a TMA box takes
  int heads_in_groups;   // HND: the maps' groups of 8 slots run through the heads
  int splits;     // parts of the token range per unit
  long long most_units;  // units that sound tables can have: partial results
                         // are there for no more
  u64 timeout_ns;
};

// A unit as every role sees it.
struct TcUnit {
  Request q;
  int head, row0, rows_all;
  int tiles;          // query tiles with rows: 1 or 2
  int k0, k1;         // token tiles of this part
  int lo, hi;         // tokens some row sees: [lo, hi)
  int sinks;          // extended views: token tiles before the window's, of [0, sink_keys)
  int skip;           // tiles between the sinks' and the window's
  int sink_keys;
  int split;
  long long index;    // unit number (of the join)
};

// Token tile of a unit's tile k: extended views count the sinks' tiles first,
// then the window's.
template <bool kExt>
__device__ __forceinline__ int tile_of(const TcUnit &x, int k) {
  return kExt && k >= x.sinks ? k + x.skip : k;
}

// Finds units in growing order; every lane of a warp calls it together.
struct TcFinder {
  long long chunk = 0, before = 0;   // requests [chunk, chunk + 32) start at tile `before`

  template <bool kExt>
  __device__ __forceinline__ TcUnit find(const TcParams &p, long long u) {
    const AttnParams &a = p.a;
    const int lane = threadIdx.x & 31;
    TcUnit x;
    x.split = static_cast<int>(u % p.splits);
    x.index = u / p.splits;
    x.head = static_cast<int>(x.index % a.kv_heads);
    const long long tile = x.index / a.kv_heads;
    for (;;) {
      const long long r = chunk + lane;
      Request q;
      q.n = 0;
      if (r < a.tab.num_requests) q = read_request(a.tab, r, a.map.block_size, false);
      const long long rows = static_cast<long long>(q.n) * a.group;
      const int tiles = rows < a.row_lo || rows > a.row_hi
                            ? 0 : static_cast<int>((rows + kTcRows - 1) / kTcRows);
      int inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const int all = __shfl_sync(0xffffffffu, inc, 31);
      if (tile < before + all) {
        const int at = static_cast<int>(tile - before);
        const int src = __ffs(__ballot_sync(0xffffffffu, inc > at)) - 1;
        const int first = __shfl_sync(0xffffffffu, inc - tiles, src);
        const int n_tiles = __shfl_sync(0xffffffffu, tiles, src);
        x.q.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
        x.q.q0 = __shfl_sync(0xffffffffu, q.q0, src);
        x.q.n = __shfl_sync(0xffffffffu, q.n, src);
        x.q.keys = __shfl_sync(0xffffffffu, q.keys, src);
        x.q.at = __shfl_sync(0xffffffffu, q.at, src);
        x.q.base = kExt ? __shfl_sync(0xffffffffu, q.base, src) : 0;
        // the rows that see most tokens first
        x.row0 = (n_tiles - 1 - (at - first)) * kTcRows;
        break;
      }
      before += all;
      chunk += 32;
      if (chunk >= a.tab.num_requests) {   // beyond the last unit
        x.tiles = 0;
        return x;
      }
    }
    x.rows_all = x.q.n * a.group;
    x.tiles = x.rows_all - x.row0 > 128 ? 2 : 1;
    const int last_row = min(x.row0 + kTcRows, x.rows_all) - 1;
    const int at0 = x.q.at + x.row0 / a.group, at1 = x.q.at + last_row / a.group;
    x.lo = a.window > 0 ? max(0, at0 - a.window + 1) : 0;
    x.hi = max(0, min(x.q.keys, at1 + 1));
    if constexpr (kExt) {
      // (a tree's rows: their tokens' depths start at 0)
      if (a.place && a.window > 0) x.lo = max(0, x.q.at - a.window + 1);
      x.sink_keys = min(sink_keys_of(a, x.q), x.hi);
    }
    const int t0 = x.lo / kTcKeys;
    int t1 = x.hi > x.lo ? (x.hi + kTcKeys - 1) / kTcKeys : t0;
    if constexpr (kExt) {
      // (listed tokens may end before the window: the sinks are seen all the same)
      const int sinks = (x.sink_keys + kTcKeys - 1) / kTcKeys;
      x.sinks = min(t0, sinks);
      t1 = max(t1, sinks);
      x.skip = t0 - x.sinks;
      const int n = x.sinks + t1 - t0, per = (n + p.splits - 1) / p.splits;
      x.k0 = min(n, x.split * per);
      x.k1 = min(n, x.k0 + per);
    } else {
      const int per = (t1 - t0 + p.splits - 1) / p.splits;
      x.k0 = min(t1, t0 + x.split * per);
      x.k1 = min(t1, x.k0 + per);
    }
    return x;
  }
};

struct TcShared {
  u64 full[10], empty[10];
  u64 q_full[2], s_full[2], p_half[2], p_ready[2], o_full[2];
  u64 turns[2];                    // the products' warps hand each other the turn
  u64 fix, loaded, released;
  u64 scales[8];                   // caches of bytes: a tile's scales are there
  u64 drain[2];                    // a product warp's last products
  u32 tmem;
  int n_dirty[2];                  // noted tiles, by parity of the unit
  int dirty_tile[2][kTcDirty];
  u32 dirty[2][kTcDirty][4];
};

// Caches of bytes: what each converting warp noted of its 32 tokens of a tile.
template <bool kBytes>
struct TcNotes {
  int n[2][4];                     // by parity of the unit
  int key[2][4][kTcDirty];         // the first of the 32
  u32 bits[2][4][kTcDirty];
};
template <>
struct TcNotes<false> {};

// Whether token `key` (below the request's count) lies in a block of the pool.
__device__ __forceinline__ bool good_block(const AttnParams &a, const Request &q, int key) {
  const int b = a.tab.block_ids[q.pos0 + a.map.by_block(key)];
  return b >= 0 && b < a.map.num_blocks;
}

// Whether some block of the tokens that a unit's part needs is bad (a warp).
template <bool kExt>
__device__ __forceinline__ bool bad_blocks(const AttnParams &a, const TcUnit &x) {
  const int bs = a.map.block_size;
  int lo = max(x.k0 * kTcKeys, x.lo), hi = min(x.k1 * kTcKeys, x.hi);
  if constexpr (kExt) {
    lo = max((max(x.k0, x.sinks) + x.skip) * kTcKeys, x.lo);
    hi = x.k1 > x.sinks ? min((x.k1 + x.skip) * kTcKeys, x.hi) : 0;
  }
  bool bad = false;
  for (int b = lo / bs + (threadIdx.x & 31); b * static_cast<long long>(bs) < hi; b += 32) {
    const int id = a.tab.block_ids[x.q.pos0 + b];
    bad |= id < 0 || id >= a.map.num_blocks;
  }
  if constexpr (kExt) {   // (the sinks may reach into the window's first tile)
    hi = min(x.k1 * kTcKeys, min(x.sink_keys, x.lo));
    for (int b = x.k0 * kTcKeys / bs + (threadIdx.x & 31); b * static_cast<long long>(bs) < hi; b += 32) {
      const int id = a.tab.block_ids[x.q.pos0 + b];
      bad |= id < 0 || id >= a.map.num_blocks;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

__device__ __forceinline__ float lo_of(u32 w, bool bf16) { return half_bits_to_float(w & 0xffffu, bf16); }
__device__ __forceinline__ float hi_of(u32 w, bool bf16) { return half_bits_to_float(w >> 16, bf16); }

// Four bytes of a cache as 16-bit values, two by two; exact: int8 as 128 + its low
// seven bits, less 128 or (negative ones) 256; e4m3 as the bfloat16 of the same
// bits, its exponent off by 120.
template <int kType>
__device__ __forceinline__ void bytes_to_bf16(u32 v, u32 &lo, u32 &hi) {
  if constexpr (kType == kKvInt8Scaled) {
    const u32 x = __byte_perm(v, 0, 0x4140), y = __byte_perm(v, 0, 0x4342);
    const u32 xa = (x & 0x007f007fu) | 0x43004300u, xb = (x & 0x00800080u) | 0x43004300u;
    const u32 ya = (y & 0x007f007fu) | 0x43004300u, yb = (y & 0x00800080u) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(xa), "r"(xb));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(ya), "r"(yb));
  } else {
    const u32 x = __byte_perm(v, 0, 0x1404), y = __byte_perm(v, 0, 0x3424);
    const u32 xa = (x & 0x80008000u) | (x >> 4 & 0x07f007f0u);
    const u32 ya = (y & 0x80008000u) | (y >> 4 & 0x07f007f0u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(xa), "r"(0x7b807b80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(ya), "r"(0x7b807b80u));
  }
}
// Bit 7 of each e4m3 byte that is a NaN (all bits but the sign).
__device__ __forceinline__ u32 nan_bytes(u32 v) {
  return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// 16 tokens of K or V (half) of a cache of bytes, as pieces of 16 bytes: lane's are
// piece lane % kAcross of rows lane / kAcross + kDown t; and lane's token's scale
// (lane % 16).  Any chunk: tokens outside [lo, hi) but for those below sink_keys, and
// tokens of bad blocks, become zeros.  Returns the mask of those that are there.
template <int kType, int kDim>
__device__ __noinline__ u32 load_half_any(const AttnParams &a, const TcUnit &x, int half, int key0,
                                          uint4 *v, float *scale) {
  using L = ChunkLanes<kType, kDim>;
  const int lane = threadIdx.x & 31, key = key0 + (lane & 15);
  bool ok = (key >= x.lo || key < x.sink_keys) && key < x.hi;
  long long off = 0;
  *scale = 0.0f;
  if (ok) {
    const int pos = a.map.by_block(key), slot = key - pos * a.map.block_size;
    const int id = a.tab.block_ids[x.q.pos0 + pos];
    if (id < 0 || id >= a.map.num_blocks) {
      ok = false;
      raise(a.tab, kStatusBadBlockId);
    } else {
      off = token_offset(a.map, id, slot, x.head) + half * a.map.half_stride;
      if constexpr (kIsScaled<kType>)
        *scale = (half ? a.v_scales : a.k_scales)[(static_cast<long long>(id) * a.kv_heads + x.head) *
                                                      a.map.block_size + slot];
    }
  }
  const u32 mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
#pragma unroll 1
  for (int t = 0; t < L::kTurns; ++t) {
    const int row = t * L::kDown + lane / L::kAcross;
    const unsigned char *src = a.map.base + __shfl_sync(0xffffffffu, off, row) +
                               (lane % L::kAcross) * static_cast<long long>(a.map.chunk_stride);
    uint4 y = make_uint4(0, 0, 0, 0);
    if (mask >> row & 1u) {
      if (!a.unit8) {
        y = *reinterpret_cast<const uint4 *>(src);
      } else {
        const uint2 lo = *reinterpret_cast<const uint2 *>(src), hi = *(reinterpret_cast<const uint2 *>(src) + 1);
        y = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
    v[t] = y;
  }
  return mask;
}

// Writes them into their tile as 16-bit values; returns the rows with a value that
// is not finite, where `partly` (they are taken out).
template <int kType, int kDim, bool kNans>
__device__ __forceinline__ u32 store_half_as(const uint4 (&v)[ChunkLanes<kType, kDim>::kTurns], u32 to,
                                             bool partly) {
  using S = TcShape<kDim, true>;
  using L = ChunkLanes<kType, kDim>;
  const int lane = threadIdx.x & 31, piece = lane % L::kAcross;
  u32 odd_rows = 0;
#pragma unroll
  for (int t = 0; t < L::kTurns; ++t) {
    const int row = t * L::kDown + lane / L::kAcross;
    const u32 w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
    u32 o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) bytes_to_bf16<kType>(w[e], o[2 * e], o[2 * e + 1]);
    if constexpr (kNans) {
      u32 m[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = nan_bytes(w[e]);
        o[2 * e] |= (__byte_perm(m[e], 0, 0x1404) >> 15 & 0x00010001u) * 0x7fc0u;
        o[2 * e + 1] |= (__byte_perm(m[e], 0, 0x3424) >> 15 & 0x00010001u) * 0x7fc0u;
      }
      if (partly) {
        const u32 lanes = __ballot_sync(0xffffffffu, m[0] | m[1] | m[2] | m[3]);
        constexpr u32 kRow = (1u << L::kAcross) - 1u;
#pragma unroll
        for (int r = 0; r < L::kDown; ++r)
          if (lanes >> r * L::kAcross & kRow) odd_rows |= 1u << (t * L::kDown + r);
        if (odd_rows >> row & 1u) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0;
        }
      }
    }
    // (half of a row's eight lanes write their second unit first: all banks)
    const u32 at = to + (piece >> 2) * 1024 + (row >> 3) * (S::kHalves * 1024) + (row & 7) * 128 +
                   ((((piece & 3) * 2) ^ (row & 7)) << 4);
    const bool swap = piece >= 4;
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(swap ? at ^ 16 : at),
                 "r"(swap ? o[4] : o[0]), "r"(swap ? o[5] : o[1]), "r"(swap ? o[6] : o[2]),
                 "r"(swap ? o[7] : o[3])
                 : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(swap ? at : at ^ 16),
                 "r"(swap ? o[0] : o[4]), "r"(swap ? o[1] : o[5]), "r"(swap ? o[2] : o[6]),
                 "r"(swap ? o[3] : o[7])
                 : "memory");
  }
  return odd_rows;
}
template <int kType, int kDim>   // (out of the way: the loop's code stays small)
__device__ __noinline__ u32 store_half_nans(const uint4 *v, u32 to, bool partly) {
  uint4 y[ChunkLanes<kType, kDim>::kTurns];
#pragma unroll
  for (int t = 0; t < ChunkLanes<kType, kDim>::kTurns; ++t) y[t] = v[t];
  return store_half_as<kType, kDim, true>(y, to, partly);
}
template <int kType, int kDim>
__device__ __forceinline__ u32 store_half(const uint4 (&v)[ChunkLanes<kType, kDim>::kTurns], u32 to, bool partly) {
  if constexpr (kType != kKvInt8Scaled) {
    constexpr int kTurns = ChunkLanes<kType, kDim>::kTurns;
    u32 odd = 0;
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
      odd |= nan_bytes(v[t].x) | nan_bytes(v[t].y) | nan_bytes(v[t].z) | nan_bytes(v[t].w);
    if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
      uint4 y[kTurns];
#pragma unroll
      for (int t = 0; t < kTurns; ++t) y[t] = v[t];
      return store_half_nans<kType, kDim>(y, to, partly);
    }
  }
  return store_half_as<kType, kDim, false>(v, to, partly);
}

// The converting warps of a CTA over a cache of bytes: each has 32 tokens of a tile,
// in two chunks of K and of V that it holds in registers a tile ahead and then
// writes as 16-bit values.  false: a wait ran out.
template <int kType, int kDim>
__device__ __forceinline__ bool tc_convert(const TcParams &p, TcShared &sh, TcNotes<true> &notes, u32 ring,
                                           long long units) {
  using S = TcShape<kDim, true>;
  using L = ChunkLanes<kType, kDim>;
  const AttnParams &a = p.a;
  const int lane = threadIdx.x & 31, cw = (threadIdx.x >> 5) & 3;
  const u32 scales = ring + S::kStages * S::kTileBytes;
  const u32 full = ptx::smem_addr(sh.full), empty = ptx::smem_addr(sh.empty);
  const u64 limit = p.timeout_ns;
  bool ok = true;
  TcFinder finder;
  u32 tile = 0;               // tiles so far
  long long n_unit = 0;
  for (long long u = blockIdx.x; u < units && ok; u += gridDim.x, ++n_unit) {
    const TcUnit x = finder.find<true>(p, u);
    const int par = n_unit & 1;
    int at0 = x.q.at + x.row0 / a.group;
    const int at1 = x.q.at + (min(x.row0 + kTcRows, x.rows_all) - 1) / a.group;
    if (a.place && x.rows_all > 0) at0 = a.place[x.q.q0] < 0 ? -(1 << 30) : x.q.at - 1;
    const int *ids = a.tab.block_ids + x.q.pos0;
    const unsigned char *src = a.map.base + x.head * a.map.head_stride +
                               (lane / L::kAcross) * static_cast<long long>(a.map.slot_stride) +
                               (lane % L::kAcross) * static_cast<long long>(a.map.chunk_stride);
    auto key_of = [&](int k, int c) { return tile_of<true>(x, k) * kTcKeys + (2 * cw + c) * kChunkKeys; };
    // the block of a chunk whose tokens are all needed and lie in a row, read a tile ahead
    auto block_of = [&](int k, int c) {
      if (k >= x.k1 || !a.runs) return -1;
      const int key = key_of(k, c);
      if ((key < x.lo && key + kChunkKeys > x.sink_keys) || key + kChunkKeys > x.hi) return -1;
      return ids[a.map.by_block(key)];
    };
    uint4 v[2][2][L::kTurns];   // of K and V, by chunk
    float scale[2][2];
    u32 masks = 0;   // 16 bits a chunk: tokens that are there
    int ahead[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) ahead[c] = block_of(x.k0, c);
    auto load = [&](int half, int k, int c) {
      if (k >= x.k1) return;
      const int block = ahead[c], key = key_of(k, c);
      if (half) ahead[c] = block_of(k + 1, c);
      u32 mask = 0xffffu;
      if (__builtin_expect(block >= 0 && block < a.map.num_blocks, 1)) {
        const int slot = key - a.map.by_block(key) * a.map.block_size, sub = a.map.by_sub(slot);
        const unsigned char *from = src + block * a.map.block_stride + sub * a.map.sub_stride +
                                    (slot - sub * a.map.kbs) * static_cast<long long>(a.map.slot_stride) +
                                    half * a.map.half_stride;
#pragma unroll
        for (int t = 0; t < L::kTurns; ++t) {
          v[half][c][t] = __ldg(reinterpret_cast<const uint4 *>(from));
          from += L::kDown * static_cast<long long>(a.map.slot_stride);
        }
        if constexpr (kIsScaled<kType>)
          scale[half][c] = __ldg((half ? a.v_scales : a.k_scales) +
                                 (static_cast<long long>(block) * a.kv_heads + x.head) * a.map.block_size +
                                 slot + (lane & 15));
      } else {
        uint4 any[L::kTurns];
        float any_scale;
        mask = load_half_any<kType, kDim>(a, x, half, key, any, &any_scale);
#pragma unroll
        for (int t = 0; t < L::kTurns; ++t) v[half][c][t] = any[t];
        scale[half][c] = any_scale;
      }
      if (half) masks = (masks & (c ? 0xffffu : 0xffff0000u)) | mask << 16 * c;
    };
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int c = 0; c < 2; ++c) load(half, x.k0, c);
    int n_notes = 0;
    for (int k = x.k0; k < x.k1; ++k, ++tile) {
      const int key0 = tile_of<true>(x, k) * kTcKeys;
      u32 noted = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const u32 item = 2 * tile + half, stage = item % S::kStages, turn = item / S::kStages;
        if (turn > 0) ok = ok && tc::wait(empty + 8 * stage, (turn - 1) & 1, limit);
        if (!ok) break;
        // tiles some row sees only in part: what is not finite in V is taken out and noted
        const bool partly = half && (key0 + kTcKeys - 1 > at0 ||
                                     (a.window > 0 && key0 <= at1 - a.window &&
                                      key0 + kTcKeys > x.sink_keys));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int chunk = 2 * cw + c;   // of the tile
          u32 odd_rows = 0;
          if constexpr (kIsScaled<kType>) {
            float f = scale[half][c];
            const bool odd = partly && lane < 16 && !(fabsf(f) < __builtin_huge_valf());
            f = odd ? 0.0f : finite_or_nan(f);
            if (half) odd_rows = __ballot_sync(0xffffffffu, odd);
            if (lane < 16)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + tile % S::kScaleTiles * (8 * kTcKeys) +
                                                           (half * kTcKeys + chunk * kChunkKeys + lane) * 4),
                           "f"(f)
                           : "memory");
          }
          odd_rows |= store_half<kType, kDim>(
              v[half][c], ring + stage * S::kTileBytes + chunk * (2 * S::kHalves * 1024), partly);
          noted |= (odd_rows & masks >> 16 * c & 0xffffu) << 16 * c;
          load(half, k + 1, c);
        }
        tc::fence_async();
        __syncwarp();
        if (lane == 0) {
          if (kIsScaled<kType>) ptx::mbar_arrive(ptx::smem_addr(sh.scales) + 8 * (tile % S::kScaleTiles));
          ptx::mbar_arrive(full + 8 * stage);
        }
      }
      if (!ok) break;
      if (noted && n_notes < kTcDirty) {
        if (lane == 0) {
          notes.key[par][cw][n_notes] = key0 + 32 * cw;
          notes.bits[par][cw][n_notes] = noted;
        }
        ++n_notes;
      }
    }
    if (lane == 0) notes.n[par][cw] = n_notes;
    // one unit ahead of the softmax at most: its notes are kept twice
    if (ok && n_unit > 0) ok = tc::wait(ptx::smem_addr(&sh.released), (n_unit - 1) & 1, limit);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.loaded));
  }
  return ok;
}

// A value of a row (K or V of a token) of a cache of bytes.
template <int kType>
__device__ __noinline__ float byte_value(const unsigned char *row, int col, u32 chunk_stride) {
  u32 lo, up;
  bytes_to_half<kType>(row[static_cast<long long>(col >> 4) * chunk_stride + (col & 15)], lo, up);
  return half_bits_to_float(lo & 0xffffu, false);
}
// The weight of a noted token of a cache of bytes, by its V scale.
template <int kType, int kDim>
__device__ __noinline__ float noted_weight(const AttnParams &a, int block, int slot, int head,
                                           const unsigned char *q_row, float m) {
  const unsigned char *kp = a.map.base + token_offset(a.map, block, slot, head);
  float dot = 0.0f, vs = 1.0f;
  for (int e = 0; e < kDim; ++e)
    dot += byte_value<kType>(kp, e, a.map.chunk_stride) *
           half_bits_to_float(reinterpret_cast<const unsigned short *>(q_row)[e], true);
  if constexpr (kIsScaled<kType>) {
    const long long at = (static_cast<long long>(block) * a.kv_heads + head) * a.map.block_size + slot;
    dot *= finite_or_nan(a.k_scales[at]);
    vs = finite_or_nan(a.v_scales[at]);
  }
  return ex2(score_of(a, dot, 1.0f) - m) * vs;
}

// How a kernel makes scores of products: kPlain by a positive scale alone (on
// the way to the weights), kCapped with a cap, or by any scale, and kFarCapped
// with a cap past kNearCap.  (Both kinds of caps in one kernel: 1398 us, not
// 1260, for the chunk below.)
constexpr int kPlain = 0, kCapped = 1, kFarCapped = 2;
inline int scores_kind(const AttnParams &a) {
  return a.cap > kNearCap ? kFarCapped : a.cap != 0.0f || !(a.scale > 0.0f) ? kCapped : kPlain;
}

// A thread's raw products as scores in units of log 2, in place.  whole: its
// row sees all of them (its token is seen by all of their rows).
//
// Capped ones: tanh from its exponential is two operations of the exponential
// unit a score and six others.  The polynomial is ten operations on pairs (off
// by 1.3 * 2^-23 of the cap at most, with its roundings); it is taken in whole
// tiles until one of the thread's products has passed the cap (`past`).  So the
// form hangs on places, and on what is seen by the thread's row, alone: the two
// differ in the last bits, and nothing else may show in a row.  (A vote of the
// warp over all products let the slots behind the last token and the tiles'
// leftovers choose.)
// 4 requests of 2048 new tokens over 8192 (32 query heads to 8 KV heads of 128,
// bf16): 628 us without a cap, 1260 with one of 30 (none passes it), 1510 with
// one of 2 (one in twenty does); their mass 420, 991 and 1092.  By the vote
// 1242, 1500; 990, 1094.  Both forms for each score where any passes: 4518.
// Zeros put in the place of what is not seen, so that partly seen tiles can
// choose too: 1315 and 1568, and 138 instead of 115 for the mass of a windowed
// chunk.
template <int kScores, int kN>
__device__ __forceinline__ void make_scores(const AttnParams &a, u32 (&s)[kN], bool whole, bool &past) {
  if (a.cap != 0.0f && whole) {
    float big = 0.0f;
#pragma unroll
    for (int c = 0; c < kN; c += 2)
      big = tc::max3(big, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    past |= big * fabsf(a.inv_cap) > 1.0f;
  }
  if (a.cap == 0.0f || !whole || past) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const float v = __uint_as_float(s[c]);
      if constexpr (kScores == kFarCapped)
        s[c] = __float_as_uint(capped(a.cap, v * a.inv_cap));
      else
        s[c] = __float_as_uint(a.cap != 0.0f ? near_capped(a.cap, v * a.inv_cap) : v * a.scale);
    }
  } else {
    const u64 inv2 = tc::pair(a.inv_cap, a.inv_cap), cap2 = tc::pair(a.cap, a.cap);
#pragma unroll
    for (int c = 0; c < kN; c += 2) {
      const u64 x = tc::mul2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), inv2);
      const u64 u = tc::mul2(x, x);
      u64 y = tc::pair(tanh_p(6), tanh_p(6));
#pragma unroll
      for (int k = 5; k >= 0; --k) y = tc::fma2(y, u, tc::pair(tanh_p(k), tanh_p(k)));
      float y0, y1;
      tc::unpair(tc::mul2(tc::mul2(x, cap2), y), y0, y1);
      s[c] = __float_as_uint(y0);
      s[c + 1] = __float_as_uint(y1);
    }
  }
  __syncwarp();
}

template <int kType, int kDim, int kScores, bool kExt>
__global__ void __launch_bounds__(kTcThreadsOf<kType>, 1)
    kvcs_attend_tc_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v) {
  constexpr bool kBytes = kIs8Bit<kType>;   // (their queries and outputs are bf16, and so their values)
  constexpr bool kBf16 = kType != kKvFp16;
  constexpr int kThreads = kTcThreadsOf<kType>;
  using S = TcShape<kDim, kBytes>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TcShared sh;
  __shared__ TcNotes<kBytes> notes;
  __shared__ long long s_sum[kThreads / 32];
  const AttnParams &a = p.a;
  if (blockDim.x != kThreads) return;   // (the registers' split counts on every warp)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const u32 smem = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;   // swizzled tiles: 1 KiB
  const u32 q_smem = smem, ring = smem + 2 * S::kTileBytes;
  const u32 full = ptx::smem_addr(sh.full), empty = ptx::smem_addr(sh.empty);
  const u32 q_full = ptx::smem_addr(sh.q_full), s_full = ptx::smem_addr(sh.s_full);
  const u32 p_half = ptx::smem_addr(sh.p_half), p_ready = ptx::smem_addr(sh.p_ready);
  const u32 turns = ptx::smem_addr(sh.turns);
  const u32 o_full = ptx::smem_addr(sh.o_full);
  const u32 fix = ptx::smem_addr(&sh.fix), loaded = ptx::smem_addr(&sh.loaded);
  const u32 released = ptx::smem_addr(&sh.released), drain = ptx::smem_addr(sh.drain);
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(full + 8 * i, kBytes ? 4 : 1);
      ptx::mbar_init(empty + 8 * i, 2);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(q_full + 8 * i, 4);
      ptx::mbar_init(s_full + 8 * i, 1);
      ptx::mbar_init(p_half + 8 * i, 4);
      ptx::mbar_init(p_ready + 8 * i, 4);
      ptx::mbar_init(o_full + 8 * i, 1);
      ptx::mbar_init(turns + 8 * i, 1);
      ptx::mbar_init(drain + 8 * i, 1);
    }
    ptx::mbar_init(fix, 1);
    ptx::mbar_init(loaded, kBytes ? 4 : 1);
    for (int i = 0; i < S::kScaleTiles; ++i) ptx::mbar_init(ptx::smem_addr(sh.scales) + 8 * i, 8);
    ptx::mbar_init(released, 8);
    ptx::fence_barrier_init();
  }
  if (warp == 8) tc::tmem_alloc(ptx::smem_addr(&sh.tmem), 512);
  // units of the launch
  long long mine = 0;
  for (long long r = tid; r < a.tab.num_requests; r += kThreads) {
    const Request q = read_request(a.tab, r, a.map.block_size, blockIdx.x == 0);
    const long long rows = static_cast<long long>(q.n) * a.group;
    if (rows >= a.row_lo && rows <= a.row_hi) mine += (rows + kTcRows - 1) / kTcRows;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if constexpr (kExt) ptx::grid_dep_wait();   // the trees' masks are there from here on
  long long units = 0;
  for (int w = 0; w < kThreads / 32; ++w) units += s_sum[w];
  // (more than that only with requests that share rows, where offsets decrease
  // somewhere, which the request there has flagged)
  units = min(units * a.kv_heads, p.most_units) * p.splits;
  const u32 tmem = sh.tmem;
  // columns: S0, S1 (weights over their first half), O0, O1
  const u64 limit = p.timeout_ns;
  bool ok = true;
  TcFinder finder;

  if (kBytes && warp >= 12) {
   asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcBytesRegsConvert));
   if constexpr (kBytes) ok = tc_convert<kType, kDim>(p, sh, notes, ring, units);
  } else if (warp >= 8) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBytes ? kTcBytesRegsProducts : kTcRegsOther));
   if (kBytes && (warp & 1)) {
    // (two warps of the products' group have nothing to do)
   } else if (!kBytes && (warp == 9 || warp == 11)) {
    // ----------------------------------------------------------------- loads
    // of K (warp 9) and V (warp 11), which take turns in the ring; a lane per
    // box.  (One lane issuing all boxes, or one warp both halves, was slower
    // than the products: a TMA instruction takes an issuing warp 100 to 150
    // cycles.)
    const int half = warp == 9 ? 0 : 1;
    const int boxes = kTcKeys / p.box;
    const int bs = a.map.block_size;
    const CUtensorMap *map = half ? &map_v : &map_k;
    long long n_unit = 0;
    u32 it = half;       // position in the ring's sequence
    u32 n_fix = 0;
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x, ++n_unit) {
      const TcUnit x = finder.find<kExt>(p, u);
      const int par = n_unit & 1;
      bool bad = false;
      if (half) {
        bad = bad_blocks<kExt>(a, x);
        if (bad && lane == 0) raise(a.tab, kStatusBadBlockId);
        if (lane == 0) sh.n_dirty[par] = 0;
      }
      int at0 = x.q.at + x.row0 / a.group;
      const int at1 = x.q.at + (min(x.row0 + kTcRows, x.rows_all) - 1) / a.group;
      // every row of a tree sees the tokens up to it, none of a bad one any
      if (kExt && a.place && x.rows_all > 0) at0 = a.place[x.q.q0] < 0 ? -(1 << 30) : x.q.at - 1;
      int n_dirty = 0;
      // lane b holds the block of the tile's box b, read one tile ahead
      auto block_of = [&](int k) {
        const int key = tile_of<kExt>(x, k) * kTcKeys + lane * p.box;
        int block = -1;
        if (k < x.k1 && lane < boxes && key < x.q.keys) {
          block = a.tab.block_ids[x.q.pos0 + a.map.by_block(key)];
          if (block >= a.map.num_blocks) block = -1;
        }
        return block;
      };
      int ahead = block_of(x.k0);
      for (int k = x.k0; k < x.k1 && ok; ++k, it += 2) {
        const int key0 = tile_of<kExt>(x, k) * kTcKeys;
        const int block = ahead;
        ahead = block_of(k + 1);
        const u32 stage = it % S::kStages;
        const u32 dst = ring + stage * S::kTileBytes;
        // where the box starts, in the map's groups of 8 slots
        const int slot = (key0 + lane * p.box) % bs, sub = a.map.by_sub(slot);
        const int group = p.heads_in_groups
                              ? (sub * a.kv_heads + x.head) * (a.map.kbs / 8) + (slot - sub * a.map.kbs) / 8
                              : slot / 8;
        const int column = p.heads_in_groups ? 0 : x.head * S::kHalves;
        // tiles some row sees only in part, or with slots that hold no token
        const bool partly = key0 + kTcKeys - 1 > at0 ||
                            (a.window > 0 && key0 <= at1 - a.window &&
                             (!kExt || key0 + kTcKeys > x.sink_keys));
        const bool holes = key0 + kTcKeys > x.q.keys || bad;
        const bool mend = half == 1 && (partly || holes);
        const u32 bar = mend ? fix : full + 8 * stage;
        const int n = __popc(__ballot_sync(0xffffffffu, block >= 0));
        if (it >= S::kStages) ok = tc::wait(empty + 8 * stage, (it / S::kStages - 1) & 1, limit);
        if (!ok) break;
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar, static_cast<u32>(n) * p.box * 128 * S::kHalves);
        __syncwarp();
        if (block >= 0)
          tc::tma_load(dst + lane * p.box * 128 * S::kHalves, map, 0, 0, column, group, block, bar);
        if (mend) {
          ok = tc::wait(fix, n_fix & 1, limit);
          ++n_fix;
          u32 words = 0;   // lane i < 4: the noted rows of its quarter
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int row = i * 32 + lane, kk = key0 + row;
            const u32 at = dst + (row >> 3) * (S::kHalves * 1024) + (row & 7) * 128;
            const bool has = (kk >= x.lo || (kExt && kk < x.sink_keys)) && kk < x.hi &&
                             (!bad || good_block(a, x.q, kk));
            bool odd = false;
            if (has && partly) {
              constexpr u32 kExp = kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll 1
              for (int h = 0; h < S::kHalves; ++h)
#pragma unroll 4
                for (int c = 0; c < 8; ++c) {
                  // in an order that spreads the lanes over the banks
                  const uint4 v = lds128(at + h * 1024 + ((c ^ (lane & 7)) << 4));
                  const u32 w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    odd |= (w[e] & kExp) == kExp || (w[e] >> 16 & kExp) == kExp;
                }
            }
            if (!has || odd) {
#pragma unroll 1
              for (int h = 0; h < S::kHalves; ++h)
#pragma unroll 4
                for (int c = 0; c < 8; ++c)
                  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                   at + h * 1024 + ((c ^ (lane & 7)) << 4)),
                               "r"(0)
                               : "memory");
            }
            const u32 noted = __ballot_sync(0xffffffffu, odd);
            if (lane == i) words = noted;
          }
          if (__any_sync(0xffffffffu, words != 0)) {
            if (n_dirty < kTcDirty) {
              if (lane < 4) sh.dirty[par][n_dirty][lane] = words;
              if (lane == 0) {
                sh.dirty_tile[par][n_dirty] = tile_of<kExt>(x, k);
                sh.n_dirty[par] = n_dirty + 1;
              }
            }
            ++n_dirty;
          }
          tc::fence_async();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(full + 8 * stage);
        }
      }
      if (half) {
        // one unit ahead of the softmax at most: its notes are kept twice
        if (ok && n_unit > 0) ok = tc::wait(released, (n_unit - 1) & 1, limit);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(loaded);
      }
    }
    // Whichever role's wait ran out, nothing may still be on its way to this
    // CTA: the copies that nobody has waited for lie in the ring's last turn.
    // (Where all went well they have long come.)
    const u32 turn0 = it > S::kStages ? it - S::kStages : 0;
    for (u32 i = turn0 + ((turn0 + half) & 1); i < it; i += 2)
      tc::wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1, limit);
   } else {
    // -------------------------------------------------------------- products
    // A warp per query tile.  They take turns, each with O of token tile
    // k - 1 and then S of tile k in one go, so that the tiles settle half a
    // turn apart: one's products run while the other's weights are made, and
    // one warp's waits pass while the other's products run.  (Without turns
    // the two share the tensor cores product by product, which keeps both in
    // step and both waiting: 863 us.  One warp for both tiles shows its waits,
    // 721 us.)  A warp stays together and one lane issues: with the waits
    // inside a one-lane branch the whole took 822 us.
    // Every step is handed over and waited for, a unit's last one too (but for
    // tile 0's very first): a barrier shows its phase's parity alone, so that
    // a second turn given before the first is taken would read as none.
    // A commit speaks for its own thread's products, so a stage is free when
    // both warps have let it go.  In a unit of one query tile the other warp
    // does so too, behind its own products: the stages then become free in
    // their order, on which the loading warps rely (each waits for every other
    // use of a stage).
    constexpr u32 kDescS = tc::instr_desc(kBf16, 128, 128, false);
    constexpr u32 kDescO = tc::instr_desc(kBf16, 128, kDim, true);
    const int i = warp == 8 ? 0 : 1;
    const u32 ts = tmem + i * 128, to = tmem + 256 + i * 128;
    const u32 q_low = tc::desc_low(q_smem + i * S::kTileBytes, 16);
    const u32 k_low = tc::desc_low(ring, 16), v_low = tc::desc_low(ring, 1024);
    u32 stage = 0, turn = 0, n_q = 0, n_p = 0, n_t = 0;   // stage: ring position, turn: its phase
    bool begun = i == 1;   // tile 0 begins
    auto next_stage = [&]() {
      if (++stage == S::kStages) {
        stage = 0;
        turn ^= 1;
      }
    };
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const TcUnit x = finder.find<kExt>(p, u);
      if (i >= x.tiles) {   // the ring goes on: each stage is let go once it has come
        for (int n = 0; n < 2 * (x.k1 - x.k0); ++n) {
          ok = tc::wait(full + 8 * stage, turn, limit);
          if (!ok) break;
          if (tc::elect()) tc::commit(empty + 8 * stage);
          __syncwarp();
          next_stage();
        }
        continue;
      }
      const bool pair = x.tiles == 2;
      // ring: K0 V0 K1 V1 ...; V of tile k - 1 comes before K of tile k.
      for (int k = x.k0; k < x.k1 + (x.k1 > x.k0 ? 1 : 0) && ok; ++k) {
        const bool do_o = k > x.k0, do_s = k < x.k1;
        const u32 v_stage = stage;
        if (do_o) {
          ok = tc::wait(full + 8 * stage, turn, limit);
          next_stage();
        }
        const u32 k_stage = stage;
        if (do_s) {
          ok = ok && tc::wait(full + 8 * stage, turn, limit);
          next_stage();
          if (k == x.k0) ok = ok && tc::wait(q_full + 8 * i, n_q++ & 1, limit);
        }
        if (do_o) ok = ok && tc::wait(p_half + 8 * i, n_p & 1, limit);
        if (pair && begun) ok = ok && tc::wait(turns + 8 * i, n_t++ & 1, limit);
        if (!ok) break;
        begun |= pair;
        tc::fence_after();
        if (do_o) {
          // half of the weights at a time: the second half is made while the
          // first half's products run
          const u32 v = v_low + v_stage * (S::kTileBytes >> 4);
          if (tc::elect()) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_ts(to, ts + s * 8, tc::desc<S::kHalves * 1024>(v + s * (S::kHalves * 2048 >> 4)),
                         kDescO, k - 1 > x.k0 || s > 0);
          }
          __syncwarp();
          ok = tc::wait(p_ready + 8 * i, n_p++ & 1, limit);
          if (!ok) break;
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int s = 4; s < 8; ++s)
              tc::mma_ts(to, ts + s * 8, tc::desc<S::kHalves * 1024>(v + s * (S::kHalves * 2048 >> 4)),
                         kDescO, true);
            if (!do_s) tc::commit(o_full + 8 * i);
            tc::commit(empty + 8 * v_stage);
          }
          __syncwarp();
        }
        if (tc::elect()) {
          if (do_s) {
            const u32 kk = k_low + k_stage * (S::kTileBytes >> 4);
#pragma unroll
            for (int s = 0; s < kDim / 16; ++s)
              tc::mma_ss(ts, tc::desc<1024>(q_low + (((s >> 2) * S::kHalfBytes + (s & 3) * 32) >> 4)),
                         tc::desc<S::kHalves * 1024>(kk + (((s >> 2) * 1024 + (s & 3) * 32) >> 4)),
                         kDescS, s > 0);
            tc::commit(s_full + 8 * i);
            tc::commit(empty + 8 * k_stage);
          }
          if (pair) ptx::mbar_arrive(turns + 8 * (1 - i));
        }
        __syncwarp();
      }
    }
    // the products issued so far end before tensor memory is given back, a
    // wait of whichever role ran out (one lane issues and commits: a commit
    // speaks for its own thread's products)
    if (tc::elect()) tc::commit(drain + 8 * i);
    __syncwarp();
    if (!tc::wait(drain + 8 * i, 0, limit)) ok = false;
   }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBytes ? kTcBytesRegsSoftmax : kTcRegsSoftmax));
    const int i = warp >> 2;                 // query tile
    const int lr = (warp & 3) * 32 + lane;   // row of the tile
    const u32 lanes = static_cast<u32>((warp & 3) * 32) << 16;
    const u32 ts = tmem + i * 128 + lanes, to = tmem + 256 + i * 128 + lanes;
    u32 n_s = 0, n_o = 0, tile0 = 0;   // tile0: the tiles of the units before
    long long n_unit = 0;
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x, ++n_unit) {
      const TcUnit x = finder.find<kExt>(p, u);
      const int par = n_unit & 1;
      const bool work = i < x.tiles;
      const int row = x.row0 + i * 128 + lr;
      const bool has = row < x.rows_all;
      const int row_c = has ? row : x.rows_all - 1;
      const int tok_i = a.by_group(row_c), hq = x.head * a.group + row_c - tok_i * a.group;
      const int at = x.q.at + tok_i;
      RowSight sight = {};
      if constexpr (kExt) {
        if (work) sight = row_sight(a, x.q, tok_i);
      }
      float m = kNegInf, l = 0.0f;
      bool past = false;   // a capped score of the row has passed the cap
      const int nk = x.k1 - x.k0;
      const unsigned char *q_row =
          static_cast<const unsigned char *>(a.q) +
          ((x.q.q0 + tok_i) * a.q_stride + static_cast<long long>(hq) * kDim) * 2;
      if (work && nk > 0) {
        // the warp's query rows into shared memory, 16 bytes a lane
        const u32 qs = q_smem + i * S::kTileBytes;
        constexpr int kPieces = kDim / 8;   // 16-byte pieces of a row
#pragma unroll 8
        for (int n = 0; n < kPieces; ++n) {
          const int e = n * 32 + lane, r = e / kPieces, c = e % kPieces;
          const u64 src = __shfl_sync(0xffffffffu, reinterpret_cast<u64>(q_row), r);
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + c);
          const int tr = (warp & 3) * 32 + r;
          const u32 d = qs + (c >> 3) * S::kHalfBytes + tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(d), "r"(v.x), "r"(v.y),
                       "r"(v.z), "r"(v.w)
                       : "memory");
        }
        tc::fence_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(q_full + 8 * i);
        const bool bad = bad_blocks<kExt>(a, x);
        // what the warp's rows all see, and what none of them sees
        const int row_first = min(x.row0 + i * 128 + (warp & 3) * 32, x.rows_all - 1);
        const int row_last = min(row_first + 31, x.rows_all - 1);
        int at_min = x.q.at + row_first / a.group;
        const int at_max = x.q.at + row_last / a.group;
        if (kExt && a.place) at_min = min(sight.lim, x.q.at) - 1;   // (a bad tree is bad in all rows)
        const int upto = min(at, x.q.keys - 1);
        // The maximum to mx where that passes it by the slack, l and (added to
        // before) O relative to it; whether a row of the warp's did.
        auto raise_max = [&](float mx, bool added) {
          const bool raise_m = mx > m + kTcSlack || (m == kNegInf && mx != kNegInf);
          if (!__any_sync(0xffffffffu, raise_m)) return false;
          const float f = raise_m ? (m == kNegInf ? 0.0f : ex2(m - mx)) : 1.0f;
          if (raise_m) m = mx;
          l *= f;
          if (added) {
            const u64 ff = tc::pair(f, f);
#pragma unroll 1
            for (int c = 0; c < kDim; c += 16) {
              u32 o[16];
              tc::ld16(to + c, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float y0, y1;
                tc::unpair(tc::mul2(tc::pair(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), ff), y0, y1);
                o[e] = __float_as_uint(y0);
                o[e + 1] = __float_as_uint(y1);
              }
              tc::st16(to + c, o);
            }
          }
          return true;
        };
        for (int k = x.k0; k < x.k1; ++k) {
          ok = tc::wait(s_full + 8 * i, n_s & 1, limit);
          if (!ok) break;
          ++n_s;
          tc::fence_after();
          const int key0 = tile_of<kExt>(x, k) * kTcKeys;
          if constexpr (kBytes) {
            const u32 t = tile0 + k - x.k0;
            const u32 scales = ring + S::kStages * S::kTileBytes + t % S::kScaleTiles * (8 * kTcKeys);
            if constexpr (kIsScaled<kType>) {
              ok = tc::wait(ptx::smem_addr(sh.scales) + 8 * (t % S::kScaleTiles), t / S::kScaleTiles & 1,
                            limit);
              if (!ok) break;
            }
            const bool part = key0 + kTcKeys - 1 > min(at_min, x.q.keys - 1) ||
                              (a.window > 0 && key0 <= at_max - a.window && key0 + kTcKeys > x.sink_keys) ||
                              bad;
            const float sc = kScores == kPlain ? a.scale : 1.0f;
            // 64 tokens at a time, twice: for their maximum, and for the weights
            u32 s[64];
            auto scores = [&](int h) {
              tc::ld32(ts + 64 * h, s);
              tc::ld32(ts + 64 * h + 32, s + 32);
              tc::wait_ld();
              if constexpr (kIsScaled<kType>) {
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                  const uint4 f = lds128(scales + (64 * h + c) * 4);
                  float y[4];
                  tc::unpair(tc::mul2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                      tc::pair(__uint_as_float(f.x), __uint_as_float(f.y))), y[0], y[1]);
                  tc::unpair(tc::mul2(tc::pair(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                      tc::pair(__uint_as_float(f.z), __uint_as_float(f.w))), y[2], y[3]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) s[c + e] = __float_as_uint(y[e]);
                }
              }
              if constexpr (kScores != kPlain) make_scores<kScores>(a, s, !part, past);
              if (__builtin_expect(part, 0)) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const int first = key0 + 64 * h + 32 * w;
                  u32 see = seen_bits(a, sight, x.q.at, x.sink_keys, first) & bits_below(x.q.keys - first);
                  if (bad) {
#pragma unroll 1
                    for (int c = 0; c < 32; ++c)
                      if (see >> c & 1u && !good_block(a, x.q, first + c)) see &= ~(1u << c);
                  }
#pragma unroll
                  for (int c = 0; c < 32; ++c)
                    if (!(see >> c & 1u)) s[32 * w + c] = 0xff800000u;
                }
              }
            };
            float mx = kNegInf;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              scores(h);
              float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                m0 = tc::max3(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                m1 = tc::max3(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
              }
              mx = fmaxf(mx, fmaxf(m0, m1));
            }
            raise_max(mx * sc - kTcLift<kBf16>, k > x.k0);
            const float base = m == kNegInf ? 0.0f : -m;
            const u64 sc2 = tc::pair(sc, sc), base2 = tc::pair(base, base);
            u64 sum0 = 0, sum1 = 0;   // pairs of +0
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              scores(h);
              u32 w[32];
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                float y[4];
                tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, base2),
                           y[0], y[1]);
                tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc2,
                                    base2), y[2], y[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = ex2(y[j]);
                sum0 = tc::add2(sum0, tc::pair(y[0], y[1]));
                sum1 = tc::add2(sum1, tc::pair(y[2], y[3]));
                if constexpr (kIsScaled<kType>) {
                  const uint4 f = lds128(scales + (kTcKeys + 64 * h + c) * 4);
                  y[0] *= __uint_as_float(f.x);
                  y[1] *= __uint_as_float(f.y);
                  y[2] *= __uint_as_float(f.z);
                  y[3] *= __uint_as_float(f.w);
                }
                w[c / 2] = pack2<kBf16>(y[0], y[1]);
                w[c / 2 + 1] = pack2<kBf16>(y[2], y[3]);
              }
              tc::st32(ts + 32 * h, w);
              tc::wait_st();
              tc::fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive((h ? p_ready : p_half) + 8 * i);
            }
            float x0, x1;
            tc::unpair(tc::add2(sum0, sum1), x0, x1);
            l += x0 + x1;
            continue;
          }
          u32 s[128];
          tc::ld32(ts, s);
          tc::ld32(ts + 32, s + 32);
          tc::ld32(ts + 64, s + 64);
          tc::ld32(ts + 96, s + 96);
          tc::wait_ld();
          // scores = sc * s; capped ones, and those of a scale that would turn
          // the maximum round or make 0 of a masked score, are made first
          const bool part = key0 + kTcKeys - 1 > min(at_min, x.q.keys - 1) ||
                            (a.window > 0 && key0 <= at_max - a.window &&
                             (!kExt || key0 + kTcKeys > x.sink_keys)) || bad;
          float sc = a.scale;
          if constexpr (kScores != kPlain) {
            sc = 1.0f;
            make_scores<kScores>(a, s, !part, past);
          }
          if (__builtin_expect(part, 0)) {
            const int hi = upto - key0, lo = a.window > 0 ? at - a.window + 1 - key0 : 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              // bit c: the row sees token 32 w + c
              const int n1 = min(max(hi + 1 - 32 * w, 0), 32), n0 = min(max(lo - 32 * w, 0), 32);
              u32 see = (n1 == 32 ? 0xffffffffu : (1u << n1) - 1u) &
                        ~(n0 == 32 ? 0xffffffffu : (1u << n0) - 1u);
              if constexpr (kExt)
                see = seen_bits(a, sight, x.q.at, x.sink_keys, key0 + 32 * w) &
                      bits_below(x.q.keys - key0 - 32 * w);
              if (bad) {
#pragma unroll 1
                for (int c = 0; c < 32; ++c)
                  if (see >> c & 1u && !good_block(a, x.q, key0 + 32 * w + c)) see &= ~(1u << c);
              }
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(see >> c & 1u)) s[32 * w + c] = 0xff800000u;
            }
          }
          // The first half's weights are made with the maximum of the tiles
          // before while this tile's is found (it would stand in the way of
          // both halves otherwise); only where a row passes it are they made
          // again.
          const u64 sc2 = tc::pair(sc, sc);
          u32 w[32];
          u64 sum0, sum1, base2;
#pragma unroll 1
          for (bool first = true;; first = false) {
            const float base = m == kNegInf ? 0.0f : -m;
            base2 = tc::pair(base, base);
            sum0 = sum1 = 0;   // pairs of +0
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              float y[4];
              tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2,
                                  base2), y[0], y[1]);
              tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc2,
                                  base2), y[2], y[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = ex2(y[j]);
              sum0 = tc::add2(sum0, tc::pair(y[0], y[1]));
              sum1 = tc::add2(sum1, tc::pair(y[2], y[3]));
              w[c / 2] = pack2<kBf16>(y[0], y[1]);
              w[c / 2 + 1] = pack2<kBf16>(y[2], y[3]);
            }
            if (!first) break;
            float m0 = kNegInf, m1 = kNegInf, m2 = kNegInf, m3 = kNegInf;
#pragma unroll
            for (int c = 0; c < 128; c += 8) {
              m0 = tc::max3(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
              m1 = tc::max3(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
              m2 = tc::max3(m2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
              m3 = tc::max3(m3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
            }
            if (!raise_max(fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sc - kTcLift<kBf16>, k > x.k0)) break;
          }
          tc::st32(ts, w);
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(p_half + 8 * i);
#pragma unroll
          for (int c = 64; c < 128; c += 2) {
            float y0, y1;
            tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, base2),
                       y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            s[c] = __float_as_uint(y0);
            s[c + 1] = __float_as_uint(y1);
            w[c / 2 - 32] = pack2<kBf16>(y0, y1);
          }
          tc::st32(ts + 32, w);
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(p_ready + 8 * i);
          // this half's sum is off the products' path
#pragma unroll
          for (int c = 64; c < 128; c += 4) {
            sum0 = tc::add2(sum0, tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
            sum1 = tc::add2(sum1, tc::pair(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])));
          }
          float x0, x1;
          tc::unpair(tc::add2(sum0, sum1), x0, x1);
          l += x0 + x1;
        }
        if (ok) {
          ok = tc::wait(o_full + 8 * i, n_o & 1, limit);
          ++n_o;
          tc::fence_after();
        }
      }
      if (!ok) break;
      // all loads of the unit are noted before this
      ok = tc::wait(loaded, n_unit & 1, limit);
      if (!ok) break;
      tile0 += nk;
      const int n_dirty = kBytes ? 0 : sh.n_dirty[par];
      const bool whole = p.splits == 1;
      if (work) {
        const float inv = l > 0.0f || l != l ? a.v_scale / l : 0.0f;
        float *part = a.part + ((x.index * p.splits + x.split) * kTcRows + i * 128 + lr) *
                                   static_cast<long long>(S::kPartFloats);
        const long long out_row = (x.q.q0 + tok_i) * (a.group * a.kv_heads) + hq;
#pragma unroll
        for (int c = 0; c < kDim; c += 32) {
          u32 o[32];
          if (nk > 0) {
            tc::ld32(to + c, o);
            tc::wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          // tokens whose V was taken out of the tiles: for the rows that see them
          for (int d = 0; d < n_dirty; ++d) {
            const int key0 = sh.dirty_tile[par][d] * kTcKeys;
            for (int kk = 0; kk < kTcKeys; ++kk) {
              if (!(sh.dirty[par][d][kk >> 5] >> (kk & 31) & 1u)) continue;
              const int key = key0 + kk;
              if constexpr (kExt) {
                if (!(seen_bits(a, sight, x.q.at, x.sink_keys, key) & 1u)) continue;
              } else {
                if (key > at || (a.window > 0 && key <= at - a.window)) continue;
              }
              const int pos = a.map.by_block(key);
              const unsigned char *kp =
                  a.map.base + token_offset(a.map, a.tab.block_ids[x.q.pos0 + pos],
                                            key - pos * a.map.block_size, x.head);
              float dot = 0.0f;
              for (int e = 0; e < kDim / 2; ++e) {
                const u32 kw = reinterpret_cast<const u32 *>(kp)[e];
                const u32 qw = reinterpret_cast<const u32 *>(q_row)[e];
                dot += lo_of(kw, kBf16) * lo_of(qw, kBf16) + hi_of(kw, kBf16) * hi_of(qw, kBf16);
              }
              const float w = ex2(score_of(a, dot, 1.0f) - m);
              const u32 *vp = reinterpret_cast<const u32 *>(kp + a.map.half_stride) + c / 2;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const u32 vw = vp[e];
                o[2 * e] = __float_as_uint(__uint_as_float(o[2 * e]) + w * lo_of(vw, kBf16));
                o[2 * e + 1] = __float_as_uint(__uint_as_float(o[2 * e + 1]) + w * hi_of(vw, kBf16));
              }
            }
          }
          if constexpr (kBytes) {
            const int n0 = notes.n[par][0], n1 = n0 + notes.n[par][1], n2 = n1 + notes.n[par][2];
            const int n3 = n2 + notes.n[par][3];
#pragma unroll 1
            for (int d = 0; d < n3; ++d) {
              const int cw = (d >= n0) + (d >= n1) + (d >= n2);
              const int e = d - (cw == 0 ? 0 : cw == 1 ? n0 : cw == 2 ? n1 : n2);
              for (u32 left = notes.bits[par][cw][e]; left; left &= left - 1) {
                const int key = notes.key[par][cw][e] + __ffs(left) - 1;
                if (!(seen_bits(a, sight, x.q.at, x.sink_keys, key) & 1u)) continue;
                const int pos = a.map.by_block(key), slot = key - pos * a.map.block_size;
                const int block = a.tab.block_ids[x.q.pos0 + pos];
                const float w = noted_weight<kType, kDim>(a, block, slot, x.head, q_row, m);
                const unsigned char *vp =
                    a.map.base + token_offset(a.map, block, slot, x.head) + a.map.half_stride;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) +
                                         w * byte_value<kType>(vp, c + e, a.map.chunk_stride));
              }
            }
          }
          if (has && whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(a.out) +
                                                   (out_row * kDim + c) * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              u32 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack2<kBf16>(__uint_as_float(o[8 * e + 2 * j]) * inv,
                                    __uint_as_float(o[8 * e + 2 * j + 1]) * inv);
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (has) {
            float2 *dst = reinterpret_cast<float2 *>(part + c);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              dst[e] = make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          }
        }
        if (has && whole && a.lse) a.lse[out_row] = l == 0.0f ? kNegInf : kLn2 * (m + log2f(l));
        if (has && !whole) *reinterpret_cast<float2 *>(part + kDim) = make_float2(m, l);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(released);
    }
  }
  if (!ok && lane == 0) raise(a.tab, kStatusTimeout);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 8) tc::tmem_free(tmem, 512);
}

// Joins the parts of split units: a warp per two rows, all their loads in
// flight at once.  It waits for the parts' kernel as its programmatic
// dependent, its tables read by then.  (Joined by the last part to arrive, as
// kvcs_attend_kernel does, a warp had 32 rows one after another: 32 rows over
// 32,768 tokens took 91 us, 142 with fewer loads in flight; now 37.)
constexpr int kTcJoinThreads = 256;
constexpr int kTcJoinRows = kTcJoinThreads / 16;   // a CTA

template <bool kBf16, int kDim>
__global__ void __launch_bounds__(kTcJoinThreads)
    kvcs_attend_join_kernel(const __grid_constant__ TcParams p) {
  using S = TcShape<kDim>;
  constexpr int kCtas = kTcRows / kTcJoinRows;   // per unit
  const AttnParams &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = blockIdx.x / kCtas;
  const int first = static_cast<int>(blockIdx.x % kCtas) * kTcJoinRows + warp * 2;
  TcFinder finder;
  const TcUnit x = finder.find<false>(p, unit * p.splits);
  ptx::grid_dep_wait();
  const int rows = min(2, x.tiles == 0 ? 0 : x.rows_all - x.row0 - first);
  if (rows <= 0) return;
  const float *const part0 =
      a.part + (unit * p.splits * kTcRows + first) * static_cast<long long>(S::kPartFloats);
  constexpr long long kNext = static_cast<long long>(kTcRows) * S::kPartFloats;
  constexpr int kOwn = kDim / 32;   // columns a lane joins
  // lane: row lane / 16, part lane % 16
  const int mine = min(lane >> 4, rows - 1), s_mine = lane & 15;
  static_assert(kTcMaxSplits == 16, "half a warp's lanes hold a row's parts");
  float2 ml = make_float2(kNegInf, 0.0f);
  if (s_mine < p.splits)
    ml = __ldcg(reinterpret_cast<const float2 *>(part0 + mine * S::kPartFloats + s_mine * kNext + kDim));
  float v[2][kTcMaxSplits][kOwn];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float *row_at = part0 + min(r, rows - 1) * S::kPartFloats + lane * kOwn;
#pragma unroll
    for (int s = 0; s < kTcMaxSplits; ++s) {
#pragma unroll
      for (int c = 0; c < kOwn; ++c) v[r][s][c] = 0.0f;
      if (s < p.splits) {
        if constexpr (kOwn == 4)
          *reinterpret_cast<float4 *>(v[r][s]) =
              __ldcg(reinterpret_cast<const float4 *>(row_at + s * kNext));
        else
          *reinterpret_cast<float2 *>(v[r][s]) =
              __ldcg(reinterpret_cast<const float2 *>(row_at + s * kNext));
      }
    }
  }
  float jm = ml.x;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) jm = fmaxf(jm, __shfl_xor_sync(0xffffffffu, jm, o));
  const float f = ex2(ml.x - (jm == kNegInf ? 0.0f : jm));
  float jl = f * ml.y;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) jl += __shfl_xor_sync(0xffffffffu, jl, o);
  const float inv = jl > 0.0f || jl != jl ? a.v_scale / jl : 0.0f;
  if (s_mine == 0 && lane >> 4 < rows) store_lse(a, x.q, x.head, x.row0 + first + mine, jm, jl);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float o[kOwn];
#pragma unroll
    for (int c = 0; c < kOwn; ++c) o[c] = 0.0f;
#pragma unroll
    for (int s = 0; s < kTcMaxSplits; ++s) {
      const float fs = __shfl_sync(0xffffffffu, f, r * 16 + s);
#pragma unroll
      for (int c = 0; c < kOwn; ++c) o[c] += fs * v[r][s][c];
    }
    const float by = __shfl_sync(0xffffffffu, inv, r * 16);
    if (r < rows) {
#pragma unroll
      for (int c = 0; c < kOwn; c += 2)
        store_out(a, x.q, x.head, x.row0 + first + r, lane * kOwn + c, o[c] * by, o[c + 1] * by,
                  kBf16);
    }
  }
}

}  // namespace kvcs
