// kvcs_attend_cols.cuh -- attention of few rows over a paged cache for extended
// views: windows with first tokens kept, drafted trees, 8-bit caches with
// scales; and of any rows where the tensor-memory kernel does not take the cache.
//
// Mathematics, split of the line of tiles and join of parts as in
// kvcs_attend.cuh.  What differs is the products' orientation: tokens are their
// rows and query rows their columns,
//     S^T = K Q^T (16 tokens x 8 rows a product), O^T = V^T P^T,
// so a decode step's group of up to 8 rows fills a product where the other
// orientation leaves half of one (and of the softmax) to rows that are not there,
// and a K or V operand, which 8-bit caches have to convert first, is made once
// for kTiles products of 8 rows each (1, 2 or 4).  The weights of 8 tokens by 8
// rows become the second product's operand by one transposition of 8x8 16-bit
// values.  K chunk 4b + t of its token gives the A values of two k-steps (lane =
// 4 g + t; token pg(g), as in kvcs_attend.cuh); V chunks of the tokens t, t + 4,
// t + 8, t + 12 give, after byte permutes, those of 16 columns' rows: 8-bit ones
// are permuted before they are converted.
//
// The copies run ahead over the groups' borders: a group of a window is a dozen
// tiles, and filling the ring anew for each would cost as much as a tile or two.
//
// The running maximum is only raised when a score passes it by 2^2: most chunks
// need no maximum across lanes and no rescaling.  (fp16 weights are made 2^13 times
// larger than 2^(z - max), where kvcs_attend.cuh's, which never pass 1, are made
// 2^14 times larger: they reach 2^15 at most, and vanish below 2^-38 of the
// largest.)  Raised whenever a score passes it: 32 rows over e4m3 153 us instead of
// 142, the decode steps below 87 and 63.5 instead of 85 and 63.
//
// Scaled caches: a token's score is multiplied by its K scale, and its weight in
// the second product by its V scale, as 2^(z_ij + log2 |vs_j|) with vs_j's sign.
// 16 bits hold that product's range only relative to its own maximum: o is kept
// relative to mv_i = max_j (z_ij + log2 |vs_j|) as l is to m_i, and brought back to
// m_i at the group's end.
//
// Bound: by the bytes for 16-bit caches; for 8-bit ones by conversions, permutes and
// products waiting for one another (half of the issue slots are used, by 15 warps an
// SM; the largest share of their waits are instructions' own latencies).
// Measured (32 query heads to 8 KV heads of 128; one call after another, a replayed
// graph, as the comparisons here are, takes some 3 us more): 64 requests of 512 to
// 4096 tokens, one token each, int8 with scales, 82 us, 3.8 TB/s (replayed 84.5, e4m3 82.5); 64 of 600
// to 8192 under a window of 1024 with 4 first tokens, bf16, 59 us, 4.5 TB/s; 32 rows
// (trees of 4, 64 query heads) over 32 requests of 1000 to 4096, e4m3 with scales, 119
// us, 1.5 TB/s (read twice, half of the second time from L2).
// The step over int8 took 122 us with kvcs_attend.cuh's orientation, 97 with three
// CTAs an SM and the copies' places made anew for each.
#pragma once

#include "kvcs_attend.cuh"

namespace kvcs {

template <int kType, int kDim, int kTiles>
struct ColsShape {
  using A = AttendShape<kType, kDim>;
  static constexpr int kRows = 8 * kTiles;              // of a row tile
  static constexpr int kStageBytes = A::kStageBytes;
  // 8-bit caches: another CTA is worth more than a third stage, and with two
  // products a row tile more than queries in registers, too (a step over int8 85 and
  // 91 us; 16 rows of 64 requests of 2048 tokens, e4m3 with scales, 104 and 121)
  static constexpr bool kLean = kIs8Bit<kType> && kDim <= 128;
  static constexpr int kStages = kStageBytes >= 65536 || (kLean && kTiles < 4) ? 2 : 3;
  static constexpr int kRingBytes = kStages * kStageBytes;
  // scaled caches: a chunk's 16 K scales and 16 V scales
  static constexpr int kScaleBytes = kIsScaled<kType> ? 128 : 0;
  static constexpr int kScalesBytes = kStages * (kTileKeys / kChunkKeys) * kScaleBytes;
  static constexpr int kPartFloats = kDim + 4;           // o, m, l of a row, on 16-byte boundaries
  static constexpr int kJoinBytes = 3 * kRows * kPartFloats * 4;   // three warps' (m, l, o)
  static constexpr bool kHeld = kDim * kTiles < (kLean ? 256 : 512);   // queries in registers
  static constexpr int kQueryBytes = kHeld ? 0 : kRows * kDim * 2;
  static constexpr int kSmemBytes = kRingBytes + kScalesBytes + kJoinBytes + kQueryBytes;
  static_assert(kSmemBytes <= 224 * 1024, "with its tables a CTA takes 227 KB at most");
  // CTAs per SM: by registers (o: kDim / 4 a tile and lane, queries half of it)
  // and shared memory (228 KB, 1 KB of it reserved per CTA)
  static constexpr int kByRegs = kTiles == 1 && kDim <= (kIs8Bit<kType> ? 128 : 64) ? 4
                                 : kDim * kTiles <= (kLean ? 256 : 128)            ? 3
                                                                                   : 2;
  static constexpr int kBySmem = 228 * 1024 / (kSmemBytes + 2048);
  static constexpr int kCtas = kBySmem < 1 ? 1 : kBySmem < kByRegs ? kBySmem : kByRegs;
};

// CTAs an SM, and in all at most (the join's shared memory holds a factor for each).
struct ColsPlan {
  int ctas, most;
};
template <int kType, int kDim, int kTiles>
constexpr ColsPlan cols_plan() {
  using C = ColsShape<kType, kDim, kTiles>;
  return {C::kCtas, C::kJoinBytes / 4};
}

// Row tiles hold 8, 16 or 32 rows: as few as the most rows of a request need, 16 at
// most for heads of more than 128 (whose accumulators take the room).  Over 8-bit
// caches 16 too, up to 256 rows: tokens are read again from L2 for the next tile, by 12
// warps an SM and not 8.  For 32 rows over e4m3 with scales tiles of 8, 16 and 32 take
// 151, 122 and 142 us.  Tiles of 16 and 32, 16 requests of 2048 tokens: 32 rows 69 and
// 97, 256 rows 297 and 309, 512 rows 543 and 553; 4 of 8192: 512 rows 493 and 453, 2048
// rows 1877 and 1667.  The 4 rows of a step over int8, tiles of 8 and 16: 85 and 104.
__host__ __device__ constexpr int cols_tiles(int dim, long long rows, bool bytes) {
  return rows <= 8 ? 1 : rows <= 16 || dim > 128 || (bytes && rows <= 256) ? 2 : 4;
}

constexpr float kColsSlack = 2.0f;   // log2 of what scores pass the running maximum by
constexpr float kColsNone = -3.4028234e38f;   // a maximum of no scores: finite, so that a
                                              // masked score less it is -infinity
template <int kType>
constexpr float kColsLift = kType == kKvBf16 ? 0.0f : 13.0f;

// A request's share of the line of tiles: the tiles of the sinks, [0, sinks),
// then the window's from lo on.
struct ColsSpan {
  int row_tiles, lo, sinks, tiles;
  long long total;
};

__device__ __forceinline__ ColsSpan cols_span(const AttnParams &p, const Request &q, int rows) {
  ColsSpan s = {0, 0, 0, 0, 0};
  const long long r = static_cast<long long>(q.n) * p.group;
  if (r < p.row_lo || r > p.row_hi || q.n == 0) return s;
  s.row_tiles = static_cast<int>((r + rows - 1) / rows);
  const int first = p.window > 0 ? max(0, q.at - p.window + 1) : 0;
  const int end = min(q.keys, max(0, q.at + q.n));
  s.lo = first / kTileKeys;
  const int hi = (end + kTileKeys - 1) / kTileKeys;
  s.sinks = min(s.lo, (min(sink_keys_of(p, q), end) + kTileKeys - 1) / kTileKeys);
  s.tiles = max(1, s.sinks + max(0, hi - s.lo));   // rows that see nothing are still written
  s.total = static_cast<long long>(s.row_tiles) * s.tiles * p.kv_heads;
  return s;
}

// A place in the line: a request, one of its groups (row tile, KV head), and a
// tile k of the group's [c0, c1) that this CTA takes.
struct ColsCursor {
  long long r, before;   // request, and its first tile in the line
  Request q;
  ColsSpan sp;
  long long gs;          // the group's first tile in the line
  int head, rt;
  int k0, k1;            // the group's tiles of this CTA's run
  int k, c1;             // of these, the first one needed, and their end
  int c_window;          // the row tile's window starts at this tile
  int c_sinks;           // the sinks end before this tile
  int lo, hi, sink_keys; // tokens some row sees: [lo, hi), and those below sink_keys

  // first token of tile i
  __device__ __forceinline__ int key0(int i) const {
    return (i < sp.sinks ? i : sp.lo + i - sp.sinks) * kTileKeys;
  }
  __device__ __forceinline__ long long after() const { return gs + k1; }

  // The group of tile x, of a run that ends before b.
  __device__ __forceinline__ void open(const AttnParams &p, long long x, long long b, int rows) {
    while (x >= before + sp.total) {   // next request with tiles here
      before += sp.total;
      ++r;
      q = read_request(p.tab, r, p.map.block_size, false);
      sp = cols_span(p, q, rows);
    }
    const long long w = x - before, grp = w / sp.tiles;
    gs = before + grp * sp.tiles;
    k0 = static_cast<int>(w - grp * sp.tiles);
    k1 = static_cast<int>(min(static_cast<long long>(sp.tiles), b - gs));
    head = static_cast<int>(grp % p.kv_heads);
    rt = static_cast<int>(grp / p.kv_heads);
    const int rows_all = q.n * p.group;
    const int first = q.at + (rt * rows) / p.group;
    const int last = q.at + min(rt * rows + rows - 1, rows_all - 1) / p.group;
    // (a tree's rows: their tokens' depths start at 0)
    lo = p.window > 0 ? max(0, (p.place ? q.at : first) - p.window + 1) : 0;
    hi = min(q.keys, last + 1);
    sink_keys = sink_keys_of(p, q);
    c_window = sp.sinks + lo / kTileKeys - sp.lo;
    c_sinks = (sink_keys + kTileKeys - 1) / kTileKeys;
    k = k0 < c_sinks ? k0 : max(k0, c_window);
    c1 = min(k1, sp.sinks + max(0, (max(hi, 0) + kTileKeys - 1) / kTileKeys - sp.lo));
  }
};

// The tiles that a group needs, one after another: the sinks', then the window's.
struct ColsTiles {
  int k, end, key;       // tile, their end, the tile's first token
  int jump;              // where the sinks' tiles end, or -1
  int run_lo, run_hi;    // tokens of [run_lo, run_hi) are seen by some row
  __device__ __forceinline__ void begin(const ColsCursor &c, int first) {
    k = first;
    end = c.c1;
    key = c.key0(k);
    const bool sinks = k < c.c_sinks;
    jump = sinks ? c.c_sinks : -1;
    run_lo = sinks ? 0 : c.lo;
    // (a tile of both: its chunks' tokens are told apart where they are copied)
    run_hi = sinks && c.sink_keys <= c.lo ? min(c.sink_keys, c.hi) : c.hi;
  }
  __device__ __forceinline__ void step(const ColsCursor &c) {
    ++k;
    key += kTileKeys;
    if (k == jump) begin(c, max(c.c_sinks, c.c_window));
  }
};

// Running state of a row tile: lane 4 g + t holds rows 8 n + 2 t + i of tile n,
// and of their outputs the columns 64 jj + 8 pg(g) + 0 .. 7: o[n][4 jj + e][i]
// column 2 e, [2 + i] column 2 e + 1.
template <int kDim, int kTiles>
struct ColsState {
  float m[kTiles][2], l[kTiles][2], mv[kTiles][2];
  float o[kTiles][kDim / 16][4];
};

// What decides whether a chunk has tokens that some row does not see.
struct ColsSight {
  int lim_min;      // every row sees what is below it, but for the window
  int at_max;
  int tail, sink_keys;
};

// Queries of one tile: in registers (kHeld), or in shared memory at `at`, as
// [step][lane] pairs of words, where the accumulators leave no room for them.
template <bool kHeld, int kDim>
struct ColsQueries {
  u32 f[kHeld ? kDim / 8 : 1];
  u32 at;
  __device__ __forceinline__ void step(int s, u32 &b0, u32 &b1) const {
    if constexpr (kHeld) {
      b0 = f[2 * s];
      b1 = f[2 * s + 1];
    } else {
      const uint2 v = lds64(at + s * 256);
      b0 = v.x;
      b1 = v.y;
    }
  }
};

template <int kType, int kDim, int kTiles, bool kHeld>
__device__ __forceinline__ void cols_chunk(const AttnParams &p,
                                           const ColsQueries<kHeld, kDim> (&qf)[kTiles],
                                           ColsState<kDim, kTiles> &st, u32 ks, u32 vs, u32 scales,
                                           u32 valid, int key0, const ColsSight &sight,
                                           const RowSight *rows, const float *row_scales) {
  using S = AttendShape<kType, kDim>;
  constexpr bool kBf16 = kType == kKvBf16;
  constexpr int kMask = (S::kChunks < 8 ? S::kChunks : 8) - 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int pg = (g >> 1) | ((g & 1) << 2);   // token (and V chunk) of lane group g
  float s[kTiles][4];   // tokens pg (0, 1) and pg + 8 (2, 3), rows 2 t + i
  float s2[4] = {0.f, 0.f, 0.f, 0.f};          // (one tile: two chains of products)
#pragma unroll
  for (int n = 0; n < kTiles; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
  // Piece 4 b + t of row pg (or pg + 8) lies at piece (4 b + t) ^ (row & mask).
  const u32 k_even = ks + pg * S::kRowBytes + ((t ^ (pg & kMask)) << 4);
  const u32 k_odd = ks + pg * S::kRowBytes + (((t + 4) ^ (pg & kMask)) << 4);
  if constexpr (kIs8Bit<kType>) {
#pragma unroll
    for (int b = 0; b < kDim / 64; ++b) {
      const u32 a = (b & 1 ? k_odd : k_even) + (b >> 1) * 128;
      const uint4 x = lds128(a), y = lds128(a + 8 * S::kRowBytes);
      const u32 wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u32 lo0, hi0, lo1, hi1;
        bytes_to_half<kType>(wx[i], lo0, hi0);
        bytes_to_half<kType>(wy[i], lo1, hi1);
        const int step = 4 * b + i;
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          u32 b0, b1;
          qf[n].step(step, b0, b1);
          mma16816<false>(kTiles == 1 && (i & 1) ? s2 : s[n], lo0, lo1, hi0, hi1, b0, b1);
        }
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < kDim / 32; ++b) {
      const u32 a = (b & 1 ? k_odd : k_even) + (b >> 1) * 128;
      const uint4 x = lds128(a), y = lds128(a + 8 * S::kRowBytes);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        u32 b0, b1;
        qf[n].step(2 * b, b0, b1);
        mma16816<kBf16>(s[n], x.x, y.x, x.y, y.y, b0, b1);
        qf[n].step(2 * b + 1, b0, b1);
        mma16816<kBf16>(kTiles == 1 ? s2 : s[n], x.z, y.z, x.w, y.w, b0, b1);
      }
    }
  }
  if (kTiles == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] += s2[i];
  }
  float vsc[2];   // V scales of tokens pg, pg + 8 (an infinite one makes NaN of the row's own maximum)
  if constexpr (kIsScaled<kType>) {
    const float k0 = finite_or_nan(lds32f(scales + pg * 4)), k1 = finite_or_nan(lds32f(scales + pg * 4 + 32));
    vsc[0] = lds32f(scales + pg * 4 + 64);
    vsc[1] = lds32f(scales + pg * 4 + 96);
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[n][i] *= k0;
        s[n][i + 2] *= k1;
      }
  }
  // scores = sc * s; capped ones, and those of a scale that would turn the
  // maximum round or make NaN of a masked score, are made first
  float sc[kTiles][2];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    sc[n][0] = sc[n][1] = p.scale;
    if constexpr (kIs8Bit<kType>) {
      const float2 x = *reinterpret_cast<const float2 *>(row_scales + 8 * n + 2 * t);
      sc[n][0] = x.x;
      sc[n][1] = x.y;
    }
  }
  if (__builtin_expect(p.cap != 0.0f || p.scale <= 0.0f, 0)) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = score_of(p, s[n][i], kIs8Bit<kType> ? sc[n][i & 1] : 1.0f);
      sc[n][0] = sc[n][1] = 1.0f;
    }
  }
  const bool partly = valid != 0xffffu || key0 + kChunkKeys > sight.lim_min ||
                      (p.window > 0 && key0 <= sight.at_max - p.window &&
                       key0 + kChunkKeys > sight.sink_keys);
  u32 mine = 0;   // bits of the chunk's tokens that row `lane` sees
  if (__builtin_expect(partly, 0)) {
    if (lane < 8 * kTiles) mine = seen_bits(p, rows[lane], sight.tail, sight.sink_keys, key0) & valid;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32 see = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t + i) >> pg;
        if (!(see & 1u)) s[n][i] = kNegInf;
        if (!(see >> 8 & 1u)) s[n][i + 2] = kNegInf;
      }
  }
  // z - m; where one passes the slack, or is its row's first, the maxima are
  // found anew
  float lv[2], z[kTiles][4], y[kTiles][4];
  if constexpr (kIsScaled<kType>) {
    lv[0] = lg2(fabsf(vsc[0]));
    lv[1] = lg2(fabsf(vsc[1]));
  }
  float top = kNegInf;
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[n][i] = fmaf(s[n][i], sc[n][i & 1], -st.m[n][i & 1]);
      top = fmaxf(top, z[n][i]);
      if constexpr (kIsScaled<kType>) {
        y[n][i] = fmaf(s[n][i], sc[n][i & 1], lv[i >> 1] - st.mv[n][i & 1]);
        top = fmaxf(top, y[n][i]);
      }
    }
  if (__builtin_expect(__any_sync(0xffffffffu, top > kColsSlack + kColsLift<kType>), 0)) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      float fo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = fmaxf(s[n][i], s[n][i + 2]) * sc[n][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        const float old = st.m[n][i], now = fmaxf(old, v - kColsLift<kType>);
        fo[i] = ex2(old - now);
        st.l[n][i] *= fo[i];
        st.m[n][i] = now;
        z[n][i] = fmaf(s[n][i], sc[n][i], -now);
        z[n][i + 2] = fmaf(s[n][i + 2], sc[n][i], -now);
        if constexpr (kIsScaled<kType>) {
          float u = fmaxf(fmaf(s[n][i], sc[n][i], lv[0]), fmaf(s[n][i + 2], sc[n][i], lv[1]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
          const float oldv = st.mv[n][i], nowv = fmaxf(oldv, u - kColsLift<kType>);
          fo[i] = ex2(oldv - nowv);
          st.mv[n][i] = nowv;
          y[n][i] = fmaf(s[n][i], sc[n][i], lv[0] - nowv);
          y[n][i + 2] = fmaf(s[n][i + 2], sc[n][i], lv[1] - nowv);
        }
      }
#pragma unroll
      for (int e = 0; e < kDim / 16; ++e) {
        st.o[n][e][0] *= fo[0];
        st.o[n][e][1] *= fo[1];
        st.o[n][e][2] *= fo[0];
        st.o[n][e][3] *= fo[1];
      }
    }
  }
  // The weights, as the products' B operand: rounded to the cache's 16-bit type
  // (fp16 for 8-bit caches), each by 2^-8 (2^-11) of itself at most, as an
  // output's own rounding; fp16 ones below 2^-27 of the largest by up to 2^-38 of
  // that.  l counts them whole.
  u32 pb[kTiles][2];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = ex2(z[n][i]);
      st.l[n][i & 1] += w;
      s[n][i] = kIsScaled<kType> ? copysignf(ex2(y[n][i]), vsc[i >> 1]) : w;
    }
    if (kIsScaled<kType> && __builtin_expect(partly, 0)) {
      // (the scale of a token that a row does not see may be anything)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32 see = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t + i) >> pg;
        if (!(see & 1u)) s[n][i] = 0.0f;
        if (!(see >> 8 & 1u)) s[n][i + 2] = 0.0f;
      }
    }
    pb[n][0] = movmatrix(pack2<kBf16>(s[n][0], s[n][1]));
    pb[n][1] = movmatrix(pack2<kBf16>(s[n][2], s[n][3]));
  }
  // pieces 8 jj + pg of rows t + 4 k (8-bit: 8-byte halves of pieces)
  const int vp = kIs8Bit<kType> ? pg >> 1 : pg, vh = kIs8Bit<kType> ? (pg & 1) << 3 : 0;
  const u32 v_even = vs + t * S::kRowBytes + ((vp ^ (t & kMask)) << 4) + vh;
  const u32 v_odd = vs + (t + 4) * S::kRowBytes + ((vp ^ ((t + 4) & kMask)) << 4) + vh;
#pragma unroll
  for (int jj = 0; jj < kDim / 64; ++jj) {
    u32 v[4][4];   // tokens t + 4 k: eight values (8-bit: in two words)
    u32 odd = 0;   // a non-finite value, in chunks that some row sees only partly
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u32 at = (k & 1 ? v_odd : v_even) + (k >> 1) * 8 * S::kRowBytes;
      if constexpr (kIs8Bit<kType>) {
        // jj moves by 4 pieces: bit 2 of the XORed place
        const u32 flip = (jj & 1) << 6;
        const uint2 w = lds64((S::kChunks >= 8 ? vs + ((at - vs) ^ flip) : at) + (jj >> 1) * 128);
        v[k][0] = w.x;
        v[k][1] = w.y;
        if (kType != kKvInt8Scaled && partly) {   // e4m3's NaN: all bits but the sign
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32 x = v[k][e] & 0x7f7f7f7fu;   // (adding 1 carries into a byte's top bit there alone)
            odd |= (x + 0x01010101u) & 0x80808080u;
          }
        }
      } else {
        const uint4 w = lds128(at + jj * 128);
        v[k][0] = w.x;
        v[k][1] = w.y;
        v[k][2] = w.z;
        v[k][3] = w.w;
        if (partly) {
          constexpr u32 kExp = kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            odd |= (v[k][e] & kExp) == kExp || (v[k][e] >> 16 & kExp) == kExp;
        }
      }
    }
    if (kType != kKvInt8Scaled && __builtin_expect(partly, 0) && __any_sync(0xffffffffu, odd)) {
      // A weight of 0 times a non-finite value is NaN: add the chunk's values one
      // token at a time, and only to the rows that see it.
#pragma unroll 1
      for (int kk = 0; kk < kChunkKeys; ++kk) {
        const int k8 = kk & 7, src = ((k8 & 3) << 1 | k8 >> 2) * 4 + t;   // lane group of token kk
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w0 = __shfl_sync(0xffffffffu, s[n][i], src);
            const float w1 = __shfl_sync(0xffffffffu, s[n][i + 2], src);
            const u32 see = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t + i);
            if (!(see >> kk & 1u)) continue;
            const float w = kk < 8 ? w0 : w1;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int col = 64 * jj + 8 * pg + c;
              u32 raw;
              float x;
              if constexpr (kIs8Bit<kType>) {
                const u32 a = vs + kk * S::kRowBytes + (((col >> 4) ^ (kk & kMask)) << 4) + (col & 15);
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(raw) : "r"(a));
                u32 lo, up;
                bytes_to_half<kType>(raw, lo, up);
                x = half_bits_to_float(lo & 0xffffu, false);
              } else {
                const u32 a = vs + kk * S::kRowBytes + (((col >> 3) ^ (kk & kMask)) << 4) + (col & 7) * 2;
                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(raw) : "r"(a));
                x = half_bits_to_float(raw & 0xffffu, kBf16);
              }
              st.o[n][4 * jj + (c >> 1)][(c & 1) * 2 + i] += w * x;
            }
          }
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // columns 2 e and 2 e + 1
      u32 a0, a1, a2, a3;
      if constexpr (kIs8Bit<kType>) {
        const u32 sel = e & 1 ? 0x7362u : 0x5140u;
        bytes_to_half<kType>(__byte_perm(v[0][e >> 1], v[1][e >> 1], sel), a0, a1);
        bytes_to_half<kType>(__byte_perm(v[2][e >> 1], v[3][e >> 1], sel), a2, a3);
      } else {
        a0 = __byte_perm(v[0][e], v[1][e], 0x5410u);
        a1 = __byte_perm(v[0][e], v[1][e], 0x7632u);
        a2 = __byte_perm(v[2][e], v[3][e], 0x5410u);
        a3 = __byte_perm(v[2][e], v[3][e], 0x7632u);
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
        mma16816<kBf16>(st.o[n][4 * jj + e], a0, a1, a2, a3, pb[n][0], pb[n][1]);
    }
  }
}

// The rows of a row tile as B fragments: word pairs of lane 4 g + t's 16-byte
// (8-bit caches: 32-byte) pieces of row g of each tile.  8-bit caches multiply in
// fp16: bf16 queries are brought near 1 by a power of two per row (in rs, of the
// rows 2 t + i), so only values 2^-24 below the row's largest are lost.
// (In shared memory: each warp makes the tiles whose number is its own, modulo
// four, and all read them after a barrier.)
template <int kType, int kDim, int kTiles, bool kHeld>
__device__ __forceinline__ void cols_queries(const AttnParams &p, const Request &q, int head, int row0,
                                             ColsQueries<kHeld, kDim> (&qf)[kTiles], u32 smem,
                                             float *row_scales) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const unsigned char *base = static_cast<const unsigned char *>(p.q);
  const int rows_all = q.n * p.group;
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    if (!kHeld) qf[n].at = smem + n * (kDim / 16 * 256) + lane * 8;
    if (!kHeld && (n & 3) != warp) continue;
    const int row = row0 + 8 * n + g;
    const bool has = row < rows_all;
    const int token = p.by_group(has ? row : 0);
    const int hq = head * p.group + (has ? row : 0) - token * p.group;
    const unsigned char *src =
        base + ((q.q0 + token) * p.q_stride + static_cast<long long>(hq) * p.head_dim) * 2;
    constexpr int kPiece = kIs8Bit<kType> ? 16 : 8;   // elements a lane takes at once
    u32 f[kDim / 8];
#pragma unroll
    for (int b = 0; b < kDim / (4 * kPiece); ++b) {
      const int d = (4 * b + t) * kPiece;
#pragma unroll
      for (int h = 0; h < kPiece / 8; ++h) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (has && d + 8 * h < p.head_dim) v = __ldg(reinterpret_cast<const uint4 *>(src + (d + 8 * h) * 2));
        const int w = (kPiece / 2) * b + 4 * h;
        f[w] = v.x;
        f[w + 1] = v.y;
        f[w + 2] = v.z;
        f[w + 3] = v.w;
      }
    }
    if (kIs8Bit<kType>) {
      float own = 1.0f;
      if (p.q_bf16) {
        float top = 0.0f;
#pragma unroll
        for (int w = 0; w < kDim / 8; ++w)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(f[w] << 16)),
                                 fabsf(__uint_as_float(f[w] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = top > 0.0f && top < __builtin_huge_valf() ? ilogbf(top) : 0;
        own = ldexpf(1.0f, ex < -126 ? -126 : ex);
        const float inv = ldexpf(1.0f, ex < -126 ? 126 : -ex);
#pragma unroll
        for (int w = 0; w < kDim / 8; ++w)
          f[w] = pack2<false>(__uint_as_float(f[w] << 16) * inv, __uint_as_float(f[w] & 0xffff0000u) * inv);
      }
      // what a product is multiplied by (capped scores and scales that are not
      // positive: the power of two alone); a factor may underflow: 0 would make
      // NaN of a masked score
      if (!(p.cap != 0.0f || p.scale <= 0.0f)) own = fmaxf(own * p.scale, __int_as_float(1));
      if (t == 0 && (!kHeld || warp == 0)) row_scales[8 * n + g] = own;
    }
    if constexpr (kHeld) {
#pragma unroll
      for (int w = 0; w < kDim / 8; ++w) qf[n].f[w] = f[w];
    } else {
#pragma unroll
      for (int w = 0; w < kDim / 16; ++w)
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(qf[n].at + w * 256), "r"(f[2 * w]),
                     "r"(f[2 * w + 1])
                     : "memory");
    }
  }
}

// Any chunk; returns its mask of readable tokens.  Tokens outside [lo, hi) but
// for those below sink_keys, and tokens of bad blocks, become zeros.  `scales`:
// where the chunk's scales go.  It takes all chunks of pools without runs of 16 tokens
// or of other widths: 64 requests under a window of 1024 (above), blocks of 8 and 24
// slots 92 us and 91 where 16 take 62, heads of 96 92; int8 with scales, heads of 96 and
// blocks of 24 slots 68.  (X-split pools have runs, whose pieces lie apart: 94.)
template <int kType, int kDim>
__device__ __noinline__ u32 cols_load_any(const AttnParams &p, long long pos0, int head, u32 chunk,
                                          int key0, int lo, int hi, int sink_keys, u32 scales) {
  using S = AttendShape<kType, kDim>;
  using L = ChunkLanes<kType, kDim>;
  const int lane = threadIdx.x & 31;
  const u32 first = L::first();
  const int row_bytes = p.head_dim * S::kElem;
  // lane's token (of each half of the warp): its place in the pool
  const int key = key0 + (lane & 15);
  bool ok = (key >= lo || key < sink_keys) && key < hi;
  long long off = 0, at = 0;
  if (ok) {
    const int pos = p.map.by_block(key), slot = key - pos * p.map.block_size;
    const int block = p.tab.block_ids[pos0 + pos];
    if (block < 0 || block >= p.map.num_blocks) {
      ok = false;
      raise(p.tab, kStatusBadBlockId);
    } else {
      off = token_offset(p.map, block, slot, head);
      at = (static_cast<long long>(block) * p.kv_heads + head) * p.map.block_size + slot;
    }
  }
  const u32 mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
  if constexpr (kIsScaled<kType>)
    cp_async4z(scales + lane * 4, (lane < 16 ? p.k_scales : p.v_scales) + at, ok ? 4u : 0u);
#pragma unroll 1
  for (int j = 0; j < L::kTurns; ++j) {
    const int row = j * L::kDown + lane / L::kAcross;
    const long long row_off = __shfl_sync(0xffffffffu, off, row);
    const bool row_ok = mask >> row & 1u;
#pragma unroll 1
    for (int k = 0; k < L::kSpans; ++k) {
      const int c = k * L::kAcross + lane % L::kAcross, left = row_ok ? row_bytes - c * 16 : 0;
      const u32 d = chunk + (first ^ L::flip(j)) + L::place(j, k);
      const unsigned char *src =
          p.map.base + (left > 0 ? row_off + static_cast<long long>(c) * p.map.chunk_stride : 0);
      const long long vh = left > 0 ? p.map.half_stride : 0;
      if (!p.unit8) {
        const u32 bytes = left > 0 ? 16u : 0u;
        cp_async16(d, src, bytes);
        cp_async16(d + S::kChunkBytes, src + vh, bytes);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const u32 bytes = left > 8 * e ? 8u : 0u;
          cp_async8z(d + 8 * e, src + (bytes ? 8 * e : 0), bytes);
          cp_async8z(d + S::kChunkBytes + 8 * e, src + vh + (bytes ? 8 * e : 0), bytes);
        }
      }
    }
  }
  return mask;
}

// Eight values of a row's output, times f, in 16 bytes.
__device__ __forceinline__ uint4 packed8(const float (&v)[8], float f, bool bf16) {
  u32 w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = bf16 ? pack2<true>(v[2 * e] * f, v[2 * e + 1] * f) : pack2<false>(v[2 * e] * f, v[2 * e + 1] * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kType, int kDim, int kTiles>
__global__ void __launch_bounds__(kAttendThreads, (ColsShape<kType, kDim, kTiles>::kCtas))
    kvcs_attend_cols_kernel(const __grid_constant__ AttnParams p) {
  using S = AttendShape<kType, kDim>;
  using C = ColsShape<kType, kDim, kTiles>;
  using L = ChunkLanes<kType, kDim>;
  constexpr int kRows = C::kRows;
  extern __shared__ __align__(1024) unsigned char cols_smem[];   // (pieces' places are XORed)
  __shared__ long long s_scan[4], s_req[2];
  __shared__ u32 s_mask[C::kStages][4];
  __shared__ RowSight s_rows[kRows];
  __shared__ __align__(8) float s_scales[kRows];   // 8-bit caches: what rows' products are multiplied by
  __shared__ ColsCursor s_group, s_next[4];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int pg = (g >> 1) | ((g & 1) << 2);
  const long long R = p.tab.num_requests;

  // the line of tiles: its length, then the request this CTA's run starts in
  long long sum = 0;
  for (long long r = tid; r < R; r += kAttendThreads)
    sum += cols_span(p, read_request(p.tab, r, p.map.block_size, blockIdx.x == 0), kRows).total;
  long long total;
  const long long ahead_of_me = block_scan(sum, &total, s_scan);
  const long long grid = min(static_cast<long long>(gridDim.x), total);
  if (blockIdx.x >= grid) {
    ptx::grid_dep_wait();
    return;
  }
  const long long a = total * blockIdx.x / grid, b = total * (blockIdx.x + 1ll) / grid;
  long long before = 0;
  for (long long c = 0;; c += kAttendThreads) {
    const long long rr = c + tid;
    long long v = sum, all = total, ex = ahead_of_me;
    if (R > kAttendThreads) {   // (otherwise the first scan tells)
      v = rr < R ? cols_span(p, read_request(p.tab, rr, p.map.block_size, false), kRows).total : 0;
      ex = before + block_scan(v, &all, s_scan);
    }
    if (before + all > a) {
      if (v > 0 && ex <= a && a < ex + v) {
        s_req[0] = rr;
        s_req[1] = ex;
      }
      __syncthreads();
      break;
    }
    before += all;
  }

  const u32 ring = ptx::smem_addr(cols_smem);
  float *const js = reinterpret_cast<float *>(cols_smem + C::kRingBytes + C::kScalesBytes);
  const u32 lane_first = L::first();
  const bool out_bf16 = kType == kKvBf16 || (kIs8Bit<kType> && p.q_bf16);
  auto stage_at = [&](int stage) { return ring + (stage * 4 + warp) * 2 * S::kChunkBytes; };
  auto scales_at = [&](int stage) { return ring + C::kRingBytes + (stage * 4 + warp) * C::kScaleBytes; };

  // The group being computed, and per warp the group of the tile copied next
  // (in shared memory: both at hand would take 70 registers).  A tile's block is
  // looked up before the copies of the tile before it.
  if (tid == 0) {
    ColsCursor c;
    c.r = s_req[0];
    c.before = s_req[1];
    c.q = read_request(p.tab, c.r, p.map.block_size, false);
    c.sp = cols_span(p, c.q, kRows);
    c.open(p, a, b, kRows);
    s_group = c;
    for (int w = 0; w < 4; ++w) s_next[w] = c;
  }
  __syncthreads();
  ColsCursor &f = s_next[warp];
  ColsTiles next;    // its tiles, the next one first
  const int *ids;    // its request's blocks
  const unsigned char *src;   // the pool's first byte for this lane and the KV head
  const long long lane_src = static_cast<long long>(lane / L::kAcross) * p.map.slot_stride +
                             (lane % L::kAcross) * static_cast<long long>(p.map.chunk_stride);
  bool more = true;
  // of the next tile's 16 tokens that are this warp's: their block (-1: none that
  // holds them all in a row), their first slot, and which of them some row sees
  int ahead = -1, slot = 0;
  u32 seen = 0;
  auto enter = [&]() {
    next.begin(f, f.k);
    ids = p.tab.block_ids + f.q.pos0;
    src = p.map.base + f.head * p.map.head_stride + lane_src;
    // its queries into L2 (a tile's are read by four lanes a row, 128 bytes each at most)
    const int row = f.rt * kRows + lane / 4;
    if (warp == 0 && row < f.q.n * p.group) {
      const int token = p.by_group(row);
      const unsigned char *at = static_cast<const unsigned char *>(p.q) +
                                ((f.q.q0 + token) * p.q_stride +
                                 static_cast<long long>(f.head * p.group + row - token * p.group) * p.head_dim) * 2;
      if ((lane & 3) * 128 < p.head_dim * 2)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + (lane & 3) * 128));
    }
  };
  enter();
  auto settle = [&]() {   // to a tile that is needed, if there is one
    while (next.k >= next.end) {
      if (f.after() >= b) {
        more = false;
        return;
      }
      ColsCursor n = f;
      n.open(p, n.after(), b, kRows);
      __syncwarp();
      if (lane == 0) f = n;
      __syncwarp();
      enter();
    }
    const int key = next.key + warp * kChunkKeys;
    ahead = -1;
    seen = 0xffffu;
    if (__builtin_expect(key < next.run_lo || key + kChunkKeys > next.run_hi, 0)) {
      seen = bits_below(f.hi - key) & (~bits_below(f.lo - key) | bits_below(f.sink_keys - key)) & 0xffffu;
      if (seen == 0) return;
    }
    if (p.runs) {
      const int pos = p.map.by_block(key);
      ahead = ids[pos];
      slot = key - pos * p.map.block_size;
    }
  };
  settle();
  int put = 0;
  auto fetch = [&]() {
    if (more) {
      const u32 dst = stage_at(put), sdst = scales_at(put);
      u32 mask = seen;   // (of none: nothing is copied)
      const int block = ahead;
      if (__builtin_expect(block >= 0 && block < p.map.num_blocks, 1)) {
        const int sub = p.map.by_sub(slot);
        load_run<kType, kDim>(p, dst, lane_first,
                              src + block * p.map.block_stride + sub * p.map.sub_stride +
                                  static_cast<long long>(slot - sub * p.map.kbs) * p.map.slot_stride);
        if constexpr (kIsScaled<kType>) {
          // 16 scales of K in four pieces, 16 of V
          if (lane < 8) {
            const long long first =
                (static_cast<long long>(block) * p.kv_heads + f.head) * p.map.block_size + slot;
            cp_async16(sdst + lane * 16, (lane < 4 ? p.k_scales : p.v_scales) + first + (lane & 3) * 4, 16);
          }
        }
      } else if (mask != 0) {
        mask = cols_load_any<kType, kDim>(p, f.q.pos0, f.head, dst, next.key + warp * kChunkKeys, f.lo,
                                          f.hi, f.sink_keys, sdst);
      }
      next.step(f);
      settle();
      if (lane == 0) s_mask[put][warp] = mask;
      put = put + 1 == C::kStages ? 0 : put + 1;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int k = 0; k < C::kStages - 1; ++k) fetch();
  if (p.place) ptx::grid_dep_wait();   // the trees' masks are there from here on

  int stage = 0;
  for (;;) {
    const ColsCursor &c = s_group;
    const int rows_all = c.q.n * p.group, row0 = c.rt * kRows;
    const bool whole = c.k0 == 0 && c.k1 == c.sp.tiles;
    ColsQueries<C::kHeld, kDim> qf[kTiles];
    cols_queries<kType, kDim, kTiles, C::kHeld>(
        p, c.q, c.head, row0, qf, ring + C::kRingBytes + C::kScalesBytes + C::kJoinBytes, s_scales);
    if (tid < kRows) s_rows[tid] = row_sight(p, c.q, p.by_group(min(row0 + tid, rows_all - 1)));
    ColsSight sight;
    sight.lim_min = c.q.at + row0 / p.group + 1;
    sight.at_max = c.q.at + (min(row0 + kRows, rows_all) - 1) / p.group;
    sight.tail = c.q.at;
    sight.sink_keys = c.sink_keys;
    if (p.place) {   // (a bad tree is bad in all rows)
      sight.lim_min = p.place[c.q.q0] < 0 ? -(1 << 30) : c.q.at;
      sight.at_max = c.q.at + c.q.n - 1;
    }
    __syncthreads();
    ColsState<kDim, kTiles> st;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        st.m[n][i] = st.mv[n][i] = kColsNone;
        st.l[n][i] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < kDim / 16; ++e) st.o[n][e][0] = st.o[n][e][1] = st.o[n][e][2] = st.o[n][e][3] = 0.0f;
    }
    ColsTiles tiles;
    tiles.begin(c, c.k);
    for (; tiles.k < tiles.end; tiles.step(c)) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      fetch();
      const u32 at = stage_at(stage);
      if (s_mask[stage][warp] != 0)
        cols_chunk<kType, kDim, kTiles, C::kHeld>(p, qf, st, at, at + S::kChunkBytes, scales_at(stage),
                                                s_mask[stage][warp], tiles.key + warp * kChunkKeys,
                                                sight, s_rows, s_scales);
      __syncwarp();   // the stage is filled again
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) st.l[n][i] += __shfl_xor_sync(0xffffffffu, st.l[n][i], o);
        if constexpr (kIsScaled<kType>) {
          // o relative to m, both without the products' lift: values have all of 32
          // bits' range, and a sum of weights 2^13 times larger would leave them 2^97
          st.l[n][i] *= ex2(-kColsLift<kType>);
          st.m[n][i] += kColsLift<kType>;
          const float f2 = ex2(st.mv[n][i] - st.m[n][i]);   // (of no scores: o is 0)
#pragma unroll
          for (int e = 0; e < kDim / 16; ++e) {
            st.o[n][e][i] *= f2;
            st.o[n][e][2 + i] *= f2;
          }
        }
      }

    // join the four warps' (m, l, o): the others hand theirs to warp 0
    float *const part_of_cta = p.part + static_cast<long long>(blockIdx.x) * 2 * kRows * C::kPartFloats;
    float *const part = part_of_cta + (c.k0 == 0 ? 1 : 0) * kRows * C::kPartFloats;
    if (warp > 0) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float *dst = js + ((warp - 1) * kRows + 8 * n + 2 * t + i) * C::kPartFloats;
#pragma unroll
          for (int jj = 0; jj < kDim / 64; ++jj)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              *reinterpret_cast<float4 *>(dst + 64 * jj + 8 * pg + 2 * e) =
                  make_float4(st.o[n][4 * jj + e][i], st.o[n][4 * jj + e][2 + i],
                              st.o[n][4 * jj + e + 1][i], st.o[n][4 * jj + e + 1][2 + i]);
          if (g == 0) *reinterpret_cast<float2 *>(dst + kDim) = make_float2(st.m[n][i], st.l[n][i]);
        }
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int lr = 8 * n + 2 * t + i;
          const float *src = js + lr * C::kPartFloats;
          float2 ml[3];
          float m = st.m[n][i];
#pragma unroll
          for (int w = 0; w < 3; ++w) {
            ml[w] = *reinterpret_cast<const float2 *>(src + w * kRows * C::kPartFloats + kDim);
            m = fmaxf(m, ml[w].x);
          }
          const float f0 = ex2(st.m[n][i] - m);
          float l = f0 * st.l[n][i], fw[3];
#pragma unroll
          for (int w = 0; w < 3; ++w) {
            fw[w] = ex2(ml[w].x - m);
            l += fw[w] * ml[w].y;
          }
          const bool has = row0 + lr < rows_all;
          const float inv = l > 0.0f || l != l ? p.v_scale / l : 0.0f;
#pragma unroll
          for (int jj = 0; jj < kDim / 64; ++jj) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[2 * e] = f0 * st.o[n][4 * jj + e][i];
              v[2 * e + 1] = f0 * st.o[n][4 * jj + e][2 + i];
            }
            const int col = 64 * jj + 8 * pg;
#pragma unroll
            for (int w = 0; w < 3; ++w) {
              const float4 x = *reinterpret_cast<const float4 *>(src + w * kRows * C::kPartFloats + col);
              const float4 y = *reinterpret_cast<const float4 *>(src + w * kRows * C::kPartFloats + col + 4);
              const float u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaf(fw[w], u[e], v[e]);
            }
            if (!has) continue;
            if (whole) {
              if (col < p.head_dim) {
                const long long tok = c.q.q0 + p.by_group(row0 + lr);
                const int hq = c.head * p.group + (row0 + lr - p.by_group(row0 + lr) * p.group);
                *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.out) +
                                           ((tok * (p.group * p.kv_heads) + hq) * p.head_dim + col) * 2) =
                    packed8(v, inv, out_bf16);
              }
            } else {
              float *dst = part + lr * C::kPartFloats + col;
              *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<float4 *>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
          if (g == 0 && has) {
            if (whole) store_lse(p, c.q, c.head, row0 + lr, m, l);
            else *reinterpret_cast<float2 *>(part + lr * C::kPartFloats + kDim) = make_float2(m, l);
          }
        }
    }
    if (!whole) {
      // CTAs whose runs hold tiles of this group
      const long long first = ((c.gs + 1) * grid - 1) / total;
      const long long last = ((c.gs + c.sp.tiles) * grid - 1) / total;
      ptx::grid_dep_wait();   // the counters are zero from here on
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(p.tickets + first, 1u) == static_cast<u32>(last - first);
      __syncthreads();
      if (s_last) {
        // some rows at a time: the parts' (m, l), their factors, then the sums
        // over the parts, whose loads do not wait for one another
        __threadfence();
        const int rows_here = min(kRows, rows_all - row0);
        const int parts = static_cast<int>(last - first) + 1;
        float *const factor = js;   // [rows][parts]
        const int at_once = max(1, min(4, C::kJoinBytes / 4 / parts));   // (parts: the launch's grid at most)
        __shared__ float2 s_ml[4];
        auto part_at = [&](int k, int lr) {
          return p.part + (((first + k) * 2 + (k == 0 ? 1 : 0)) * kRows + lr) *
                              static_cast<long long>(C::kPartFloats);
        };
        for (int lr0 = 0; lr0 < rows_here; lr0 += at_once) {
          const int rows = min(at_once, rows_here - lr0);
          __syncthreads();
          if (warp < rows) {
            float m = kColsNone, l = 0.0f;
            for (int k = lane; k < parts; k += 32) {
              const float pm = __ldcg(part_at(k, lr0 + warp) + kDim);
              factor[warp * parts + k] = pm;
              m = fmaxf(m, pm);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            for (int k = lane; k < parts; k += 32) {
              const float f2 = ex2(factor[warp * parts + k] - m);
              factor[warp * parts + k] = f2;
              l += f2 * __ldcg(part_at(k, lr0 + warp) + kDim + 1);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) s_ml[warp] = make_float2(m, l);
          }
          __syncthreads();
          for (int u = tid; u < rows * (kDim / 2); u += kAttendThreads) {
            const int lr = u / (kDim / 2), col = u % (kDim / 2) * 2;
            const float *fr = factor + lr * parts;
            float o0 = 0.0f, o1 = 0.0f;
#pragma unroll 8
            for (int k = 0; k < parts; ++k) {
              const float2 o = __ldcg(reinterpret_cast<const float2 *>(part_at(k, lr0 + lr) + col));
              o0 += fr[k] * o.x;
              o1 += fr[k] * o.y;
            }
            const float m = s_ml[lr].x, l = s_ml[lr].y;
            const float inv = l > 0.0f || l != l ? p.v_scale / l : 0.0f;
            if (col < p.head_dim)
              store_out(p, c.q, c.head, row0 + lr0 + lr, col, o0 * inv, o1 * inv, out_bf16);
            if (col == 0) store_lse(p, c.q, c.head, row0 + lr0 + lr, m, l);
          }
        }
      }
    }
    if (c.after() >= b) break;
    __syncthreads();   // js, s_group, s_rows and s_last are free again
    if (tid == 0) s_group.open(p, s_group.after(), b, kRows);
    __syncthreads();
  }
  cp_async_wait<0>();
  ptx::grid_dep_wait();
}

}  // namespace kvcs
