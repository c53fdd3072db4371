// kvcs_attend.cuh -- attention of a few new tokens over a paged cache
// (decode, drafted tokens, and every geometry the tensor-memory kernel does
// not take): work split over the cache's length.
//
// For query row i (one new token under one query head) with visible tokens j,
//     z_ij = score(q_i . k_j),  m_i = max_j z_ij,  l_i = sum_j 2^(z_ij - m_i),
//     o_i = sum_j 2^(z_ij - m_i) v_j / l_i,        lse_i = ln 2 (m_i + log2 l_i),
// in one pass over K and V: m, l and o are running values, rescaled when m
// grows; partial (m, l, o) of parts of the cache join by the same rule.
//
// Bound: a decode step reads every cached K and V once for 2 * group
// multiply-adds a value, so DRAM bandwidth is the floor.  The rows of one KV
// head's query group share each K and V value (16 rows a warp, filled with
// zeros past the group), and the products run on mma.sync, whose rate such
// shapes leave mostly idle: tensor-memory accumulators would only add
// latency here.
//
// Split: the tiles of kTileKeys tokens of all (request, row tile, KV head)
// groups form one line, cut into equal runs, one per CTA, whatever the
// requests' lengths.  A group inside one run is finished by its CTA; a group
// that crosses runs leaves partial (m, l, o) in the workspace, and the last
// of its CTAs to arrive (a counter per group, zeroed by a small kernel that
// runs ahead) joins them in CTA order, so results do not depend on timing.
//
// kWide = false (up to 16 rows a group): the four warps of a CTA take 16
// tokens of a tile each, with their own (m, l, o) and their own ring of
// cp.async stages, so the loop has no CTA barrier; they join at the group's
// end.  kWide = true (up to 64 rows a tile): the warps take 16 rows each and
// share the tile's tokens.
//
// Fragments: a product's inner index may run in any order as long as both
// operands agree, so every lane reads whole 16-byte chunks of shared memory
// and takes its fragment values from them: K chunk 4b + t of its key gives
// the B values of two k-steps (lane = 4 g + t), and V chunks of the four keys
// t, t + 4, t + 8, t + 12 give, after byte permutes, the B values of eight
// n-tiles.  Chunks are stored XORed with the row index; keys and V columns
// are assigned to lanes so that the eight lanes of a shared-memory phase hit
// different banks for 128- and 256-byte rows.
//
// Measured: 64 requests of 512 to 4096 tokens (8 KV heads of 128, bf16, one
// token each) 116 us, 5.2 TB/s, where reading the same pages without any
// arithmetic takes 106; fp8 with 64 query heads, 128 requests of 2048, 139 us
// (3.9 TB/s; conversions and products, not DRAM, set that pace: 125 us with
// the copies left out); two requests of 99,001 and 131,072 tokens with three
// drafted ones 168 us, 5.6 TB/s; one request of 709 tokens 12 us.  Two CTAs an
// SM with three stages; three CTAs with two stages took 114, 143 and 208 us.
#pragma once

#include "kvcs_attn_common.cuh"

namespace kvcs {

constexpr int kAttendThreads = 128;
constexpr int kTileKeys = 64;
constexpr int kChunkKeys = 16;   // tokens a warp takes at once
constexpr float kNegInf = -__builtin_huge_valf();

template <int kType, int kDim>
struct AttendShape {
  static constexpr int kElem = kType == kKvFp8 ? 1 : 2;
  static constexpr int kRowBytes = kDim * kElem;            // of one token's K or V
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kChunkBytes = kChunkKeys * kRowBytes;  // K (or V) of 16 tokens
  static constexpr int kStageBytes = kTileKeys / kChunkKeys * 2 * kChunkBytes;
  static constexpr int kStages = kStageBytes >= 65536 ? 3 : kStageBytes >= 32768 ? 3 : 4;
  static constexpr int kRows = 16;
  static constexpr int kPartFloats = kDim + 2;               // o, m, l of a row
  static constexpr int kJoinBytes = 4 * 16 * (kDim + 4) * 4;  // four warps' (m, l, o)
  static constexpr int kRingBytes =
      kStages * kStageBytes > kJoinBytes ? kStages * kStageBytes : kJoinBytes;
  static constexpr int kSmemBytes = kRingBytes;
};

// Rows of a row tile.
__host__ __device__ constexpr int attend_rows(bool wide) { return wide ? 64 : 16; }

// A request's share of the line of tiles.
struct GroupSpan {
  int row_tiles;
  int lo;            // first tile
  int tiles;         // tiles per (row tile, head)
  long long total;   // tiles of the request
};

__device__ __forceinline__ GroupSpan span_of(const AttnParams &p, const Request &q, int rows) {
  GroupSpan s;
  s.row_tiles = 0;
  s.lo = 0;
  s.tiles = 0;
  s.total = 0;
  const long long r = static_cast<long long>(q.n) * p.group;
  if (r < p.row_lo || r > p.row_hi || q.n == 0) return s;
  s.row_tiles = static_cast<int>((r + rows - 1) / rows);
  int first = 0;
  if (p.window > 0) first = max(0, q.at - p.window + 1);
  const int end = min(q.keys, max(0, q.at + q.n));
  s.lo = first / kTileKeys;
  const int hi = (end + kTileKeys - 1) / kTileKeys;
  s.tiles = max(1, hi - s.lo);   // rows that see nothing are still written
  s.total = static_cast<long long>(s.row_tiles) * s.tiles * p.kv_heads;
  return s;
}

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long *total, long long *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  return before + inc - v;
}

// What is taken off a running maximum, in units of log 2.  Weights 2^(z - m)
// are multiplied in 16 bits.  In fp16 they lose bits below 2^-14 and vanish
// below 2^-25, while l counts them whole: with one token far above a long tail,
// the tail's share of the output would be lost.  Made 2^14 times larger (the
// largest weight is 2^14 then, of 65504) they vanish below 2^-39 of the largest
// only; l grows alike, so the quotient and the log-sum-exp stay.  bf16 has
// 32-bit floats' exponents.
template <int kType>
constexpr float kLift = kType == kKvBf16 ? 0.0f : 14.0f;

// Running state of the 16 rows of a warp: lane 4 g + t holds rows g and g + 8.
template <int kDim>
struct RowState {
  float m[2], l[2];
  float o[kDim / 8][4];   // n-tile 8 jj + e: row g, columns c(0), c(1); row g + 8 likewise
};

// Column of the output that lane t holds in n-tile 8 jj + e, value i (0, 1).
__device__ __forceinline__ int out_column(int tile, int t, int i) {
  return (tile >> 3) * 64 + 8 * (t + 4 * i) + (tile & 7);
}

// One chunk of 16 tokens against a warp's 16 rows.
template <int kType, int kDim>
__device__ __forceinline__ void attend_chunk(const AttnParams &p, const u32 (&qf)[kDim / 8][2],
                                             RowState<kDim> &st, u32 ks, u32 vs, u32 valid,
                                             int key0, const int (&at)[2], int at_min, int at_max,
                                             const float (&rs)[2]) {
  using S = AttendShape<kType, kDim>;
  constexpr bool kBf16 = kType == kKvBf16;
  constexpr int kMask = (S::kChunks < 8 ? S::kChunks : 8) - 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int pg = (g >> 1) | ((g & 1) << 2);   // key (and V chunk) of lane group g
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  float s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // (two chains of products each)
  // Piece 4 b + t of row pg (or pg + 8) lies at piece (4 b + t) ^ (row & mask):
  // two places, for even and odd b, from which the others differ by constants.
  const u32 k_even = ks + pg * S::kRowBytes + ((t ^ (pg & kMask)) << 4);
  const u32 k_odd = ks + pg * S::kRowBytes + (((t + 4) ^ (pg & kMask)) << 4);
  if constexpr (kType == kKvFp8) {
#pragma unroll
    for (int b = 0; b < kDim / 64; ++b) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 k = lds128((b & 1 ? k_odd : k_even) + (b >> 1) * 128 + j * 8 * S::kRowBytes);
        const u32 w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u32 lo, hi;
          fp8x4_to_half(w[i], lo, hi);
          const int step = 4 * b + i;
          mma16816<false>(i & 1 ? s2[j] : s[j], qf[2 * step][0], qf[2 * step][1],
                          qf[2 * step + 1][0], qf[2 * step + 1][1], lo, hi);
        }
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < kDim / 32; ++b) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 k = lds128((b & 1 ? k_odd : k_even) + (b >> 1) * 128 + j * 8 * S::kRowBytes);
        mma16816<kBf16>(s[j], qf[4 * b][0], qf[4 * b][1], qf[4 * b + 1][0], qf[4 * b + 1][1], k.x,
                        k.y);
        mma16816<kBf16>(s2[j], qf[4 * b + 2][0], qf[4 * b + 2][1], qf[4 * b + 3][0],
                        qf[4 * b + 3][1], k.z, k.w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] += s2[j][i];
  // scores = sc * s; capped ones, and those of a scale that would turn the
  // maximum round or make NaN of a masked score, are made first
  float sc[2] = {rs[0] * p.scale, rs[1] * p.scale};
  if constexpr (kType == kKvFp8) {
    // (a row's factor may underflow: 0 would make NaN of a masked score too)
    sc[0] = fmaxf(sc[0], __int_as_float(1));
    sc[1] = fmaxf(sc[1], __int_as_float(1));
  }
  if (p.cap != 0.0f || p.scale <= 0.0f) {
    scores_of(p, s, rs);
    sc[0] = sc[1] = 1.0f;
  }
  // s[j][2 r + i]: row g + 8 r, token j * 8 + t + 4 i
  const bool partly = valid != 0xffffu || key0 + kChunkKeys - 1 > at_min ||
                      (p.window > 0 && key0 <= at_max - p.window);
  if (partly) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kk = j * 8 + t + 4 * (i & 1), a = at[i >> 1];
        const bool see = (valid >> kk & 1u) && key0 + kk <= a &&
                         (p.window == 0 || key0 + kk > a - p.window);
        if (!see) s[j][i] = kNegInf;
      }
  }
  float mx[2], base[2], scale[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float v = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    mx[r] = fmaxf(st.m[r], v * sc[r] - kLift<kType>);
    base[r] = mx[r] == kNegInf ? 0.0f : mx[r];
  }
  if (__any_sync(0xffffffffu, mx[0] != st.m[0] || mx[1] != st.m[1])) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      scale[r] = ex2(st.m[r] - base[r]);
      st.l[r] *= scale[r];
      st.m[r] = mx[r];
    }
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) {
      st.o[n][0] *= scale[0];
      st.o[n][1] *= scale[0];
      st.o[n][2] *= scale[1];
      st.o[n][3] *= scale[1];
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[j][i] = ex2(fmaf(s[j][i], sc[i >> 1], -base[i >> 1]));
      st.l[i >> 1] += s[j][i];
    }
  // the weights as the A operand, rounded to the cache's 16-bit type (fp16 for
  // fp8 caches), which the products take: each by 2^-8 (2^-11) of itself at
  // most, as an output's own rounding; fp16 ones below 2^-28 of the largest by
  // up to 2^-39 of that
  const u32 a0 = pack2<kBf16>(s[0][0], s[0][1]), a1 = pack2<kBf16>(s[0][2], s[0][3]);
  const u32 a2 = pack2<kBf16>(s[1][0], s[1][1]), a3 = pack2<kBf16>(s[1][2], s[1][3]);
  u32 seen_bad = 0;   // a non-finite V value, in chunks that some row sees only partly
  // pieces 8 jj + pg of rows t + 4 k, as above: two places, for even and odd k
  // (fp8: 8-byte halves of pieces)
  const int vp = kType == kKvFp8 ? pg >> 1 : pg, vh = kType == kKvFp8 ? (pg & 1) << 3 : 0;
  const u32 v_even = vs + t * S::kRowBytes + ((vp ^ (t & kMask)) << 4) + vh;
  const u32 v_odd = vs + (t + 4) * S::kRowBytes + ((vp ^ ((t + 4) & kMask)) << 4) + vh;
#pragma unroll
  for (int jj = 0; jj < kDim / 64; ++jj) {
    u32 v[4][4];   // keys t + 4 k: eight values, as pairs
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u32 at = (k & 1 ? v_odd : v_even) + (k >> 1) * 8 * S::kRowBytes;
      if constexpr (kType == kKvFp8) {
        // jj moves by 4 pieces: bit 2 of the XORed place
        const u32 flip = ((jj & 1) << 6);
        const uint2 w = lds64((S::kChunks >= 8 ? vs + (((at - vs) ^ flip)) : at) + (jj >> 1) * 128);
        fp8x4_to_half(w.x, v[k][0], v[k][1]);
        fp8x4_to_half(w.y, v[k][2], v[k][3]);
      } else {
        const uint4 w = lds128(at + jj * 128);
        v[k][0] = w.x;
        v[k][1] = w.y;
        v[k][2] = w.z;
        v[k][3] = w.w;
      }
    }
    if (partly) {
      constexpr u32 kExp = kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          seen_bad |= (v[k][e] & kExp) == kExp || (v[k][e] >> 16 & kExp) == kExp;
    }
    if (partly && __any_sync(0xffffffffu, seen_bad)) {
      // A weight of 0 times a non-finite value is NaN: add the chunk's
      // values one token at a time, and only to the rows that see it.
#pragma unroll 1
      for (int kk = 0; kk < kChunkKeys; ++kk) {
        const int src = g * 4 + (kk & 3), hi = kk >> 2 & 1;
        const float w0 = __shfl_sync(0xffffffffu, kk < 8 ? (hi ? s[0][1] : s[0][0])
                                                         : (hi ? s[1][1] : s[1][0]), src);
        const float w1 = __shfl_sync(0xffffffffu, kk < 8 ? (hi ? s[0][3] : s[0][2])
                                                         : (hi ? s[1][3] : s[1][2]), src);
        const bool ok = valid >> kk & 1u;
        const bool see0 = ok && key0 + kk <= at[0] && (p.window == 0 || key0 + kk > at[0] - p.window);
        const bool see1 = ok && key0 + kk <= at[1] && (p.window == 0 || key0 + kk > at[1] - p.window);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = out_column(8 * jj + e, t, i);
            float x;
            if constexpr (kType == kKvFp8) {
              u32 raw;
              const u32 a = vs + kk * S::kRowBytes + (((col >> 4) ^ (kk & kMask)) << 4) + (col & 15);
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(raw) : "r"(a));
              u32 lo, up;
              fp8x4_to_half(raw, lo, up);
              x = half_bits_to_float(lo & 0xffffu, false);
            } else {
              u32 raw;
              const u32 a = vs + kk * S::kRowBytes + (((col >> 3) ^ (kk & kMask)) << 4) +
                            (col & 7) * 2;
              asm volatile("ld.shared.u16 %0, [%1];" : "=r"(raw) : "r"(a));
              x = half_bits_to_float(raw & 0xffffu, kBf16);
            }
            if (see0) st.o[8 * jj + e][i] += w0 * x;
            if (see1) st.o[8 * jj + e][2 + i] += w1 * x;
          }
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const u32 sel = e & 1 ? 0x7632u : 0x5410u;
      const u32 b0 = __byte_perm(v[0][e >> 1], v[1][e >> 1], sel);
      const u32 b1 = __byte_perm(v[2][e >> 1], v[3][e >> 1], sel);
      mma16816<kBf16>(st.o[8 * jj + e], a0, a1, a2, a3, b0, b1);
    }
  }
}

// The rows of a warp as A fragments, read straight from global memory: word
// pairs of the lane's 16-byte (fp8: 32-byte) pieces.  fp8 caches multiply in
// fp16: bf16 queries are brought near 1 by a power of two per row (returned
// in rs), so only values 2^-24 below the row's largest are lost.
template <int kType, int kDim>
__device__ __forceinline__ void load_queries(const AttnParams &p, const Request &q, int head,
                                             const int (&row)[2], bool (&has)[2],
                                             u32 (&qf)[kDim / 8][2], float (&rs)[2]) {
  const int t = threadIdx.x & 3;
  const unsigned char *base = static_cast<const unsigned char *>(p.q);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    rs[r] = 1.0f;
    const long long tok = q.q0 + p.by_group(row[r]);
    const int hq = head * p.group + (row[r] - p.by_group(row[r]) * p.group);
    const unsigned char *src =
        base + (tok * p.q_stride + static_cast<long long>(hq) * p.head_dim) * 2;
    constexpr int kPiece = kType == kKvFp8 ? 16 : 8;   // elements a lane takes at once
#pragma unroll
    for (int b = 0; b < kDim / (4 * kPiece); ++b) {
      const int d = (4 * b + t) * kPiece;
#pragma unroll
      for (int h = 0; h < kPiece / 8; ++h) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (has[r] && d + 8 * h < p.head_dim)
          v = __ldg(reinterpret_cast<const uint4 *>(src + (d + 8 * h) * 2));
        const int w = (kPiece / 2) * b + 4 * h;   // word pairs of the lane, in order
        qf[w][r] = v.x;
        qf[w + 1][r] = v.y;
        qf[w + 2][r] = v.z;
        qf[w + 3][r] = v.w;
      }
    }
    if (kType == kKvFp8 && p.q_bf16) {
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kDim / 8; ++w)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[w][r] << 16)),
                               fabsf(__uint_as_float(qf[w][r] & 0xffff0000u))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = top > 0.0f && top < __builtin_huge_valf() ? ilogbf(top) : 0;
      rs[r] = ldexpf(1.0f, ex < -126 ? -126 : ex);
      const float inv = ldexpf(1.0f, ex < -126 ? 126 : -ex);
#pragma unroll
      for (int w = 0; w < kDim / 8; ++w)
        qf[w][r] = pack2<false>(__uint_as_float(qf[w][r] << 16) * inv,
                                __uint_as_float(qf[w][r] & 0xffff0000u) * inv);
    }
  }
}

// How a warp's lanes share the 16-byte pieces of a chunk of 16 tokens: kAcross
// lanes side by side on a row (128 bytes, or a shorter row), 32 / kAcross rows
// at once.  A lane's pieces then differ by constants, in global memory and,
// with the XOR of the row index, in shared memory too.
template <int kType, int kDim>
struct ChunkLanes {
  using S = AttendShape<kType, kDim>;
  static constexpr int kAcross = S::kChunks < 8 ? S::kChunks : 8;
  static constexpr int kDown = 32 / kAcross;                // rows at once: 4 or 8
  static constexpr int kTurns = kChunkKeys / kDown;         // groups of rows
  static constexpr int kSpans = S::kChunks / kAcross;       // spans of kAcross pieces

  // A lane's first piece, from the chunk's start; turn j, span k follow at
  // (first ^ flip(j)) + place(j, k).
  static __device__ __forceinline__ u32 first() {
    const int lane = threadIdx.x & 31, r = lane / kAcross, a = lane % kAcross;
    return r * S::kRowBytes + ((a ^ (r & (kAcross - 1))) << 4);
  }
  static constexpr __device__ u32 flip(int j) { return kDown == 4 ? (j & 1) << 6 : 0; }
  static constexpr __device__ u32 place(int j, int k) { return j * kDown * S::kRowBytes + k * 128; }
};

// A chunk whose 16 tokens lie in one page, one after another, all readable.
template <int kType, int kDim>
__device__ __forceinline__ void load_run(const AttnParams &p, u32 chunk, u32 first,
                                         const unsigned char *src) {
  using S = AttendShape<kType, kDim>;
  using L = ChunkLanes<kType, kDim>;
  const unsigned char *v = src + p.map.half_stride;
  const long long down = static_cast<long long>(L::kDown) * p.map.slot_stride;
  if (p.map.chunk_stride == 16) {   // (spans are then 128 bytes apart: no address arithmetic)
#pragma unroll
    for (int j = 0; j < L::kTurns; ++j, src += down, v += down)
#pragma unroll
      for (int k = 0; k < L::kSpans; ++k) {
        const u32 d = chunk + (first ^ L::flip(j)) + L::place(j, k);
        cp_async16(d, src + k * 128, 16);
        cp_async16(d + S::kChunkBytes, v + k * 128, 16);
      }
  } else {
    const long long step = static_cast<long long>(L::kAcross) * p.map.chunk_stride;
#pragma unroll
    for (int j = 0; j < L::kTurns; ++j, src += down, v += down)
#pragma unroll
      for (int k = 0; k < L::kSpans; ++k) {
        const u32 d = chunk + (first ^ L::flip(j)) + L::place(j, k);
        cp_async16(d, src + k * step, 16);
        cp_async16(d + S::kChunkBytes, v + k * step, 16);
      }
  }
}

// Any chunk; returns its mask of readable tokens.  Tokens outside [lo, hi)
// and tokens of bad blocks become zeros.
template <int kType, int kDim>
__device__ __noinline__ u32 load_any(const AttnParams &p, long long pos0, int head, u32 chunk,
                                     int key0, int lo, int hi) {
  using S = AttendShape<kType, kDim>;
  using L = ChunkLanes<kType, kDim>;
  const int lane = threadIdx.x & 31;
  const u32 first = L::first();
  const int row_bytes = p.head_dim * S::kElem;
  u32 mask = 0;
#pragma unroll 1
  for (int j = 0; j < L::kTurns; ++j) {
    const int row = j * L::kDown + lane / L::kAcross, key = key0 + row;
    bool ok = key >= lo && key < hi;
    long long off = 0;
    if (ok) {
      const int pos = p.map.by_block(key);
      const int block = p.tab.block_ids[pos0 + pos];
      if (block < 0 || block >= p.map.num_blocks) {
        ok = false;
        raise(p.tab, kStatusBadBlockId);
      } else {
        off = token_offset(p.map, block, key - pos * p.map.block_size, head);
      }
    }
    const u32 good = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int r = 0; r < L::kDown; ++r) mask |= (good >> (r * L::kAcross) & 1u) << (j * L::kDown + r);
#pragma unroll 1
    for (int k = 0; k < L::kSpans; ++k) {
      const int c = k * L::kAcross + lane % L::kAcross, left = ok ? row_bytes - c * 16 : 0;
      const u32 d = chunk + (first ^ L::flip(j)) + L::place(j, k);
      const unsigned char *src =
          p.map.base + (left > 0 ? off + static_cast<long long>(c) * p.map.chunk_stride : 0);
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

// Final values of one row: o / l, the log-sum-exp, in the output's type.
__device__ __forceinline__ void store_out(const AttnParams &p, const Request &q, int head, int row,
                                          int col, float a, float b, bool bf16) {
  const long long tok = q.q0 + p.by_group(row);
  const int hq = head * p.group + (row - p.by_group(row) * p.group);
  unsigned char *dst = static_cast<unsigned char *>(p.out) +
                       ((tok * (p.group * p.kv_heads) + hq) * p.head_dim + col) * 2;
  *reinterpret_cast<u32 *>(dst) = bf16 ? pack2<true>(a, b) : pack2<false>(a, b);
}

__device__ __forceinline__ void store_lse(const AttnParams &p, const Request &q, int head, int row,
                                          float m, float l) {
  if (!p.lse) return;
  const long long tok = q.q0 + p.by_group(row);
  const int hq = head * p.group + (row - p.by_group(row) * p.group);
  p.lse[tok * (p.group * p.kv_heads) + hq] = l == 0.0f ? kNegInf : kLn2 * (m + log2f(l));
}

template <int kType, int kDim, bool kWide>
__global__ void __launch_bounds__(kAttendThreads)
    kvcs_attend_kernel(const __grid_constant__ AttnParams p) {
  using S = AttendShape<kType, kDim>;
  extern __shared__ __align__(1024) unsigned char attend_smem[];   // (pieces' places are XORed)
  __shared__ long long s_scan[4];
  __shared__ u32 s_mask[S::kStages][4];
  __shared__ int s_last;
  constexpr int kRows = attend_rows(kWide);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const long long R = p.tab.num_requests;

  // the line of tiles: its length, then the request this CTA's run starts in
  long long sum = 0;
  for (long long r = tid; r < R; r += kAttendThreads)
    sum += span_of(p, read_request(p.tab, r, p.map.block_size, blockIdx.x == 0), kRows).total;
  long long total;
  const long long ahead_of_me = block_scan(sum, &total, s_scan);
  const long long grid = min(static_cast<long long>(gridDim.x), total);
  if (blockIdx.x >= grid) {
    ptx::grid_dep_wait();
    return;
  }
  const long long a = total * blockIdx.x / grid, b = total * (blockIdx.x + 1ll) / grid;
  long long before = 0, r = 0;
  __shared__ long long s_req[2];
  for (long long c = 0;; c += kAttendThreads) {
    const long long rr = c + tid;
    long long v = sum, all = total, ex = ahead_of_me;
    if (R > kAttendThreads) {   // (otherwise the first scan tells)
      v = rr < R ? span_of(p, read_request(p.tab, rr, p.map.block_size, false), kRows).total : 0;
      ex = before + block_scan(v, &all, s_scan);
    }
    if (before + all > a) {
      if (v > 0 && ex <= a && a < ex + v) {
        s_req[0] = rr;
        s_req[1] = ex;
      }
      __syncthreads();
      r = s_req[0];
      before = s_req[1];
      break;
    }
    before += all;
  }

  Request q = read_request(p.tab, r, p.map.block_size, false);
  GroupSpan sp = span_of(p, q, kRows);
  const u32 ring = ptx::smem_addr(attend_smem);
  const u32 lane_first = ChunkLanes<kType, kDim>::first();
  const bool out_bf16 = kType == kKvBf16 || (kType == kKvFp8 && p.q_bf16);

  for (long long x = a; x < b;) {
    while (x >= before + sp.total) {   // next request with tiles here
      before += sp.total;
      ++r;
      q = read_request(p.tab, r, p.map.block_size, false);
      sp = span_of(p, q, kRows);
    }
    const long long w = x - before;
    const long long grp = w / sp.tiles;               // (row tile, head) of the request
    const int k0 = static_cast<int>(w - grp * sp.tiles);
    const long long gs = before + grp * sp.tiles;      // the group's first tile
    const int k1 = static_cast<int>(min(static_cast<long long>(sp.tiles), b - gs));
    const int head = static_cast<int>(grp % p.kv_heads);
    const int rt = static_cast<int>(grp / p.kv_heads);
    const bool whole = k0 == 0 && k1 == sp.tiles;
    x = gs + k1;

    // rows of this warp, and what they see
    const int rows_all = q.n * p.group;
    const int row0 = rt * kRows + (kWide ? warp * 16 : 0);
    int row[2], at[2];
    bool has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = row0 + g + 8 * i;
      has[i] = rr < rows_all;
      row[i] = has[i] ? rr : rows_all - 1;   // spare rows repeat the last one
      at[i] = q.at + p.by_group(row[i]);
    }
    const int warp_last = min(row0 + 15, rows_all - 1);
    const int at_min = q.at + min(row0, rows_all - 1) / p.group;
    const int at_max = q.at + warp_last / p.group;
    // tokens some row of the tile sees
    const int tile_first = q.at + (rt * kRows) / p.group;
    const int tile_last = q.at + min(rt * kRows + kRows - 1, rows_all - 1) / p.group;
    const int lo = p.window > 0 ? max(0, tile_first - p.window + 1) : 0;
    const int hi = min(q.keys, tile_last + 1);
    const int c0 = max(k0, lo / kTileKeys - sp.lo);
    const int c1 = min(k1, (max(hi, 0) + kTileKeys - 1) / kTileKeys - sp.lo);

    u32 qf[kDim / 8][2];
    float rs[2];
    load_queries<kType, kDim>(p, q, head, row, has, qf, rs);
    RowState<kDim> st;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      st.m[i] = kNegInf;
      st.l[i] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[n][i] = 0.0f;

    // The ring: a stage holds a tile, in its chunks' order.  The block of a
    // chunk is looked up a tile ahead of its copies.
    auto stage_at = [&](int stage, int chunk) {
      return ring + stage * S::kStageBytes + chunk * 2 * S::kChunkBytes;
    };
    const bool runs = p.runs && lo <= (sp.lo + c0) * kTileKeys;
    using L = ChunkLanes<kType, kDim>;
    const long long lane_src = static_cast<long long>(lane / L::kAcross) * p.map.slot_stride +
                               (lane % L::kAcross) * static_cast<long long>(p.map.chunk_stride) +
                               head * p.map.head_stride;
    auto block_of = [&](int k) {
      const int key = (sp.lo + k) * kTileKeys + warp * kChunkKeys;
      return runs && k < c1 && key + kChunkKeys <= hi ? p.tab.block_ids[q.pos0 + p.map.by_block(key)]
                                                      : -1;
    };
    int ahead = block_of(c0), put = 0;
    auto fetch = [&](int k) {
      if (k < c1) {
        const int key = (sp.lo + k) * kTileKeys + warp * kChunkKeys;
        const int block = ahead;
        ahead = block_of(k + 1);
        const u32 dst = stage_at(put, warp);
        u32 mask = 0xffffu;
        if (block >= 0 && block < p.map.num_blocks) {
          const int slot = key - p.map.by_block(key) * p.map.block_size, sub = p.map.by_sub(slot);
          load_run<kType, kDim>(p, dst, lane_first, p.map.base + block * p.map.block_stride +
                                            sub * p.map.sub_stride +
                                            static_cast<long long>(slot - sub * p.map.kbs) *
                                                p.map.slot_stride + lane_src);
        } else {
          mask = load_any<kType, kDim>(p, q.pos0, head, dst, key, lo, hi);
        }
        if (lane == 0) s_mask[put][warp] = mask;
        put = put + 1 == S::kStages ? 0 : put + 1;
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int k = 0; k < S::kStages - 1; ++k) fetch(c0 + k);
    int stage = 0;
    for (int k = c0; k < c1; ++k) {
      cp_async_wait<S::kStages - 2>();
      if (kWide) __syncthreads(); else __syncwarp();
      fetch(k + S::kStages - 1);
      const int key0 = (sp.lo + k) * kTileKeys;
      if (kWide) {
        if (row0 < rows_all) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int kc = key0 + c * kChunkKeys;
            if (kc > at_max || (p.window > 0 && kc + kChunkKeys - 1 <= at_min - p.window)) continue;
            attend_chunk<kType, kDim>(p, qf, st, stage_at(stage, c), stage_at(stage, c) + S::kChunkBytes,
                                      s_mask[stage][c], kc, at, at_min, at_max, rs);
          }
        }
      } else {
        attend_chunk<kType, kDim>(p, qf, st, stage_at(stage, warp),
                                  stage_at(stage, warp) + S::kChunkBytes, s_mask[stage][warp],
                                  key0 + warp * kChunkKeys, at, at_min, at_max, rs);
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 1);
      st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 2);
    }

    float *const part_of_cta =
        p.part + static_cast<long long>(blockIdx.x) * 2 * kRows * S::kPartFloats;
    float *const part = part_of_cta + (k0 == 0 ? 1 : 0) * kRows * S::kPartFloats;
    if (kWide) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lr = warp * 16 + g + 8 * i;
        if (!has[i]) continue;
        if (whole) {
          const float inv = st.l[i] > 0.0f || st.l[i] != st.l[i] ? p.v_scale / st.l[i] : 0.0f;
#pragma unroll
          for (int n = 0; n < kDim / 8; n += 2)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = out_column(n, t, c);
              if (col < p.head_dim)
                store_out(p, q, head, row[i], col, st.o[n][2 * i + c] * inv,
                          st.o[n + 1][2 * i + c] * inv, out_bf16);
            }
          if (t == 0) store_lse(p, q, head, row[i], st.m[i], st.l[i]);
        } else {
          float *dst = part + lr * S::kPartFloats;
#pragma unroll
          for (int n = 0; n < kDim / 8; n += 2)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<float2 *>(dst + out_column(n, t, c)) =
                  make_float2(st.o[n][2 * i + c], st.o[n + 1][2 * i + c]);
          if (t == 0) *reinterpret_cast<float2 *>(dst + kDim) = make_float2(st.m[i], st.l[i]);
        }
      }
    } else {
      // join the four warps' (m, l, o) in shared memory (the ring is drained)
      __syncthreads();
      float *js = reinterpret_cast<float *>(attend_smem);
      constexpr int kJ = kDim + 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float *dst = js + (warp * 16 + g + 8 * i) * kJ;
#pragma unroll
        for (int n = 0; n < kDim / 8; n += 2)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<float2 *>(dst + out_column(n, t, c)) =
                make_float2(st.o[n][2 * i + c], st.o[n + 1][2 * i + c]);
        if (t == 0) *reinterpret_cast<float2 *>(dst + kDim) = make_float2(st.m[i], st.l[i]);
      }
      __syncthreads();
      const int rows_here = min(kRows, rows_all - rt * kRows);
      for (int u = tid; u < rows_here * (kDim / 2); u += kAttendThreads) {
        const int lr = u / (kDim / 2), col = u % (kDim / 2) * 2;
        float m = kNegInf;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, js[(k * 16 + lr) * kJ + kDim]);
        const float mb = m == kNegInf ? 0.0f : m;
        float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float *src = js + (k * 16 + lr) * kJ;
          const float f = ex2(src[kDim] - mb);
          l += f * src[kDim + 1];
          o0 += f * src[col];
          o1 += f * src[col + 1];
        }
        if (whole) {
          const float inv = l > 0.0f || l != l ? p.v_scale / l : 0.0f;
          if (col < p.head_dim)
            store_out(p, q, head, rt * kRows + lr, col, o0 * inv, o1 * inv, out_bf16);
          if (col == 0) store_lse(p, q, head, rt * kRows + lr, m, l);
        } else {
          float *dst = part + lr * S::kPartFloats;
          *reinterpret_cast<float2 *>(dst + col) = make_float2(o0, o1);
          if (col == 0) *reinterpret_cast<float2 *>(dst + kDim) = make_float2(m, l);
        }
      }
    }
    if (!whole) {
      // CTAs whose runs hold tiles of this group
      const long long first = ((gs + 1) * grid - 1) / total;
      const long long last = ((gs + sp.tiles) * grid - 1) / total;
      ptx::grid_dep_wait();   // the counters are zero from here on
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const u32 before_me = atomicAdd(p.tickets + first, 1u);
        s_last = before_me == static_cast<u32>(last - first);
      }
      __syncthreads();
      if (s_last) {
        // 16 rows at a time: the parts' (m, l), their factors, then the sums
        // over the parts, whose loads do not wait for one another
        __threadfence();
        const int rows_here = min(kRows, rows_all - rt * kRows);
        const int parts = static_cast<int>(last - first) + 1;
        float *const factor = reinterpret_cast<float *>(attend_smem);   // [16][parts]
        __shared__ float2 s_ml[16];
        auto part_at = [&](int c, int lr) {
          return p.part + (((first + c) * 2 + (c == 0 ? 1 : 0)) * kRows + lr) *
                              static_cast<long long>(S::kPartFloats);
        };
        for (int lr0 = 0; lr0 < rows_here; lr0 += 16) {
          const int rows = min(16, rows_here - lr0);
          __syncthreads();
          for (int lr = warp; lr < rows; lr += kAttendThreads / 32) {
            float m = kNegInf, l = 0.0f;
            for (int c = lane; c < parts; c += 32) {
              const float pm = __ldcg(part_at(c, lr0 + lr) + kDim);
              factor[lr * parts + c] = pm;
              m = fmaxf(m, pm);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float mb = m == kNegInf ? 0.0f : m;
            for (int c = lane; c < parts; c += 32) {
              const float f = ex2(factor[lr * parts + c] - mb);
              factor[lr * parts + c] = f;
              l += f * __ldcg(part_at(c, lr0 + lr) + kDim + 1);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) s_ml[lr] = make_float2(m, l);
          }
          __syncthreads();
          for (int u = tid; u < rows * (kDim / 2); u += kAttendThreads) {
            const int lr = u / (kDim / 2), col = u % (kDim / 2) * 2;
            const float *f = factor + lr * parts;
            float o0 = 0.0f, o1 = 0.0f;
#pragma unroll 8
            for (int c = 0; c < parts; ++c) {
              const float2 o = __ldcg(reinterpret_cast<const float2 *>(part_at(c, lr0 + lr) + col));
              o0 += f[c] * o.x;
              o1 += f[c] * o.y;
            }
            const float m = s_ml[lr].x, l = s_ml[lr].y;
            const float inv = l > 0.0f || l != l ? p.v_scale / l : 0.0f;
            if (col < p.head_dim)
              store_out(p, q, head, rt * kRows + lr0 + lr, col, o0 * inv, o1 * inv, out_bf16);
            if (col == 0) store_lse(p, q, head, rt * kRows + lr0 + lr, m, l);
          }
        }
      }
    }
    __syncthreads();   // the ring and s_last are free again
  }
  ptx::grid_dep_wait();
}

}  // namespace kvcs
