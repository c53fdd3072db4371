// kvcs_evict.cuh -- eviction of cached tokens by score, and the move of the
// kept ones to the front of the request's blocks.
//
// Per row (request, cache, KV head) with N cached tokens and a budget B < N:
// the first `sinks` and the last `recent` tokens stay, and of the others the
// B - sinks - recent with the greatest scores (equal scores: the lowest
// index).  Kept tokens move, in order, to tokens 0 .. B-1 of the target
// blocks, with their scores.
//
// Bound: the kept tokens' K and V are read and written once, so DRAM
// bandwidth is the floor; the scores are 1/128 of that.
//
// Two kernels.  kvcs_evict_select_kernel, a CTA per row, finds the kept
// tokens: scores (held in shared memory where they fit) become 32-bit keys
// whose unsigned order is the scores' order, four counting passes over 8-bit
// digits find the least key kept and how many tokens of exactly that key are,
// and one pass leaves a bit per token, the count of kept tokens ahead of each
// window, and the moved scores.  kvcs_evict_move_kernel moves the bytes.  Each
// 16-byte piece of a token moves independently of the others, so a row is
// split by halves and columns where rows are few (and, into fresh blocks, by
// windows); a CTA goes through the kept tokens of its columns in order.
//
// In place: the new token j comes from token src(j) >= j, both growing, so a
// write never lands on a token that a later step still reads.  A step's
// pieces are in registers before any of them is written (a CTA barrier), and
// the next step's loads are already on their way by then.
//
// Words: the new blocks' checksum words, sum_h m_h sum_p x_p (2 (t P + p) + 1)
// with t the token's new position, are added while the bytes pass through.
#pragma once

#include "kvcs_attn_common.cuh"

namespace kvcs {

constexpr int kEvictThreads = 256;
constexpr int kEvictWindow = 1024;   // tokens a step of either kernel looks over
constexpr int kEvictPieces = 8;      // pieces a thread moves at once

struct EvictCache {
  PageMap map;
  float *scores;      // [num_blocks][heads][block_size]
  u64 m0;             // checksum factor of local head 0
  int heads;
  int head_bytes;
  int first_row;      // first (cache, head) index of this cache in the launch
  int unit;           // bytes of a piece: 16, or 8 on 8-byte boundaries
  int parts;          // column groups per half
  int part_pieces;    // pieces of a column group (the last may hold fewer)
  FastDiv by_part;    // division by part_pieces
};

struct EvictParams {
  Tables tab;
  const long long *keep;
  const int *new_block_ids;   // or null: in place
  u64 *block_sums;            // or null
  u32 *bits;                  // [rows][bit_words]: kept tokens
  u32 *ahead;                 // [rows][windows]: kept tokens before each window
  long long bit_words, windows;
  long long num_blocks;       // smallest pool of the call
  int block_size;
  FastDiv by_block;
  int sinks, recent;
  int num_caches;
  int rows;                   // (cache, head) pairs of the launch
  int smem_tokens;            // scores that shared memory holds
  int halves_parts;           // most column groups of a row, over both halves
  int spans;                  // fresh blocks: CTAs that share a row's windows
  EvictCache c[kMaxCachesPerLaunch];
};

// Unsigned keys in the order of the scores; -0 equals 0, every NaN is the
// greatest.
__device__ __forceinline__ u32 score_key(u32 bits) {
  const float f = __uint_as_float(bits);
  if (f != f) return 0xffffffffu;
  const u32 b = __float_as_uint(f + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Tokens and budget of a request; false when it is to be left alone (bad
// tables or block ids, which are flagged if `report`).  Called by a whole CTA.
__device__ inline bool evict_request(const EvictParams &p, long long r, Request *q, int *budget,
                                     bool report) {
  const long long a = p.tab.pos_offsets[r], b = p.tab.pos_offsets[r + 1];
  const bool speak = report && threadIdx.x == 0;
  *q = read_tokens(p.tab, r, p.block_size, speak);
  const long long keep = p.keep[r];
  // tables read_tokens has refused hold no tokens and are left alone too
  if (keep < 0 && speak) raise(p.tab, kStatusBadRequests);
  const bool none = keep < 0 || q->keys == 0 || a < 0 || b > p.tab.total_positions;
  *budget = static_cast<int>(min(max(keep, 0ll), static_cast<long long>(q->keys)));
  bool bad = false;
  if (!none) {
    const int blocks = (q->keys + p.block_size - 1) / p.block_size;
    const int targets = (*budget + p.block_size - 1) / p.block_size;
    for (int i = threadIdx.x; i < blocks; i += blockDim.x) {
      const int id = p.tab.block_ids[q->pos0 + i];
      bad |= id < 0 || id >= p.num_blocks;
      if (p.new_block_ids && i < targets) {
        const int to = p.new_block_ids[q->pos0 + i];
        bad |= to < 0 || to >= p.num_blocks;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && speak) raise(p.tab, kStatusBadBlockId);
  return !none && !bad;
}

// Zeroes the checksum words of the blocks the call fills (in place: of every
// block that held a token).
__global__ void __launch_bounds__(256) kvcs_evict_zero_kernel(const __grid_constant__ EvictParams p) {
  for (long long r = blockIdx.x; r < p.tab.num_requests; r += gridDim.x) {
    Request q;
    int budget;
    if (evict_request(p, r, &q, &budget, false)) {
      const int *ids = (p.new_block_ids ? p.new_block_ids : p.tab.block_ids) + q.pos0;
      const int n = ((p.new_block_ids ? budget : q.keys) + p.block_size - 1) / p.block_size;
      for (int i = threadIdx.x; i < n; i += blockDim.x) p.block_sums[ids[i]] = 0;
    }
  }
}

// The cache of a launch's (cache, head) row.
__device__ __forceinline__ const EvictCache &cache_of_row(const EvictParams &p, int row) {
  int lo = 0, hi = p.num_caches - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.c[mid].first_row <= row) lo = mid; else hi = mid - 1;
  }
  return p.c[lo];
}

// Where a request's bits and window counts start.
__device__ __forceinline__ long long first_word(const EvictParams &p, long long r, const Request &q) {
  return q.pos0 * p.block_size / 32 + r;
}
__device__ __forceinline__ long long first_window(const EvictParams &p, long long r, const Request &q) {
  return q.pos0 * p.block_size / kEvictWindow + r;
}

__global__ void __launch_bounds__(kEvictThreads)
    kvcs_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ u32 s_score[];   // the row's scores, if they fit
  __shared__ u32 s_hist[256];
  __shared__ u32 s_pick[2];
  __shared__ int s_count[kEvictWindow / 32], s_tie[kEvictWindow / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x / p.rows;
  const int row = static_cast<int>(blockIdx.x % p.rows);
  const EvictCache &c = cache_of_row(p, row);
  const int head = row - c.first_row;
  Request q;
  int B;
  if (!evict_request(p, r, &q, &B, true)) return;
  const int bs = p.block_size, N = q.keys;
  const int *ids = p.tab.block_ids + q.pos0;
  const int *to_ids = p.new_block_ids ? p.new_block_ids + q.pos0 : ids;
  const bool in_place = to_ids == ids;
  if (B == 0 || (B == N && in_place && !p.block_sums)) return;
  const int sinks = min(p.sinks, B), recent = min(p.recent, B - sinks);
  const int lo = sinks, hi = N - recent, want = B - sinks - recent;   // candidates [lo, hi)
  const bool held = N <= p.smem_tokens;
  u32 *const scores = reinterpret_cast<u32 *>(c.scores);
  auto place = [&](const int *blocks, int j) -> u32 * {
    const int pos = p.by_block(j);
    return scores + (static_cast<long long>(blocks[pos]) * c.heads + head) * bs + (j - pos * bs);
  };
  if (held)
    for (int j = tid; j < N; j += kEvictThreads) s_score[j] = *place(ids, j);
  auto score = [&](int j) { return held ? s_score[j] : *place(ids, j); };

  // the least key kept, and how many tokens of that key are
  u32 least = 0xffffffffu, ties = 0;
  const bool all = want == hi - lo;
  if (!all && want > 0) {
    u32 prefix = 0, left = static_cast<u32>(want);
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      s_hist[tid] = 0;
      __syncthreads();
      for (int j0 = lo; j0 < hi; j0 += kEvictThreads) {
        const int j = j0 + tid;
        bool in = j < hi;
        u32 k = 0;
        if (in) {
          k = score_key(score(j));
          in = shift == 24 || (k >> (shift + 8)) == prefix;
        }
        // scores crowd into few digits: lanes of one digit add once
        const u32 digit = in ? k >> shift & 255u : 256u;
        const u32 peers = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(peers) - 1) atomicAdd(&s_hist[digit], __popc(peers));
      }
      __syncthreads();
      if (warp == 0) {
        // digits from the greatest down: the one where the count reaches `left`
        u32 mine[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mine[i] = s_hist[255 - (lane * 8 + i)];
          sum += mine[i];
        }
        u32 inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u32 u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        u32 at = inc - sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (at < left && left <= at + mine[i]) {
            s_pick[0] = 255 - (lane * 8 + i);
            s_pick[1] = left - at;
          }
          at += mine[i];
        }
      }
      __syncthreads();
      prefix = prefix << 8 | s_pick[0];
      left = s_pick[1];
    }
    least = prefix;
    ties = left;
  }

  u32 *const bits = p.bits + row * p.bit_words + first_word(p, r, q);
  u32 *const ahead = p.ahead + row * p.windows + first_window(p, r, q);
  int done = 0;         // tokens kept before the window
  u32 ties_seen = 0;    // tokens of key `least` before the window
  for (int w0 = 0, win = 0; w0 < N; w0 += kEvictWindow, ++win) {
    // a warp takes every eighth group of 32 tokens
    constexpr int kEach = kEvictWindow / kEvictThreads;
    u32 keep[kEach], tie[kEach], value[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = w0 + (i * 8 + warp) * 32 + lane;
      bool stay = j < N && (all || j < lo || j >= hi), equal = false;
      value[i] = j < N ? score(j) : 0u;
      if (j < N && !stay && want > 0) {
        const u32 k = score_key(value[i]);
        stay = k > least;
        equal = k == least;
      }
      keep[i] = __ballot_sync(0xffffffffu, stay);
      tie[i] = __ballot_sync(0xffffffffu, equal);
      if (lane == 0) s_tie[i * 8 + warp] = __popc(tie[i]);
    }
    __syncthreads();
    const u32 t = lane < kEvictWindow / 32 ? s_tie[lane] : 0;
    u32 inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u32 u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      // the first of the equal ones, as far as they are wanted
      const u32 before = ties_seen + __shfl_sync(0xffffffffu, inc - t, i * 8 + warp);
      const int room = static_cast<int>(min(max(static_cast<long long>(ties) - before, 0ll), 32ll));
      u32 take = tie[i];
      for (int extra = __popc(take) - room; extra > 0; --extra) take &= ~(1u << (31 - __clz(take)));
      keep[i] |= take;
      if (lane == 0) s_count[i * 8 + warp] = __popc(keep[i]);
    }
    ties_seen += __shfl_sync(0xffffffffu, inc, 31);
    __syncthreads();
    const int n = s_count[lane];
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (tid == 0) ahead[win] = done;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int g = i * 8 + warp;
      const int first = done + __shfl_sync(0xffffffffu, sum - n, g);
      if (w0 + g * 32 < N) {
        if (lane == 0) bits[(w0 >> 5) + g] = keep[i];
        const int j = first + __popc(keep[i] & ((1u << lane) - 1u));
        // (the window's scores were read before the barriers above)
        if (keep[i] >> lane & 1u) *place(to_ids, j) = value[i];
      }
    }
    done += __shfl_sync(0xffffffffu, sum, 31);
  }
}

__global__ void __launch_bounds__(kEvictThreads)
    kvcs_evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ long long s_from[kEvictWindow], s_to[kEvictWindow];   // kept tokens' byte offsets
  __shared__ int s_block[kEvictWindow];                            // and target blocks
  __shared__ int s_before[kEvictWindow / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::grid_dep_wait();   // the selection's bits
  long long idx = blockIdx.x;
  const int span = static_cast<int>(idx % p.spans);
  idx /= p.spans;
  const int hp = static_cast<int>(idx % p.halves_parts);
  idx /= p.halves_parts;
  const int row = static_cast<int>(idx % p.rows);
  const long long r = idx / p.rows;
  const EvictCache &c = cache_of_row(p, row);
  const int head = row - c.first_row;
  const int half = hp / c.parts, part = hp - half * c.parts;
  if (half >= c.map.halves) return;
  Request q;
  int B;
  if (!evict_request(p, r, &q, &B, false)) return;
  const int bs = p.block_size, N = q.keys;
  const int *ids = p.tab.block_ids + q.pos0;
  const int *to_ids = p.new_block_ids ? p.new_block_ids + q.pos0 : ids;
  const bool in_place = to_ids == ids;
  if (B == 0 || (B == N && in_place && !p.block_sums)) return;
  const u32 *const bits = p.bits + row * p.bit_words + first_word(p, r, q);
  const u32 *const ahead = p.ahead + row * p.windows + first_window(p, r, q);
  const int piece0 = part * c.part_pieces;
  const int pieces = min(c.part_pieces, c.head_bytes / c.unit - piece0);   // of a token, here
  const bool even = pieces == c.part_pieces;
  const u64 P = static_cast<u64>(c.map.halves) * (c.head_bytes / 8);
  const u64 m = c.m0 + 2ull * head;
  unsigned char *const base = const_cast<unsigned char *>(c.map.base) + half * c.map.half_stride;

  for (int w0 = span * kEvictWindow; w0 < N; w0 += p.spans * kEvictWindow) {
    // the window's kept tokens: where they are and where they go
    __syncthreads();   // the lists of the window before are read
    const int words = min(kEvictWindow / 32, (N - w0 + 31) / 32);
    if (warp == 0) {
      const int n = lane < words ? __popc(bits[(w0 >> 5) + lane]) : 0;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
      s_before[lane] = sum - n;
    }
    __syncthreads();
    const int done = static_cast<int>(ahead[w0 / kEvictWindow]);
    for (int g = warp; g < words; g += kEvictThreads / 32) {
      const u32 k = bits[(w0 >> 5) + g];
      if (k >> lane & 1u) {
        const int at = s_before[g] + __popc(k & ((1u << lane) - 1u));
        const int src = w0 + g * 32 + lane, sp = p.by_block(src);
        const int j = done + at, dp = p.by_block(j);
        s_from[at] = token_offset(c.map, ids[sp], src - sp * bs, head);
        s_block[at] = to_ids[dp];
        s_to[at] = token_offset(c.map, to_ids[dp], j - dp * bs, head);
      }
    }
    const int kept = s_before[words - 1] + __popc(bits[(w0 >> 5) + words - 1]);
    __syncthreads();
    const int total = kept * pieces;
    uint4 v[2][kEvictPieces];
    auto split = [&](int u, int *tok, long long *col) {
      *tok = even ? c.by_part(u) : u / pieces;
      const int x = (piece0 + u - *tok * pieces) * c.unit;
      *col = static_cast<long long>(x >> 4) * c.map.chunk_stride + (x & 15);
      return x;
    };
    auto fetch = [&](uint4 (&d)[kEvictPieces], int u0) {
#pragma unroll
      for (int i = 0; i < kEvictPieces; ++i) {
        const int u = u0 + i * kEvictThreads + tid;
        if (u >= total) continue;
        int tok;
        long long col;
        split(u, &tok, &col);
        // tokens that stay where they are pass through only for their words
        if (!p.block_sums && s_from[tok] == s_to[tok]) continue;
        const unsigned char *from = base + s_from[tok] + col;
        if (c.unit == 16) {
          d[i] = *reinterpret_cast<const uint4 *>(from);
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(from);
          d[i] = make_uint4(w.x, w.y, 0, 0);
        }
      }
    };
    auto put = [&](const uint4 (&d)[kEvictPieces], int u0) {
#pragma unroll
      for (int i = 0; i < kEvictPieces; ++i) {
        const int u = u0 + i * kEvictThreads + tid;
        u64 word = 0;
        int block = -1;
        if (u < total) {
          int tok;
          long long col;
          const int x = split(u, &tok, &col);
          if (s_from[tok] != s_to[tok]) {
            unsigned char *to = base + s_to[tok] + col;
            if (c.unit == 16)
              *reinterpret_cast<uint4 *>(to) = d[i];
            else
              *reinterpret_cast<uint2 *>(to) = make_uint2(d[i].x, d[i].y);
          }
          if (p.block_sums) {
            block = s_block[tok];
            const u64 x0 = static_cast<u64>(d[i].y) << 32 | d[i].x;
            const u64 x1 = static_cast<u64>(d[i].w) << 32 | d[i].z;
            const u64 piece = static_cast<u64>(half) * (c.head_bytes / 8) + x / 8;
            const u64 f = 2ull * ((static_cast<u64>(q.base) + done + tok) * P + piece) + 1;
            word = m * (x0 * f + x1 * (f + 2));
          }
        }
        if (p.block_sums) {
          // one add per warp where its pieces share a block
          const int b0 = __shfl_sync(0xffffffffu, block, 0);
          if (__all_sync(0xffffffffu, block == b0 || block < 0)) {
            word = warp_sum(word);
            if (lane == 0 && b0 >= 0) atomicAdd(p.block_sums + b0, word);
          } else if (block >= 0) {
            atomicAdd(p.block_sums + block, word);
          }
        }
      }
    };
    constexpr int kStep = kEvictThreads * kEvictPieces;
    fetch(v[0], 0);
    for (int u0 = 0; u0 < total; u0 += 2 * kStep) {
      fetch(v[1], u0 + kStep);
      __syncthreads();
      put(v[0], u0);
      fetch(v[0], u0 + 2 * kStep);
      __syncthreads();
      put(v[1], u0 + kStep);
    }
  }
}

}  // namespace kvcs
