// kvcs_evict.cuh -- eviction of cached tokens by score, and the move of the
// kept ones to the front of the request's blocks.
//
// Per row (request, cache, KV head) with N cached tokens and a budget B < N:
// the first `sinks` and the last `recent` tokens stay, and of the others the
// B - sinks - recent with the greatest scores (equal scores: the lowest
// index).  Kept tokens move, in order, to tokens 0 .. B-1 of the target
// blocks, with their scores.
//
// Selection: scores become 32-bit keys whose unsigned order is the scores'
// order; four counting passes over 8-bit digits find the key of the last
// token kept, and how many tokens of exactly that key are kept.
//
// Move: the new token j comes from token src(j) >= j, both growing, so in
// place a write never lands on a token that a later step still reads; a step
// reads its tokens into registers, waits for the CTA and writes them.
//
// Words: the new blocks' checksum words, sum_h m_h sum_p x_p (2 (t P + p) + 1)
// with t the token's new position, are added while the bytes pass through.
#pragma once

#include "kvcs_attn_common.cuh"

namespace kvcs {

constexpr int kEvictThreads = 256;
constexpr int kEvictWindow = 1024;   // tokens looked over per step
constexpr int kEvictUnits = 8;       // pieces a thread holds at once

struct EvictCache {
  PageMap map;
  float *scores;      // [num_blocks][heads][block_size]
  u64 m0;             // checksum factor of local head 0
  int heads;
  int head_bytes;
  int first_row;      // first (cache, head) index of this cache in the launch
  int unit8;
};

struct EvictParams {
  Tables tab;
  const long long *keep;
  const int *new_block_ids;   // or null: in place
  u64 *block_sums;            // or null
  long long num_blocks;       // smallest pool of the call
  int block_size;
  int sinks, recent;
  int num_caches;
  int rows;                   // (cache, head) pairs of the launch
  EvictCache c[kMaxCachesPerLaunch];
};

// Unsigned keys in the order of the scores; -0 equals 0, every NaN is the
// greatest.
__device__ __forceinline__ u32 score_key(float f) {
  if (f != f) return 0xffffffffu;
  const u32 b = __float_as_uint(f + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Tokens and budget of a request; false when it is to be left alone (bad
// tables or block ids, which are flagged).  Called by a whole CTA.
__device__ inline bool evict_request(const EvictParams &p, long long r, Request *q, int *budget) {
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  const long long a = p.tab.pos_offsets[r], b = p.tab.pos_offsets[r + 1];
  *q = read_tokens(p.tab, r, p.block_size, threadIdx.x == 0);
  const long long keep = p.keep[r];
  // tables read_tokens has refused hold no tokens and are left alone too
  if (keep < 0 && threadIdx.x == 0) raise(p.tab, kStatusBadRequests);
  if (keep < 0 || q->keys == 0 || a < 0 || b > p.tab.total_positions) return false;
  *budget = static_cast<int>(min(keep, static_cast<long long>(q->keys)));
  const int blocks = (q->keys + p.block_size - 1) / p.block_size;
  const int targets = (*budget + p.block_size - 1) / p.block_size;
  for (int i = threadIdx.x; i < blocks; i += blockDim.x) {
    const int id = p.tab.block_ids[q->pos0 + i];
    bool bad = id < 0 || id >= p.num_blocks;
    if (p.new_block_ids && i < targets) {
      const int to = p.new_block_ids[q->pos0 + i];
      bad |= to < 0 || to >= p.num_blocks;
    }
    if (bad) s_bad = 1;
  }
  __syncthreads();
  if (s_bad && threadIdx.x == 0) raise(p.tab, kStatusBadBlockId);
  return !s_bad;
}

// Zeroes the checksum words of the blocks the call fills (in place: of every
// block that held a token).
__global__ void __launch_bounds__(256) kvcs_evict_zero_kernel(const __grid_constant__ EvictParams p) {
  for (long long r = blockIdx.x; r < p.tab.num_requests; r += gridDim.x) {
    Request q;
    int budget;
    if (evict_request(p, r, &q, &budget)) {
      const int *ids = (p.new_block_ids ? p.new_block_ids : p.tab.block_ids) + q.pos0;
      const int n = ((p.new_block_ids ? budget : q.keys) + p.block_size - 1) / p.block_size;
      for (int i = threadIdx.x; i < n; i += blockDim.x) p.block_sums[ids[i]] = 0;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kEvictThreads)
    kvcs_evict_kernel(const __grid_constant__ EvictParams p) {
  __shared__ u32 s_hist[256];
  __shared__ u32 s_pick[2];
  __shared__ int s_src[kEvictWindow];
  __shared__ int s_warp[2][kEvictThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x / p.rows;
  const int row = static_cast<int>(blockIdx.x % p.rows);
  int ci = 0;
  while (ci + 1 < p.num_caches && p.c[ci + 1].first_row <= row) ++ci;
  const EvictCache &c = p.c[ci];
  const int head = row - c.first_row;
  Request q;
  int B;
  if (!evict_request(p, r, &q, &B)) return;
  const int bs = p.block_size, N = q.keys;
  const int *ids = p.tab.block_ids + q.pos0;
  const int *to_ids = p.new_block_ids ? p.new_block_ids + q.pos0 : ids;
  const bool in_place = to_ids == ids;
  if (B == 0 || (B == N && in_place && !p.block_sums)) return;
  const int sinks = min(p.sinks, B), recent = min(p.recent, B - sinks);
  const int lo = sinks, hi = N - recent, want = B - sinks - recent;   // candidates [lo, hi)

  auto score_at = [&](int j) -> float * {
    const int pos = j / bs;
    return c.scores + (static_cast<long long>(ids[pos]) * c.heads + head) * bs + (j - pos * bs);
  };

  // the least key kept, and how many tokens of that key are
  u32 least = 0xffffffffu, ties = 0;
  if (want == hi - lo) {
    least = 0;
    ties = 0xffffffffu;
  } else if (want > 0) {
    u32 prefix = 0, left = static_cast<u32>(want);
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      s_hist[tid] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kEvictThreads) {
        const u32 k = score_key(*score_at(j));
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[k >> shift & 255u], 1u);
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

  const int unit = c.unit8 ? 8 : 16;
  const int per_half = c.head_bytes / unit;
  const int per_token = c.map.halves * per_half;   // pieces of a token
  const u64 P = static_cast<u64>(c.map.halves) * (c.head_bytes / 8);
  const u64 m = c.m0 + 2ull * head;
  int done = 0;       // tokens kept before the window
  int ties_seen = 0;  // tokens of key `least` before the window
  for (int w0 = 0; w0 < N; w0 += kEvictWindow) {
    // which of the window's tokens stay: four consecutive tokens a thread
    constexpr int kEach = kEvictWindow / kEvictThreads;
    bool stay[kEach], tie[kEach];
    int n_tie = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = w0 + tid * kEach + i;
      stay[i] = j < N && (j < lo || j >= hi);
      tie[i] = false;
      if (j < N && !stay[i]) {
        if (ties == 0xffffffffu) {
          stay[i] = true;
        } else if (want > 0) {
          const u32 k = score_key(*score_at(j));
          stay[i] = k > least;
          tie[i] = k == least;
        }
      }
      n_tie += tie[i];
    }
    int inc = n_tie;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();   // s_src and s_warp of the window before are read
    if (lane == 31) s_warp[0][warp] = inc;
    __syncthreads();
    int tie_at = ties_seen + inc - n_tie, n_stay = 0;
    for (int k = 0; k < kEvictThreads / 32; ++k) {
      if (k < warp) tie_at += s_warp[0][k];
      ties_seen += s_warp[0][k];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (tie[i]) stay[i] = static_cast<u32>(tie_at++) < ties;
      n_stay += stay[i];
    }
    inc = n_stay;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s_warp[1][warp] = inc;
    __syncthreads();
    int at = inc - n_stay, kept = 0;
    for (int k = 0; k < kEvictThreads / 32; ++k) {
      if (k < warp) at += s_warp[1][k];
      kept += s_warp[1][k];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (stay[i]) s_src[at++] = w0 + tid * kEach + i;
    __syncthreads();

    // scores
    float moved[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = i * kEvictThreads + tid;
      if (k < kept) moved[i] = *score_at(s_src[k]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = i * kEvictThreads + tid;
      if (k < kept) {
        const int j = done + k, pos = j / bs;
        c.scores[(static_cast<long long>(to_ids[pos]) * c.heads + head) * bs + (j - pos * bs)] =
            moved[i];
      }
    }
    // K and V (or latent rows)
    const int pieces = kept * per_token;
    for (int u0 = 0; u0 < pieces; u0 += kEvictThreads * kEvictUnits) {
      uint4 v[kEvictUnits];
#pragma unroll
      for (int i = 0; i < kEvictUnits; ++i) {
        const int u = u0 + i * kEvictThreads + tid;
        if (u >= pieces) continue;
        const int k = u / per_token, e = u - k * per_token;
        const int half = e >= per_half, x = (e - half * per_half) * unit;
        const int src = s_src[k], pos = src / bs;
        if (in_place && src == done + k && !p.block_sums) continue;   // stays where it is
        const unsigned char *from = c.map.base + half * c.map.half_stride +
                                    token_offset(c.map, ids[pos], src - pos * bs, head) +
                                    static_cast<long long>(x >> 4) * c.map.chunk_stride + (x & 15);
        if (unit == 16) {
          v[i] = *reinterpret_cast<const uint4 *>(from);
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(from);
          v[i] = make_uint4(w.x, w.y, 0, 0);
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kEvictUnits; ++i) {
        const int u = u0 + i * kEvictThreads + tid;
        u64 word = 0;
        int block = -1;
        if (u < pieces) {
          const int k = u / per_token, e = u - k * per_token;
          const int half = e >= per_half, x = (e - half * per_half) * unit;
          const int j = done + k, pos = j / bs;
          block = to_ids[pos];
          if (!(in_place && s_src[k] == j)) {
            unsigned char *to = const_cast<unsigned char *>(c.map.base) +
                                half * c.map.half_stride +
                                token_offset(c.map, block, j - pos * bs, head) +
                                static_cast<long long>(x >> 4) * c.map.chunk_stride + (x & 15);
            if (unit == 16)
              *reinterpret_cast<uint4 *>(to) = v[i];
            else
              *reinterpret_cast<uint2 *>(to) = make_uint2(v[i].x, v[i].y);
          }
          if (p.block_sums) {
            const u64 x0 = static_cast<u64>(v[i].y) << 32 | v[i].x;
            const u64 x1 = static_cast<u64>(v[i].w) << 32 | v[i].z;
            const u64 piece = static_cast<u64>(half) * (c.head_bytes / 8) + x / 8;
            const u64 f = 2ull * ((static_cast<u64>(q.base) + j) * P + piece) + 1;
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
    }
    done += kept;
  }
}

}  // namespace kvcs
