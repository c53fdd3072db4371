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
// whose unsigned order is the scores' order, three counting passes over digits
// of 11, 11 and 10 bits find the least key kept and how many tokens of exactly
// that key are, and two more leave the list of kept tokens; the scores move on
// the way, or behind it in steps where they are not all held (one warp alone
// marking and moving such a row, in order, took 1974 us for 131,072 tokens,
// this 247).
// kvcs_evict_move_kernel moves the bytes.  Each 16-byte piece of a token moves
// independently of the others, so a row is split by halves and columns where
// rows are few (and, into fresh blocks, by runs of the list); a CTA goes
// through the kept tokens of its columns in order, the addresses of the next
// kEvictChunk tokens being worked out while the current ones move.
//
// In place: the new token j comes from token src(j) >= j, both growing, so a
// write never lands on a token that a later step still reads.  A step's
// pieces are in registers before any of them is written (a CTA barrier), and
// the next step's loads are already on their way by then.
//
// Words: the new blocks' checksum words, sum_h m_h sum_p x_p (2 (t P + p) + 1)
// with t the token's new position, are added while the bytes pass through.
//
// Measured: 8 layers of 16 requests of 512 to 4096 tokens (8 KV heads of 128,
// bf16) down to 1024 in place: 203 us from fresh caches (885 MB, 4.4 TB/s),
// about 46 of them the selection; 32 layers of 32 requests 1460 us, 5.9 TB/s;
// three requests of 6001 to 20,011 tokens, 4 layers, into fresh HND blocks with
// their words: 131 us; one request of 613 tokens, one layer: 14 us, of 131,072
// down to 65,536 628 us.  The first form, one kernel a row, took 277 us for the
// first, 628 for the fresh blocks and 49 for the short request.
#pragma once

#include "kvcs_attn_common.cuh"

namespace kvcs {

constexpr int kEvictThreads = 256;
constexpr int kEvictSelectThreads = 1024;   // at most
constexpr int kEvictChunk = 512;     // kept tokens whose addresses are held at once
constexpr int kEvictPieces = 4;      // pieces a thread moves at once

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
};

// Caches of one launch, at most.  (The parameters travel with every launch:
// 25 KB of them, room for 128 caches, took a launch 10 us on the host.)
constexpr int kEvictCaches = 32;
constexpr int kEvictFewCaches = 2;

struct EvictCall {
  Tables tab;
  const long long *keep;
  const int *new_block_ids;   // or null: in place
  u64 *block_sums;            // or null
  int *list;                  // [rows][total_positions * block_size]: kept tokens
  long long num_blocks;       // smallest pool of the call
  int block_size;
  FastDiv by_block;
  int sinks, recent;
  int num_caches;
  int rows;                   // (cache, head) pairs of the launch
  int smem_tokens;            // scores that shared memory holds
  int halves_parts;           // most column groups of a row, over both halves
  int spans;                  // fresh blocks: CTAs that share a row's list
};

template <int kCaches>
struct EvictParams : EvictCall {
  EvictCache c[kCaches];
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
__device__ inline bool evict_request(const EvictCall &p, long long r, Request *q, int *budget,
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
__global__ void __launch_bounds__(256) kvcs_evict_zero_kernel(const __grid_constant__ EvictCall p) {
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
template <int kCaches>
__device__ __forceinline__ const EvictCache &cache_of_row(const EvictParams<kCaches> &p, int row) {
  int lo = 0, hi = p.num_caches - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.c[mid].first_row <= row) lo = mid; else hi = mid - 1;
  }
  return p.c[lo];
}

// Where the list of a row's kept tokens starts.
__device__ __forceinline__ int *row_list(const EvictCall &p, int row, const Request &q) {
  return p.list + (row * p.tab.total_positions + q.pos0) * p.block_size;
}

// Sum of a value over the CTA's threads before this one; *total: over all.
__device__ __forceinline__ int cta_scan(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int w = lane < warps ? warp_sums[lane] : 0;
  int sum = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  *total = __shfl_sync(0xffffffffu, sum, 31);
  return __shfl_sync(0xffffffffu, sum - w, warp) + inc - v;
}

// Digits of the counting passes: 11, 11 and 10 bits from the top.
constexpr int kEvictBins = 2048;

template <int kCaches>
__global__ void __launch_bounds__(kEvictSelectThreads)
    kvcs_evict_select_kernel(const __grid_constant__ EvictParams<kCaches> p) {
  extern __shared__ u32 s_score[];   // the row's scores, if they fit
  __shared__ u32 s_hist[kEvictBins];
  __shared__ int s_sums[32];
  __shared__ u32 s_pick[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
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
  const long long per_block = static_cast<long long>(c.heads) * bs, at_head = static_cast<long long>(head) * bs;
  auto place = [&](const int *blocks, int j) -> u32 * {
    const int pos = p.by_block(j);
    return scores + blocks[pos] * per_block + at_head + (j - pos * bs);
  };
  const int n_held = min(N, p.smem_tokens);
#pragma unroll 4
  for (int j = tid; j < n_held; j += threads) s_score[j] = *place(ids, j);
  auto score = [&](int j) { return j < n_held ? s_score[j] : *place(ids, j); };
  constexpr int kAhead = 8;   // scores a thread asks for at once

  // the least key kept, and how many tokens of that key are
  u32 least = 0xffffffffu, ties = 0;
  const bool all = want == hi - lo;
  if (!all && want > 0) {
    u32 prefix = 0, left = static_cast<u32>(want);
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const u32 bins = shift == 0 ? 1024u : 2048u, above = shift == 0 ? 10u : 11u;
      __syncthreads();
      for (u32 i = tid; i < bins; i += threads) s_hist[i] = 0;
      __syncthreads();
      for (int j0 = lo + tid; j0 < hi; j0 += kAhead * threads) {
        u32 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (j0 + i * threads < hi) v[i] = score(j0 + i * threads);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (j0 + i * threads >= hi) continue;
          const u32 k = score_key(v[i]);
          if (shift == 21 || (k >> (shift + above)) == prefix)
            atomicAdd(&s_hist[k >> shift & (bins - 1)], 1u);
        }
      }
      __syncthreads();
      // digits from the greatest down: the one where the count reaches `left`
      const u32 each = bins / threads > 0 ? bins / threads : 1;   // per thread
      u32 sum = 0;
      for (u32 i = 0; i < each; ++i) {
        const u32 bin = tid * each + i;
        if (bin < bins) sum += s_hist[bins - 1 - bin];
      }
      int total;
      u32 at = static_cast<u32>(cta_scan(static_cast<int>(sum), s_sums, &total));
      for (u32 i = 0; i < each; ++i) {
        const u32 bin = tid * each + i;
        const u32 n = bin < bins ? s_hist[bins - 1 - bin] : 0;
        if (at < left && left <= at + n) {
          s_pick[0] = bins - 1 - bin;
          s_pick[1] = left - at;
        }
        at += n;
      }
      __syncthreads();
      prefix = prefix << above | s_pick[0];
      left = s_pick[1];
    }
    least = prefix;
    ties = left;
  }

  // Kept tokens in order.  A warp takes a run of words of 32 tokens, first
  // counting, then, from the counts before it, marking.  Scores that are held
  // move on the way; others follow behind, in steps.
  int *const list = row_list(p, row, q);
  const int words = (N + 31) / 32;
  const int run = (words + warps - 1) / warps;
  const int w0 = min(words, warp * run), w1 = min(words, w0 + run);
  auto read = [&](int w, u32 (&v)[kAhead]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = (w + i) * 32 + lane;
      v[i] = w + i < w1 && j < N ? score(j) : 0u;
    }
  };
  auto look = [&](int w, u32 value, u32 *tie) {
    const int j = w * 32 + lane;
    bool stay = j < N && (all || j < lo || j >= hi), equal = false;
    if (j < N && !stay && want > 0) {
      const u32 k = score_key(value);
      stay = k > least;
      equal = k == least;
    }
    *tie = __ballot_sync(0xffffffffu, equal);
    return __ballot_sync(0xffffffffu, stay);
  };
  int sure = 0, equal = 0;
  for (int w = w0; w < w1; w += kAhead) {
    u32 v[kAhead];
    read(w, v);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (w + i >= w1) break;
      u32 tie;
      sure += __popc(look(w + i, v[i], &tie));
      equal += __popc(tie);
    }
  }
  int total;
  const int tie0 = cta_scan(lane == 0 ? equal : 0, s_sums, &total);
  // of the equal ones the first are kept, as far as they are wanted
  auto taken = [&](int before, int n) {
    return static_cast<int>(min(max(static_cast<long long>(ties) - before, 0ll),
                                static_cast<long long>(n)));
  };
  const int mine_tie0 = __shfl_sync(0xffffffffu, tie0, 0);
  int seen = mine_tie0;
  const int kept = sure + taken(seen, equal);
  int done = cta_scan(lane == 0 ? kept : 0, s_sums, &total);
  done = __shfl_sync(0xffffffffu, done, 0);
  for (int w = w0; w < w1; w += kAhead) {
    u32 v[kAhead];
    read(w, v);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (w + i >= w1) break;
      u32 tie;
      u32 keep = look(w + i, v[i], &tie);
      const int n = __popc(tie);
      u32 take = tie;
      for (int extra = n - taken(seen, n); extra > 0; --extra) take &= ~(1u << (31 - __clz(take)));
      keep |= take;
      seen += n;
      if (keep >> lane & 1u) {
        const int j = done + __popc(keep & ((1u << lane) - 1u));
        list[j] = (w + i) * 32 + lane;
        if (held) *place(to_ids, j) = v[i];
      }
      done += __popc(keep);
    }
  }
  if (held) return;
  // The score of new token j comes from list[j] >= j: a step reads all of its
  // scores before it writes any, and no later step reads what it wrote.
  for (int j0 = 0; j0 < B; j0 += kAhead * threads) {
    u32 v[kAhead];
    __syncthreads();   // the list is there, the step before has written
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * threads + tid;
      if (j < B)
        v[i] = *place(ids, static_cast<int>(min(static_cast<u32>(list[j]), static_cast<u32>(N - 1))));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * threads + tid;
      if (j < B) *place(to_ids, j) = v[i];
    }
  }
}

template <int kCaches, bool kWords, bool kUnit16>
__global__ void __launch_bounds__(kEvictThreads)
    kvcs_evict_move_kernel(const __grid_constant__ EvictParams<kCaches> p) {
  // two chunks' byte offsets of the kept tokens and their targets
  __shared__ long long s_from[2][kEvictChunk], s_to[2][kEvictChunk];
  __shared__ int s_block[2][kWords ? kEvictChunk : 1];   // and target blocks
  const int tid = threadIdx.x, lane = tid & 31;
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
  if (half >= c.map.halves || (c.unit == 16) != kUnit16) return;
  Request q;
  int B;
  if (!evict_request(p, r, &q, &B, false)) return;
  const int bs = p.block_size;
  const int *ids = p.tab.block_ids + q.pos0;
  const int *to_ids = p.new_block_ids ? p.new_block_ids + q.pos0 : ids;
  const bool in_place = to_ids == ids;
  if (B == 0 || (B == q.keys && in_place && !kWords)) return;
  const int *const list = row_list(p, row, q);
  constexpr int kUnit = kUnit16 ? 16 : 8;
  const int piece0 = part * c.part_pieces;
  const int pieces = min(c.part_pieces, c.head_bytes / kUnit - piece0);   // of a token, here
  // a thread has one column, and eight consecutive tokens of every step
  const int slot = tid / pieces;
  const int tokens = kEvictThreads / pieces;   // threads side by side on tokens
  const bool active = slot < tokens;
  const int x = (piece0 + tid - slot * pieces) * kUnit;
  unsigned char *const base = const_cast<unsigned char *>(c.map.base) + half * c.map.half_stride +
                              static_cast<long long>(x >> 4) * c.map.chunk_stride + (x & 15);
  const u64 P = static_cast<u64>(c.map.halves) * (c.head_bytes / 8);
  const u64 m = c.m0 + 2ull * head;
  const u64 piece = static_cast<u64>(half) * (c.head_bytes / 8) + x / 8;
  const PageMap &map = c.map;

  // addresses of a chunk, in the steps between which other work goes on: the
  // list, the blocks, and the offsets.  (Requests that share positions, which
  // is flagged, share their lists: an entry may be another request's.)
  constexpr int kOwn = kEvictChunk / kEvictThreads;
  int src[kOwn], from_id[kOwn], to_id[kOwn];
  auto look_list = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = j0 + i * kEvictThreads + tid;
      src[i] = j < B ? static_cast<int>(min(static_cast<u32>(list[j]), static_cast<u32>(q.keys - 1)))
                     : -1;
    }
  };
  auto look_blocks = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (src[i] < 0) continue;
      from_id[i] = ids[p.by_block(src[i])];
      to_id[i] = to_ids[p.by_block(j0 + i * kEvictThreads + tid)];
    }
  };
  auto note = [&](int buf, int j0) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (src[i] < 0) continue;
      const int at = i * kEvictThreads + tid, j = j0 + at;
      s_from[buf][at] = token_offset(map, from_id[i], src[i] - p.by_block(src[i]) * bs, head);
      s_to[buf][at] = token_offset(map, to_id[i], j - p.by_block(j) * bs, head);
      if (kWords) s_block[buf][at] = to_id[i];
    }
  };
  const int stride = p.spans * kEvictChunk;
  int buf = 0;
  look_list(span * kEvictChunk);
  look_blocks(span * kEvictChunk);
  note(0, span * kEvictChunk);
  for (int j0 = span * kEvictChunk; j0 < B; j0 += stride, buf ^= 1) {
    const int kept = min(kEvictChunk, B - j0), done = j0;
    __syncthreads();   // the chunk's addresses are there
    look_list(j0 + stride);
    const long long *const from_at = s_from[buf], *const to_at = s_to[buf];
    const int *const block_at = s_block[buf];
    uint4 v[2][kEvictPieces];
    auto fetch = [&](uint4 (&d)[kEvictPieces], int t0) {
      const int t = t0 + slot * kEvictPieces;
#pragma unroll
      for (int i = 0; i < kEvictPieces; ++i) {
        if (!active || t + i >= kept) continue;
        // tokens that stay where they are pass through only for their words
        if (!kWords && from_at[t + i] == to_at[t + i]) continue;
        const unsigned char *from = base + from_at[t + i];
        if (kUnit16) {
          d[i] = *reinterpret_cast<const uint4 *>(from);
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(from);
          d[i] = make_uint4(w.x, w.y, 0, 0);
        }
      }
    };
    auto put = [&](const uint4 (&d)[kEvictPieces], int t0) {
      const int t = t0 + slot * kEvictPieces;
#pragma unroll
      for (int i = 0; i < kEvictPieces; ++i) {
        if (!active || t + i >= kept || from_at[t + i] == to_at[t + i]) continue;
        unsigned char *to = base + to_at[t + i];
        if (kUnit16)
          *reinterpret_cast<uint4 *>(to) = d[i];
        else
          *reinterpret_cast<uint2 *>(to) = make_uint2(d[i].x, d[i].y);
      }
      if constexpr (kWords) {
        // sums of runs of tokens of one block, then of the warp's lanes
        u64 sum = 0;
        int block = -1;
        auto flush = [&]() {
          u32 open = __ballot_sync(0xffffffffu, block >= 0);
          while (open) {
            const int b = __shfl_sync(0xffffffffu, block, __ffs(open) - 1);
            const bool same = block == b;
            const u64 all = warp_sum(same ? sum : 0ull);
            if (lane == __ffs(open) - 1) atomicAdd(p.block_sums + b, m * all);
            open &= ~__ballot_sync(0xffffffffu, same);
          }
        };
#pragma unroll
        for (int i = 0; i < kEvictPieces; ++i) {
          const bool in = active && t + i < kept;
          const int b = in ? block_at[t + i] : block;
          if (__any_sync(0xffffffffu, b != block && block >= 0)) {
            flush();
            sum = 0;
            block = -1;
          }
          if (in) {
            const u64 x0 = static_cast<u64>(d[i].y) << 32 | d[i].x;
            const u64 x1 = static_cast<u64>(d[i].w) << 32 | d[i].z;
            const u64 f = 2ull * ((static_cast<u64>(q.base) + done + t + i) * P + piece) + 1;
            sum += (x0 + x1) * f + 2ull * x1;
            block = b;
          }
        }
        flush();
      }
    };
    const int step = tokens * kEvictPieces;
    fetch(v[0], 0);
    look_blocks(j0 + stride);
    for (int t0 = 0; t0 < kept; t0 += 2 * step) {
      fetch(v[1], t0 + step);
      if (in_place) __syncthreads();
      put(v[0], t0);
      fetch(v[0], t0 + 2 * step);
      if (in_place) __syncthreads();
      put(v[1], t0 + step);
    }
    note(buf ^ 1, j0 + stride);
  }
}

}  // namespace kvcs
