// kvcs_mass.cuh -- attention mass of cached tokens: for every cached token j
// of every KV head, the weights it gets from the observed queries,
//     mass_j += sum_i 2^(z_ij - lse_i / ln 2),
// with z and the visible (i, j) as in the attention, and lse from it.
//
// Bound: one product per (query row, token) and a read of K, so a decode
// step is bound by the read of K.  A warp owns 16 tokens of one head while the
// query rows pass, so every token's sum is made by one warp in row order and
// added to memory once: the result does not depend on timing (unless requests
// share the block).  K comes through shared memory, each lane copying just
// what it reads, two chunks ahead.
//
// Measured: 64 requests of 512 to 4096 tokens (8 KV heads of 128, bf16), one
// token each: 57 us, 5.4 TB/s of K.  With the keys loaded to registers 88 (a
// chunk ahead 160 registers, three CTAs an SM, 104); with divisions for each
// chunk's place, a test for each piece and four additions to memory of four
// lanes each, 74.  Four CTAs with three stages; three with four 60, five with
// two 58.  fp8 takes 52 (59, 68): conversions and products, not DRAM.
#pragma once

#include "kvcs_attend.cuh"

namespace kvcs {

constexpr int kMassThreads = 128;
constexpr int kMassStages = 3;   // chunks of a warp on their way or in use

// A request's chunks of 16 tokens that some observed query may see.
struct MassSpan {
  int lo;            // first chunk
  int chunks;
  int first;         // first observed new token
  long long total;
};

__device__ __forceinline__ MassSpan mass_span(const AttnParams &p, const Request &q) {
  MassSpan s;
  s.lo = s.chunks = 0;
  s.first = p.observe > 0 ? max(0, q.n - p.observe) : 0;
  s.total = 0;
  const long long r = static_cast<long long>(q.n - s.first) * p.group;
  if (r < p.row_lo || r > p.row_hi) return s;
  const int first = p.window > 0 ? max(0, q.at + s.first - p.window + 1) : 0;
  const int end = min(q.keys, max(0, q.at + q.n));
  s.lo = first / kChunkKeys;
  s.chunks = max(0, (end + kChunkKeys - 1) / kChunkKeys - s.lo);
  s.total = static_cast<long long>(s.chunks) * p.kv_heads;
  return s;
}

template <int kType, int kDim>
struct MassShape {
  static constexpr int kWords = kDim * (kType == kKvFp8 ? 1 : 2) / 64;   // 16-byte pieces of a key per lane
  static constexpr int kStageBytes = 2 * kWords * 512;                   // a chunk of a warp
  static constexpr int kStages = kWords > 4 ? 2 : kMassStages;
  static constexpr int kSmemBytes = kMassThreads / 32 * kStages * kStageBytes;
  static constexpr int kCtas = kDim > 128 ? 3 : 4;                       // per SM
};

// A chunk on its way: whose it is, and which of its tokens are there.
struct MassChunk {
  long long r;
  int head, key0;
  u32 valid;
};

template <int kType, int kDim>
__global__ void __launch_bounds__(kMassThreads, MassShape<kType, kDim>::kCtas)
    kvcs_mass_kernel(const __grid_constant__ AttnParams p) {
  using S = MassShape<kType, kDim>;
  constexpr int kElem = kType == kKvFp8 ? 1 : 2;
  constexpr bool kBf16 = kType == kKvBf16;
  constexpr int kWords = S::kWords;
  extern __shared__ __align__(1024) unsigned char attend_smem[];
  __shared__ MassChunk s_chunk[kMassThreads / 32][S::kStages];
  __shared__ long long s_scan[4];
  __shared__ long long s_req[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int pg = (g >> 1) | ((g & 1) << 2);
  const long long R = p.tab.num_requests;
  long long sum = 0;
  for (long long r = tid; r < R; r += kMassThreads)
    sum += mass_span(p, read_request(p.tab, r, p.map.block_size, blockIdx.x == 0)).total;
  long long total;
  const long long ahead_of_me = block_scan(sum, &total, s_scan);
  const long long a_cta = total * blockIdx.x / gridDim.x, b_cta = total * (blockIdx.x + 1ll) / gridDim.x;
  if (a_cta >= b_cta) return;
  long long before = 0, r = 0;
  for (long long c = 0;; c += kMassThreads) {
    const long long rr = c + tid;
    long long v = sum, all = total, ex = ahead_of_me;
    if (R > kMassThreads) {   // (otherwise the first scan tells)
      v = rr < R ? mass_span(p, read_request(p.tab, rr, p.map.block_size, false)).total : 0;
      ex = before + block_scan(v, &all, s_scan);
    }
    if (before + all > a_cta) {
      if (v > 0 && ex <= a_cta && a_cta < ex + v) {
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
  MassSpan sp = mass_span(p, q);
  constexpr int kWarps = kMassThreads / 32;
  // The CTA's run goes round its warps.  A lane copies the pieces that it will
  // read itself, so a stage needs no more than the lane's own wait.
  const u32 ring = ptx::smem_addr(attend_smem) + warp * S::kStages * S::kStageBytes + lane * 16;
  int put = 0, f_head = 0, f_chunk = -1;   // the next chunk's, counted on
  auto fetch = [&](long long x) {
    if (x < b_cta) {
      while (x >= before + sp.total) {
        before += sp.total;
        ++r;
        q = read_request(p.tab, r, p.map.block_size, false);
        sp = mass_span(p, q);
        f_chunk = -1;
      }
      if (f_chunk < 0) {
        f_head = static_cast<int>((x - before) / sp.chunks);
        f_chunk = static_cast<int>((x - before) % sp.chunks);
      } else {
        f_chunk += kWarps;
        while (f_chunk >= sp.chunks) {
          f_chunk -= sp.chunks;
          ++f_head;
        }
      }
      const int key0 = (sp.lo + f_chunk) * kChunkKeys;
      const int key = key0 + (lane & 15);
      // (blocks of tokens that no observed row sees are not looked at)
      bool ok = key < q.keys && key < q.at + q.n &&
                (p.window == 0 || key > q.at + sp.first - p.window);
      long long off = 0;
      if (ok) {
        const int pos = p.map.by_block(key);
        const int block = p.tab.block_ids[q.pos0 + pos];
        if (block < 0 || block >= p.map.num_blocks) {
          ok = false;
          raise(p.tab, kStatusBadBlockId);
        } else {
          off = token_offset(p.map, block, key - pos * p.map.block_size, f_head);
        }
      }
      const u32 valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int row_bytes = p.head_dim * kElem;
      const bool plain = !p.unit8 && row_bytes == kDim * kElem;   // whole 16-byte pieces
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // this lane's two keys, j * 8 + pg
        const long long o = __shfl_sync(0xffffffffu, off, j * 8 + pg);   // (0 where nothing is)
        const int there = valid >> (j * 8 + pg) & 1u ? row_bytes : 0;
        const u32 dst = ring + put * S::kStageBytes + j * kWords * 512;
        const unsigned char *src = p.map.base + o + t * static_cast<long long>(p.map.chunk_stride);
        if (plain) {
#pragma unroll
          for (int b = 0; b < kWords; ++b)
            cp_async16(dst + b * 512, src + b * (4ll * p.map.chunk_stride), there ? 16 : 0);
        } else {
#pragma unroll
          for (int b = 0; b < kWords; ++b) {
            const int c = 4 * b + t;
            const unsigned char *at = c * 16 < there ? src + b * (4ll * p.map.chunk_stride) : p.map.base;
            if (!p.unit8) {
              cp_async16(dst + b * 512, at, c * 16 < there ? 16 : 0);
            } else {
              cp_async8z(dst + b * 512, at, c * 16 < there ? 8 : 0);
              cp_async8z(dst + b * 512 + 8, c * 16 + 8 < there ? at + 8 : at,
                         c * 16 + 8 < there ? 8 : 0);
            }
          }
        }
      }
      if (lane == 0) s_chunk[warp][put] = MassChunk{r, f_head, key0, valid};
      put = put + 1 == S::kStages ? 0 : put + 1;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) fetch(a_cta + warp + i * kWarps);
  // A warp keeps the queries of a group that fits one tile of 16 rows (a
  // decode step) from chunk to chunk.
  u32 qf[kDim / 8][2];
  float rs[2], lse[2];
  int at[2];
  long long held_r = -1, now_r = -1;
  int held_head = -1, stage = 0;
  Request now;
  int now_first = 0;
  for (long long x = a_cta + warp; x < b_cta; x += kWarps) {
    cp_async_wait<S::kStages - 2>();
    __syncwarp();
    const MassChunk chunk = s_chunk[warp][stage];
    const int head = chunk.head, key0 = chunk.key0;
    const u32 valid = chunk.valid;
    const u32 keys = ring + stage * S::kStageBytes;
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    fetch(x + (S::kStages - 1) * kWarps);
    if (chunk.r != now_r) {
      now_r = chunk.r;
      now = read_request(p.tab, now_r, p.map.block_size, false);
      now_first = mass_span(p, now).first;
    }
    float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};   // tokens j * 8 + t + 4 i
    // observed tokens that see some key of the chunk (all of a small group)
    const bool small = (now.n - now_first) * p.group <= 16;
    const int i0 = small ? now_first : max(now_first, key0 - now.at);
    int i1 = now.n;
    if (p.window > 0 && !small)
      i1 = static_cast<int>(min(static_cast<long long>(i1),
                                static_cast<long long>(key0) + kChunkKeys - 1 + p.window - now.at));
    const int rows_end = i1 * p.group;
#pragma unroll 1
    for (int row0 = i0 * p.group; row0 < rows_end; row0 += 16) {
      if (!small || now_r != held_r || head != held_head) {
        int row[2];
        bool has[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rr = row0 + g + 8 * i;
          has[i] = rr < rows_end;
          row[i] = has[i] ? rr : row0;
          const int ti = p.by_group(row[i]);
          at[i] = has[i] ? now.at + ti : -1;   // spare rows see nothing
          lse[i] = kLog2e * __ldg(p.lse + (now.q0 + ti) * (p.group * p.kv_heads) + head * p.group +
                                  row[i] - ti * p.group);
        }
        load_queries<kType, kDim>(p, now, head, row, has, qf, rs);
        held_r = small ? now_r : -1;
        held_head = head;
      }
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int b = 0; b < kWords; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 k = lds128(keys + (j * kWords + b) * 512);
          if constexpr (kType == kKvFp8) {
            const u32 kw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              u32 lo, hi;
              fp8x4_to_half(kw[i], lo, hi);
              const int step = 4 * b + i;
              mma16816<false>(s[j], qf[2 * step][0], qf[2 * step][1], qf[2 * step + 1][0],
                              qf[2 * step + 1][1], lo, hi);
            }
          } else {
            mma16816<kBf16>(s[j], qf[4 * b][0], qf[4 * b][1], qf[4 * b + 1][0], qf[4 * b + 1][1],
                            k.x, k.y);
            mma16816<kBf16>(s[j], qf[4 * b + 2][0], qf[4 * b + 2][1], qf[4 * b + 3][0],
                            qf[4 * b + 3][1], k.z, k.w);
          }
        }
      scores_of(p, s, rs);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + j * 8 + t + 4 * (i & 1);
          const int a = at[i >> 1];
          if (key <= a && (p.window == 0 || key > a - p.window))
            acc[j][i & 1] += ex2(s[j][i] - lse[i >> 1]);
        }
    }
    // over the 8 lanes of a token: each exchange halves what a lane holds, and
    // lane kk ends up with token kk
    const bool hi_i = lane & 4, hi_j = lane & 8;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      v[j] = (hi_i ? acc[j][1] : acc[j][0]) +
             __shfl_xor_sync(0xffffffffu, hi_i ? acc[j][0] : acc[j][1], 4);
    float sum_kk = (hi_j ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi_j ? v[0] : v[1], 8);
    sum_kk += __shfl_xor_sync(0xffffffffu, sum_kk, 16);
    if (lane < 16 && (valid >> lane & 1u)) {
      const int key = key0 + lane, pos = p.map.by_block(key);
      const long long block = p.tab.block_ids[now.pos0 + pos];
      atomicAdd(p.mass + (block * p.kv_heads + head) * p.map.block_size +
                    (key - pos * p.map.block_size), sum_kk);
    }
  }
}

}  // namespace kvcs
