// kvcs_mass_tc.cuh -- attention mass of many observed queries on the
// tensor-memory tensor cores (16-bit caches, heads of 64 or 128).
//
// Mathematics as in kvcs_mass.cuh.  Bound: 2 * head_dim operations and one
// exponential per visible (row, token) pair; with heads of 128 the tensor
// cores and the exponentials take about the same time.
//
// The products are made the other way round than in the attention: a unit's
// 256 tokens are the rows of the product (two tiles of 128, their K resident),
// and the query rows pass by in tiles of up to 128 as its columns.  A thread
// then owns one token, adds up its row of weights in registers, and adds the
// sum to memory once: no exchange between threads, and a sum whose order does
// not depend on timing.
//
// Roles: warps 0-7 and 8-15 sum a token tile each (four of them the first half
// of the columns, four the second); warps 16 and 18 issue its products into
// two buffers of tensor memory in turn; warp 17 loads K pages and query tiles
// with TMA; warp 19 the rows' log-sum-exps.
//
// Measured (4 requests of 2048 new tokens over 8192, 32 query heads to 8 KV
// heads of 128, bf16): 427 us, 1127 TFLOP/s; 315 with the exponentials and
// sums left out, 381 with the products left out.  The small kernel takes 4310.
#pragma once

#include <type_traits>

#include "kvcs_attend_tc.cuh"
#include "kvcs_mass.cuh"

namespace kvcs {

constexpr int kMtKeys = 256;       // tokens of a unit
constexpr int kMtQStages = 3;      // query tiles in flight
constexpr int kMtLseStages = 3;
constexpr int kMtControl = 3 * 1024;   // bytes ahead of the tiles
// Five warpgroups: four for the sums (two per token tile, each for one half of
// a query tile's rows: with one, a scheduler had two warps to hide each step's
// latencies with, and 4 x 2048 queries over 8192 tokens took 435 us, not 423),
// one for the rest.  96 registers a thread at launch, 5 * 96 = 4 * 104 + 64.
constexpr int kMtThreads = 640;
constexpr int kMtSumWarps = 16;
constexpr int kMtRegsSum = 104;
constexpr int kMtRegsOther = 64;

template <int kDim>
struct MtShape {
  static constexpr int kHalves = kDim / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;
  // K of two units, and the query ring
  static constexpr int kSmemBytes = kMtControl + (4 + kMtQStages) * kTileBytes;
};

struct MtParams {
  AttnParams a;
  int box;               // slots a TMA box of K takes
  int heads_in_groups;   // as in TcParams
  int tile_tokens;       // new tokens of a query tile: 128 / group
  u64 timeout_ns;
};

struct MtShared {
  u64 k_full[4], k_empty[4];
  u64 q_full[kMtQStages], q_empty[kMtQStages];
  u64 lse_full[kMtLseStages], lse_empty[kMtLseStages];
  u64 s_full[2][2], s_empty[2][2];   // by token tile and buffer
  u64 half_done[2], half_free[2];    // by token tile: the second half's sums
  u64 drain[2];                      // a product warp's last products
  u32 tmem;
  float half[2][128];
  long long sum[kMtThreads / 32];
  alignas(16) float lse[kMtLseStages][128];   // in units of log 2; read four at once
};
static_assert(sizeof(MtShared) <= kMtControl, "control block");

struct MtUnit {
  Request q;
  int head, key0;       // first token
  int tiles;            // token tiles: 1 or 2
  int tok0;             // first new token any of them is seen by
  int steps;            // query tiles
};

__device__ __forceinline__ int mt_units(const AttnParams &a, const Request &q, int *first_key,
                                        int *first_tok, int *end_key) {
  const int first = a.observe > 0 ? max(0, q.n - a.observe) : 0;
  const long long rows = static_cast<long long>(q.n - first) * a.group;
  *first_tok = first;
  *end_key = min(q.keys, max(0, q.at + q.n));
  *first_key = (a.window > 0 ? max(0, q.at + first - a.window + 1) : 0) / 128 * 128;
  if (rows < a.row_lo || rows > a.row_hi || *end_key <= *first_key) return 0;
  return (*end_key - *first_key + kMtKeys - 1) / kMtKeys;
}

struct MtFinder {
  long long chunk = 0, before = 0;

  __device__ __forceinline__ MtUnit find(const MtParams &p, long long u) {
    const AttnParams &a = p.a;
    const int lane = threadIdx.x & 31;
    MtUnit x;
    x.head = static_cast<int>(u % a.kv_heads);
    const long long pair = u / a.kv_heads;
    int first_key, first_tok, end_key;
    for (;;) {
      const long long r = chunk + lane;
      Request q;
      q.n = q.keys = q.at = 0;
      q.q0 = q.pos0 = 0;
      if (r < a.tab.num_requests) q = read_request(a.tab, r, a.map.block_size, false);
      int fk, ft, ek;
      const int pairs = mt_units(a, q, &fk, &ft, &ek);
      int inc = pairs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const int all = __shfl_sync(0xffffffffu, inc, 31);
      if (pair < before + all) {
        const int at = static_cast<int>(pair - before);
        const int src = __ffs(__ballot_sync(0xffffffffu, inc > at)) - 1;
        const int ahead = __shfl_sync(0xffffffffu, inc - pairs, src);
        x.q.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
        x.q.q0 = __shfl_sync(0xffffffffu, q.q0, src);
        x.q.n = __shfl_sync(0xffffffffu, q.n, src);
        x.q.keys = __shfl_sync(0xffffffffu, q.keys, src);
        x.q.at = __shfl_sync(0xffffffffu, q.at, src);
        x.q.base = 0;
        first_key = __shfl_sync(0xffffffffu, fk, src);
        first_tok = __shfl_sync(0xffffffffu, ft, src);
        end_key = __shfl_sync(0xffffffffu, ek, src);
        x.key0 = first_key + (at - ahead) * kMtKeys;
        break;
      }
      before += all;
      chunk += 32;
    }
    x.tiles = end_key - x.key0 > 128 ? 2 : 1;
    const int last_key = min(end_key, x.key0 + kMtKeys) - 1;
    x.tok0 = max(first_tok, x.key0 - x.q.at);
    int tok1 = x.q.n;
    if (a.window > 0)
      tok1 = static_cast<int>(min(static_cast<long long>(tok1),
                                  static_cast<long long>(last_key) + a.window - x.q.at));
    x.steps = max(0, (tok1 - x.tok0 + p.tile_tokens - 1) / p.tile_tokens);
    return x;
  }
};

template <bool kBf16, int kDim, int kScores>
__global__ void __launch_bounds__(kMtThreads, 1)
    kvcs_mass_tc_kernel(const __grid_constant__ MtParams p, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_q) {
  using S = MtShape<kDim>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  MtShared &sh = *reinterpret_cast<MtShared *>(smem_raw);
  const AttnParams &a = p.a;
  if (blockDim.x != kMtThreads) return;   // (the registers' split counts on every warp)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const u32 k_smem = ptx::smem_addr(smem_raw) + kMtControl, q_smem = k_smem + 4 * S::kTileBytes;
  const u32 k_full = ptx::smem_addr(sh.k_full), k_empty = ptx::smem_addr(sh.k_empty);
  const u32 q_full = ptx::smem_addr(sh.q_full), q_empty = ptx::smem_addr(sh.q_empty);
  const u32 lse_full = ptx::smem_addr(sh.lse_full), lse_empty = ptx::smem_addr(sh.lse_empty);
  const u32 s_full = ptx::smem_addr(sh.s_full), s_empty = ptx::smem_addr(sh.s_empty);
  const u32 half_done = ptx::smem_addr(sh.half_done), half_free = ptx::smem_addr(sh.half_free);
  const u32 drain = ptx::smem_addr(sh.drain);
  const u64 limit = p.timeout_ns;
  if (k_smem & 1023u) {   // the swizzled tiles lie on 1 KiB boundaries (they always do)
    if (tid == 0) raise(a.tab, kStatusTimeout);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(k_full + 8 * i, 1);
      ptx::mbar_init(k_empty + 8 * i, 2);
      ptx::mbar_init(s_full + 8 * i, 1);
      ptx::mbar_init(s_empty + 8 * i, 8);
    }
    for (int i = 0; i < kMtQStages; ++i) {
      ptx::mbar_init(q_full + 8 * i, 1);
      ptx::mbar_init(q_empty + 8 * i, 2);
    }
    for (int i = 0; i < kMtLseStages; ++i) {
      ptx::mbar_init(lse_full + 8 * i, 1);
      ptx::mbar_init(lse_empty + 8 * i, kMtSumWarps);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(half_done + 8 * i, 4);
      ptx::mbar_init(half_free + 8 * i, 4);
      ptx::mbar_init(drain + 8 * i, 1);
    }
    ptx::fence_barrier_init();
  }
  if (warp == 16) tc::tmem_alloc(ptx::smem_addr(&sh.tmem), 512);
  long long mine = 0;
  for (long long r = tid; r < a.tab.num_requests; r += kMtThreads) {
    const Request q = read_request(a.tab, r, a.map.block_size, blockIdx.x == 0);
    int fk, ft, ek;
    mine += mt_units(a, q, &fk, &ft, &ek);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sh.sum[warp] = mine;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  long long units = 0;
  for (int w = 0; w < kMtThreads / 32; ++w) units += sh.sum[w];
  units *= a.kv_heads;
  const u32 tmem = sh.tmem;   // columns: buffers (tile 0: 0, 128; tile 1: 256, 384)
  bool ok = true;
  MtFinder finder;

  if (warp >= kMtSumWarps) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMtRegsOther));
   if (warp == 17) {
    // ------------------------------------------------- loads of K and queries
    const int boxes = 128 / p.box, bs = a.map.block_size;
    u32 n_k = 0, n_q = 0;
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const MtUnit x = finder.find(p, u);
      if (x.steps == 0) continue;
      for (int i = 0; i < x.tiles && ok; ++i, ++n_k) {
        const u32 slot = n_k & 3, bar = k_full + 8 * slot;
        const int key = x.key0 + i * 128 + lane * p.box;
        int block = -1;
        if (lane < boxes && key < x.q.keys) {
          block = a.tab.block_ids[x.q.pos0 + a.map.by_block(key)];
          if (block >= a.map.num_blocks) block = -1;
        }
        const int in = key % bs, sub = a.map.by_sub(in);
        const int group = p.heads_in_groups
                              ? (sub * a.kv_heads + x.head) * (a.map.kbs / 8) + (in - sub * a.map.kbs) / 8
                              : in / 8;
        const int column = p.heads_in_groups ? 0 : x.head * S::kHalves;
        const int n = __popc(__ballot_sync(0xffffffffu, block >= 0));
        if (n_k >= 4) ok = tc::wait(k_empty + 8 * slot, (n_k / 4 - 1) & 1, limit);
        if (!ok) break;
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar, static_cast<u32>(n) * p.box * 128 * S::kHalves);
        __syncwarp();
        if (block >= 0)
          tc::tma_load(k_smem + slot * S::kTileBytes + lane * p.box * 128 * S::kHalves, &map_k, 0, 0,
                       column, group, block, bar);
      }
      for (int t = 0; t < x.steps && ok; ++t, ++n_q) {
        const u32 slot = n_q % kMtQStages, bar = q_full + 8 * slot;
        if (n_q >= kMtQStages) ok = tc::wait(q_empty + 8 * slot, (n_q / kMtQStages - 1) & 1, limit);
        if (!ok) break;
        if (lane == 0) {
          const u32 bytes = static_cast<u32>(p.tile_tokens * a.group) * 128;
          ptx::mbar_arrive_expect_tx(bar, bytes * S::kHalves);
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tc::tma_load(q_smem + slot * S::kTileBytes + h * (128 * 128), &map_q, 0,
                         x.head * a.group, static_cast<int>(x.q.q0) + x.tok0 + t * p.tile_tokens, h, 0,
                         bar);
        }
        __syncwarp();
      }
    }
    // nothing may still be on its way to this CTA, whichever role's wait ran out
    for (u32 i = n_k > 4 ? n_k - 4 : 0; i < n_k; ++i) tc::wait(k_full + 8 * (i & 3), (i / 4) & 1, limit);
    for (u32 i = n_q > kMtQStages ? n_q - kMtQStages : 0; i < n_q; ++i)
      tc::wait(q_full + 8 * (i % kMtQStages), (i / kMtQStages) & 1, limit);
   } else if (warp == 19) {
    // ------------------------------------------------------ log-sum-exps
    // read two query tiles ahead.
    u32 n_l = 0;
    int tok_of[4], head_of[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tok_of[j] = a.by_group(lane + 32 * j);
      head_of[j] = lane + 32 * j - tok_of[j] * a.group;
    }
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const MtUnit x = finder.find(p, u);
      auto read = [&](int t, float (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = x.tok0 + t * p.tile_tokens + tok_of[j];
          v[j] = tok_of[j] < p.tile_tokens && tok < x.q.n
                     ? __ldg(a.lse + (x.q.q0 + tok) * (a.group * a.kv_heads) + x.head * a.group +
                             head_of[j])
                     : 0.0f;
        }
      };
      float v[3][4];
      read(0, v[0]);
      read(1, v[1]);
      for (int t0 = 0; t0 < x.steps && ok; t0 += 3)
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const int t = t0 + e;
          if (t >= x.steps || !ok) break;
          read(t + 2, v[(e + 2) % 3]);
          const u32 slot = n_l % kMtLseStages;
          if (n_l >= kMtLseStages)
            ok = tc::wait(lse_empty + 8 * slot, (n_l / kMtLseStages - 1) & 1, limit);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) sh.lse[slot][lane + 32 * j] = -kLog2e * v[e][j];
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(lse_full + 8 * slot);
          ++n_l;
        }
    }
   } else {
    // -------------------------------------------------------------- products
    constexpr u32 kDescS = tc::instr_desc(kBf16, 128, 128, false);
    const int i = warp == 16 ? 0 : 1;
    const u32 k_low = tc::desc_low(k_smem, 16), q_low = tc::desc_low(q_smem, 16);
    u32 n_k = 0, slot = 0, turn = 0, n_s = 0;
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const MtUnit x = finder.find(p, u);
      if (x.steps == 0) continue;
      const bool work = i < x.tiles;
      const u32 k_slot = (n_k + i) & 3;
      // A warp waits for both K tiles and lets the one go that it does not read:
      // a barrier shows its phase's parity alone, so that a warp that skipped
      // some would take the parity of a slot's use before for its own.
      for (u32 j = 0; j < static_cast<u32>(x.tiles) && ok; ++j, ++n_k) {
        ok = tc::wait(k_full + 8 * (n_k & 3), (n_k / 4) & 1, limit);
        if (!ok) break;
        if (j != static_cast<u32>(i) && tc::elect()) tc::commit(k_empty + 8 * (n_k & 3));
        __syncwarp();
      }
      const u32 kk = k_low + k_slot * (S::kTileBytes >> 4);
      for (int t = 0; t < x.steps && ok; ++t) {
        ok = tc::wait(q_full + 8 * slot, turn, limit);
        if (work && n_s >= 2)
          ok = ok && tc::wait(s_empty + 16 * i + 8 * (n_s & 1), (n_s / 2 - 1) & 1, limit);
        if (!ok) break;
        tc::fence_after();
        const u32 q = q_low + slot * (S::kTileBytes >> 4);
        const u32 d = tmem + i * 256 + (n_s & 1) * 128;
        if (tc::elect()) {
          if (work) {
#pragma unroll
            for (int s = 0; s < kDim / 16; ++s)
              tc::mma_ss(d, tc::desc<S::kHalves * 1024>(kk + (((s >> 2) * 1024 + (s & 3) * 32) >> 4)),
                         tc::desc<1024>(q + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4)), kDescS,
                         s > 0);
            tc::commit(s_full + 16 * i + 8 * (n_s & 1));
          }
          tc::commit(q_empty + 8 * slot);
          if (work && t == x.steps - 1) tc::commit(k_empty + 8 * k_slot);
        }
        __syncwarp();
        n_s += work;
        if (++slot == kMtQStages) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    // the products issued so far end before tensor memory is given back, a
    // wait of whichever role ran out
    if (tc::elect()) tc::commit(drain + 8 * i);
    __syncwarp();
    if (!tc::wait(drain + 8 * i, 0, limit)) ok = false;
   }
  } else {
    // ------------------------------------------------------------------ sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMtRegsSum));
    const int i = warp >> 3, hf = warp >> 2 & 1, wq = warp & 3;
    const u32 lanes = (static_cast<u32>(wq * 32) << 16) + hf * 64;
    u32 n_s = 0, n_l = 0, n_h = 0;
    for (long long u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const MtUnit x = finder.find(p, u);
      const bool work = i < x.tiles;
      const int warp_key = x.key0 + i * 128 + wq * 32, key = warp_key + lane;
      // this token's visible rows, counted from the unit's first
      const int rows_end = (x.q.n - x.tok0) * a.group;
      const long long g0 = (static_cast<long long>(key) - x.q.at - x.tok0) * a.group;
      const int r_lo = static_cast<int>(max(0ll, min(g0, 1ll << 30)));
      const int r_hi = a.window > 0 ? static_cast<int>(max(0ll, min(
                                          static_cast<long long>(rows_end),
                                          g0 + static_cast<long long>(a.window) * a.group)))
                                    : rows_end;
      float *dst = nullptr;
      if (hf == 0 && work && r_hi > r_lo && key < x.q.keys) {
        const int pos = a.map.by_block(key);
        const long long block = a.tab.block_ids[x.q.pos0 + pos];
        if (block < 0 || block >= a.map.num_blocks)
          raise(a.tab, kStatusBadBlockId);
        else
          dst = a.mass + (block * a.kv_heads + x.head) * a.map.block_size +
                (key - pos * a.map.block_size);
      }
      // rows that every token of the warp sees
      const int all_lo = __shfl_sync(0xffffffffu, r_lo, 31), all_hi = __shfl_sync(0xffffffffu, r_hi, 0);
      const int width = p.tile_tokens * a.group;
      const float sc = kScores == kPlain ? a.scale : 1.0f;
      const u64 sc2 = tc::pair(sc, sc);
      u64 acc[4] = {0, 0, 0, 0};   // pairs of +0
      bool past = false;           // a capped score of the token has passed the cap
      for (int t = 0; t < x.steps; ++t, ++n_l) {
        const u32 slot = n_l % kMtLseStages, ls = ptx::smem_addr(sh.lse[slot]) + hf * 256;
        // (the step's log-sum-exps come from another warp's plain writes: only
        // this wait orders them, the products' commit does not)
        ok = tc::wait(lse_full + 8 * slot, (n_l / kMtLseStages) & 1, limit);
        if (work) ok = ok && tc::wait(s_full + 16 * i + 8 * (n_s & 1), (n_s / 2) & 1, limit);
        if (!ok) break;
        if (work) {
          tc::fence_after();
          u32 s[64];
          const u32 ts = tmem + i * 256 + (n_s & 1) * 128 + lanes;
          tc::ld32(ts, s);
          tc::ld32(ts + 32, s + 32);
          tc::wait_ld();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(s_empty + 16 * i + 8 * (n_s & 1));
          ++n_s;
          const int row0 = t * width + hf * 64;   // this half's first row
          const bool full = width == 128 && all_lo <= row0 && all_hi >= row0 + 64;
          if constexpr (kScores != kPlain) make_scores<kScores>(a, s, full, past);
          // weights, 0 where the row does not see the token (whatever the
          // row's scores and its log-sum-exp are)
          auto add = [&](auto masked) {
            const int lo = r_lo - row0, hi = min(r_hi - row0, width - hf * 64);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const uint4 v = lds128(ls + c * 4);   // -lse of four rows
              float y[4];
              tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2,
                                  tc::pair(__uint_as_float(v.x), __uint_as_float(v.y))), y[0], y[1]);
              tc::unpair(tc::fma2(tc::pair(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc2,
                                  tc::pair(__uint_as_float(v.z), __uint_as_float(v.w))), y[2], y[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[j] = ex2(y[j]);
                if (decltype(masked)::value && (c + j < lo || c + j >= hi)) y[j] = 0.0f;
              }
              acc[c / 2 & 3] = tc::add2(acc[c / 2 & 3], tc::pair(y[0], y[1]));
              acc[c / 2 + 1 & 3] = tc::add2(acc[c / 2 + 1 & 3], tc::pair(y[2], y[3]));
            }
          };
          if (__builtin_expect(full, 1))
            add(std::false_type());
          else
            add(std::true_type());
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(lse_empty + 8 * slot);
      }
      if (!ok) break;
      if (!work || x.steps == 0) continue;
      float a0, a1;
      tc::unpair(tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3])), a0, a1);
      // the second half hands its sums to the first
      if (hf) {
        if (n_h > 0) ok = tc::wait(half_free + 8 * i, (n_h - 1) & 1, limit);
        if (!ok) break;
        sh.half[i][wq * 32 + lane] = a0 + a1;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(half_done + 8 * i);
      } else {
        ok = tc::wait(half_done + 8 * i, n_h & 1, limit);
        if (!ok) break;
        const float other = sh.half[i][wq * 32 + lane];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(half_free + 8 * i);
        if (dst) atomicAdd(dst, a0 + a1 + other);
      }
      ++n_h;
    }
  }
  if (!ok && lane == 0) raise(a.tab, kStatusTimeout);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 16) tc::tmem_free(tmem, 512);
}

}  // namespace kvcs
