// kvcs_attn_common.cuh -- what the attention, attention-mass and eviction
// kernels share: device-side call parameters, the reading of the request
// tables, page addressing for every layout, and the small matrix product.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvcs_common.cuh"

namespace kvcs {

constexpr int kKvBf16 = 0;
constexpr int kKvFp16 = 1;
constexpr int kKvFp8 = 2;  // e4m3; queries are bf16 or fp16
// 8-bit caches with a scale for each token and head (extended views only)
constexpr int kKvInt8Scaled = 3;
constexpr int kKvFp8Scaled = 4;
template <int kType>
constexpr bool kIs8Bit = kType >= kKvFp8;
template <int kType>
constexpr bool kIsScaled = kType >= kKvInt8Scaled;

// Requests of more cached tokens than this are flagged (token indices inside
// a request are 32-bit).
constexpr long long kMaxRequestTokens = 1ll << 30;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Division of 31-bit numbers by a fixed divisor: n * m >> s with
// s = 31 + ceil(log2 d) and m = ceil(2^s / d), exact for every n < 2^31.
struct FastDiv {
  u32 m, s;
  __host__ __device__ static FastDiv of(u32 d) {
    FastDiv f;
    u32 l = 0;
    while ((1ull << l) < d) ++l;
    f.s = 31 + l;
    f.m = static_cast<u32>(((1ull << f.s) + d - 1) / d);
    return f;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(static_cast<u64>(static_cast<u32>(n)) * m >> s);
  }
};

// Where a token's bytes are: half (K, V), block, slot, head and 16-byte
// chunk each add their stride; kernel sub-blocks add sub_stride.
struct PageMap {
  const unsigned char *base;
  long long num_blocks;
  long long half_stride;
  long long block_stride;
  long long sub_stride;    // HND kernel sub-blocks: bytes between sub-blocks
  int kbs;                 // slots per sub-block (block_size if none)
  int slot_stride;
  long long head_stride;
  int chunk_stride;        // 16 but for x-split pools
  int block_size;
  int halves;
  FastDiv by_block;        // division by block_size and by kbs
  FastDiv by_sub;
};

// Byte offset of (block, slot, head) from the pool's base.
__device__ __forceinline__ long long token_offset(const PageMap &m, long long block, int slot,
                                                  int head) {
  const int sub = m.by_sub(slot);
  return block * m.block_stride + sub * m.sub_stride +
         static_cast<long long>(slot - sub * m.kbs) * m.slot_stride + head * m.head_stride;
}

struct Tables {
  const long long *pos_offsets;
  const long long *first_position;
  const long long *num_tokens;
  const int *block_ids;
  const long long *new_offsets;   // attention and mass
  long long num_requests;
  long long total_positions;
  long long total_new;
  long long max_new;
  u32 *status;
};

// One request as the kernels see it.  Tokens are counted from the first
// listed block on: token 0 is slot 0 of block position first_position.
struct Request {
  long long pos0;   // its first position index
  long long q0;     // its first new token's row
  int n;            // new tokens
  int keys;         // cached tokens in its listed blocks
  int at;           // token index of its first new token (may be negative)
  long long base;   // request position of token 0 (first_position * block_size)
};

__device__ __forceinline__ void raise(const Tables &t, u32 bit) {
  if (t.status) atomicOr(t.status, bit);
}

// A request's raw table entries.  (Loaded together: a chain of dependent
// loads at the start of every CTA would be most of a small call's time.)
struct RawRequest {
  long long a, b, first, tokens, new_a, new_b;
};

template <bool kNew>
__device__ __forceinline__ RawRequest load_request(const Tables &t, long long r) {
  RawRequest w;
  w.a = t.pos_offsets[r];
  w.b = t.pos_offsets[r + 1];
  w.first = t.first_position[r];
  w.tokens = t.num_tokens[r];
  w.new_a = kNew ? t.new_offsets[r] : 0;
  w.new_b = kNew ? t.new_offsets[r + 1] : 0;
  return w;
}

// Tokens of a request; flagged tables hold none.  Reads only entries the
// tables have, whatever these hold.
__device__ __forceinline__ Request tokens_of(const Tables &t, const RawRequest &w, int block_size,
                                             bool report) {
  Request q;
  q.n = 0;
  q.q0 = 0;
  q.at = 0;
  q.keys = 0;
  q.pos0 = w.a;
  q.base = 0;
  if (w.a < 0 || w.b < w.a || w.b > t.total_positions || w.first < 0 || w.first > (1ll << 31)) {
    if (report) raise(t, kStatusBadRequests);
    return q;
  }
  q.base = w.first * block_size;
  long long keys = max(w.tokens, 0ll) - q.base;
  const long long listed = (w.b - w.a) * block_size;
  if (keys > listed) keys = listed;
  if (keys > kMaxRequestTokens) {
    if (report) raise(t, kStatusBadRequests);
    return q;
  }
  q.keys = keys < 0 ? 0 : static_cast<int>(keys);
  return q;
}

__device__ __forceinline__ Request read_tokens(const Tables &t, long long r, int block_size,
                                               bool report) {
  return tokens_of(t, load_request<false>(t, r), block_size, report);
}

// As read_tokens, with the request's new tokens: they are its last ones.
__device__ __forceinline__ Request read_request(const Tables &t, long long r, int block_size,
                                                bool report) {
  const RawRequest w = load_request<true>(t, r);
  Request q = tokens_of(t, w, block_size, report);
  if (w.new_a < 0 || w.new_b < w.new_a || w.new_b > t.total_new || w.new_b - w.new_a > t.max_new) {
    if (report) raise(t, kStatusBadRequests);
    return q;
  }
  q.q0 = w.new_a;
  q.n = static_cast<int>(w.new_b - w.new_a);
  long long at = max(w.tokens, 0ll) - q.n - q.base;
  const long long lim = 1ll << 30;
  at = at < -lim ? -lim : at > lim ? lim : at;
  q.at = static_cast<int>(at);
  return q;
}

struct AttnParams {
  Tables tab;
  PageMap map;
  const void *q;          // [total_new] rows of q_stride elements
  long long q_stride;
  void *out;              // [total_new][q_heads][head_dim], or null (mass)
  float *lse;             // [total_new][q_heads], or null (mass: read)
  float *mass;            // mass: [num_blocks][kv_heads][block_size]
  float *part;            // partial results of groups split between CTAs
  u32 *tickets;           // one per CTA, zeroed before the launch
  int kv_heads, group, head_dim;
  FastDiv by_group;
  int q_bf16;             // fp8 caches: queries (and out) are bf16, else fp16
  int window;             // 0: none
  int observe;            // mass: last new tokens observed (0: all)
  int unit8;              // pools only 8-byte aligned: copies of 8 bytes
  int runs;               // 16 aligned tokens always lie in one page, one after
                          // another, in whole 16-byte pieces of the full width
  int row_lo, row_hi;     // requests whose rows (new tokens * group) lie in
                          // [row_lo, row_hi] belong to this launch
  float scale;            // scale * k_scale * log2(e): scores in units of log 2
  float cap, inv_cap;     // capped scores: cap * log2(e) and scale / cap; 0: none
  float v_scale;
  // extended views
  long long sinks;        // request positions below it stay visible past the window
  const int *place;       // trees: each new token's depth, -1 where its request's tree is bad; or null
  const u32 *kin;         // trees: [total_new][kin_words], bit j: the token sees new token j
  int kin_words;
  const float *k_scales;  // [num_blocks][kv_heads][block_size], or null
  const float *v_scales;
};

// ---------------------------------------------------------------------------
// Extended views: what a row sees
// ---------------------------------------------------------------------------

// Tokens of the request's listed blocks that stay visible past a window.
__device__ __forceinline__ int sink_keys_of(const AttnParams &p, const Request &q) {
  if (p.window == 0) return 0;
  const long long n = p.sinks - q.base;
  return n <= 0 ? 0 : n < q.keys ? static_cast<int>(n) : q.keys;
}

// Bits [0, n) of a word.
__device__ __forceinline__ u32 bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// A row sees the tokens below `lim` (a tree's: the cached ones before the new
// tokens) that are after at - window or below the sinks, and of a tree's new
// tokens (token index `tail` on) those of its mask.
struct RowSight {
  int lim, at;
  const u32 *kin;   // the row's mask words, or null
};

__device__ __forceinline__ RowSight row_sight(const AttnParams &p, const Request &q, int token) {
  RowSight s;
  s.at = q.at + token;
  s.lim = s.at + 1;
  s.kin = nullptr;
  if (p.place) {
    const int depth = p.place[q.q0 + token];
    s.at = q.at + depth;
    s.lim = depth < 0 ? -(1 << 30) : q.at;
    s.kin = p.kin + (q.q0 + token) * p.kin_words;   // (a bad tree's are 0)
  }
  return s;
}

// Bits of the 32 tokens from key0 on that the row sees (tokens that do not
// exist not yet taken out).
__device__ __forceinline__ u32 seen_bits(const AttnParams &p, const RowSight &s, int tail,
                                         int sink_keys, int key0) {
  u32 see = bits_below(s.lim - key0);
  if (p.window > 0)
    see &= ~bits_below(max(s.at - p.window + 1, 0) - key0) | bits_below(sink_keys - key0);
  if (s.kin) {
    const int o = key0 - tail;
    if (o >= 0) {
      const int w = o >> 5;
      const u32 lo = w < p.kin_words ? s.kin[w] : 0u;
      const u32 hi = w + 1 < p.kin_words ? s.kin[w + 1] : 0u;
      see |= __funnelshift_r(lo, hi, o & 31);
    } else if (o > -32) {
      see |= s.kin[0] << -o;
    }
  }
  return see;
}

// ---------------------------------------------------------------------------
// Arithmetic
// ---------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Coefficients, from the lowest, of P with tanh(x) = x P(x^2) for |x| <= 1: the
// Chebyshev interpolation of degree 6 of tanh(x) / x in x^2, computed in 64 bits.
__device__ __forceinline__ constexpr float tanh_p(int k) {
  constexpr float kP[7] = {9.999999404e-01f,  -3.333282769e-01f, 1.332507581e-01f, -5.345164612e-02f,
                           2.027970739e-02f, -6.194324698e-03f, 1.038025133e-03f};
  return kP[k];
}

// Caps, in units of log 2, up to which the error of tanh's definition below,
// about 2^-22 of the cap, stays under 2^-15 of a score's unit (a cap of 128),
// far below the weights' rounding. (Scores past it through `capped` too: 4
// requests of 2048 new tokens over 8192, a cap of 2, 2107 us, not 1510; their
// mass 1725, not 1092; decode over fp8, a cap of 30, 95, not 92.)
constexpr float kNearCap = 128.0f * kLog2e;

// cap * tanh(x) by the definition, 1 - 2 / (e^2x + 1).  (The hardware's tanh is
// off by 2^-11 of the cap.)
__device__ __forceinline__ float near_capped(float cap, float x) {
  return cap * (1.0f - __fdividef(2.0f, ex2(x * (2.0f * kLog2e)) + 1.0f));
}

// cap * tanh(x) for any cap, within 2^-21 of itself: below |x| = 1/2, where the
// definition's error would be many times the score (a cap of 10^6 over scores
// of 10: a quarter of a unit), x P(x^2), P the Chebyshev interpolation of
// degree 4 of tanh(x) / x.  Both are made and one is taken: a branch for each
// score costs more.
__device__ __forceinline__ float capped(float cap, float x) {
  const float u = x * x;
  float y = 0.017131345346570015f;
  y = fmaf(y, u, -0.05298423767089844f);
  y = fmaf(y, u, 0.133247509598732f);
  y = fmaf(y, u, -0.3333306908607483f);
  y = fmaf(y, u, 1.0f);
  const float small = x * cap * y;
  const float large = near_capped(cap, x);
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %1, 0f3F000000;\n\tselp.f32 %0, %2, %3, p;\n\t}"
      : "=f"(r)
      : "f"(fabsf(x)), "f"(small), "f"(large));
  return r;
}

// A raw product as a score in units of log 2.
__device__ __forceinline__ float score_of(const AttnParams &p, float raw, float row_scale) {
  if (p.cap > kNearCap) return capped(p.cap, raw * row_scale * p.inv_cap);
  if (p.cap != 0.0f) return near_capped(p.cap, raw * row_scale * p.inv_cap);
  return raw * row_scale * p.scale;
}

// A thread's products of two rows by two tokens by two, as scores.
__device__ __forceinline__ void scores_of(const AttnParams &p, float (&s)[2][4], const float (&rs)[2]) {
  if (p.cap > kNearCap) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s[i >> 2][i & 3] = capped(p.cap, s[i >> 2][i & 3] * rs[i >> 1 & 1] * p.inv_cap);
  } else if (p.cap != 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s[i >> 2][i & 3] = near_capped(p.cap, s[i >> 2][i & 3] * rs[i >> 1 & 1] * p.inv_cap);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] *= rs[i >> 1 & 1] * p.scale;
  }
}

// A token's scale: one that is not finite is NaN (an infinite K scale times a
// negative product would else be a weight of 0).
__device__ __forceinline__ float finite_or_nan(float scale) { return fmaf(scale, 0.0f, scale); }

// D += A B, m16n8k16.
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], u32 a0, u32 a1, u32 a2, u32 a3, u32 b0,
                                         u32 b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats as a pair of 16-bit values, `lo` in the low half.
template <bool kBf16>
__device__ __forceinline__ u32 pack2(float lo, float hi) {
  u32 r;
  if (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float half_bits_to_float(u32 bits, bool bf16) {
  if (bf16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// Four e4m3 values as two pairs of fp16 (exact).
__device__ __forceinline__ void fp8x4_to_half(u32 v, u32 &lo, u32 &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// An 8x8 matrix of 16-bit values, a row per four lanes, turned round.
__device__ __forceinline__ u32 movmatrix(u32 v) {
  u32 r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Four int8 values as two pairs of fp16 (exact): a byte plus 128 in the low
// bits of 1024 is the fp16 number 1152 + value.
__device__ __forceinline__ void int8x4_to_half(u32 v, u32 &lo, u32 &hi) {
  v ^= 0x80808080u;
  const __half2 off = __floats2half2_rn(1152.0f, 1152.0f);
  u32 a = __byte_perm(v, 0x64646464u, 0x4140), b = __byte_perm(v, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
  lo = *reinterpret_cast<const u32 *>(&x);
  hi = *reinterpret_cast<const u32 *>(&y);
}
template <int kType>
__device__ __forceinline__ void bytes_to_half(u32 v, u32 &lo, u32 &hi) {
  if constexpr (kType != kKvInt8Scaled) fp8x4_to_half(v, lo, hi);
  else int8x4_to_half(v, lo, hi);
}

// ---------------------------------------------------------------------------
// Asynchronous copies; `bytes` of 0 fills the destination with zeros.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cp_async16(u32 dst, const void *src, u32 bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async8z(u32 dst, const void *src, u32 bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4z(u32 dst, const void *src, u32 bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint4 lds128(u32 a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32f(u32 a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(u32 a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

}  // namespace kvcs
