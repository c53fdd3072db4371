// kvcs_attend.cu -- host side of the operators that read and thin out paged
// caches: attention of new tokens, attention mass, and eviction (kvcs.h).
// As in kvcs.cu, host arguments are checked before any CUDA call, nothing is
// allocated, and all work goes to the caller's stream.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "kvcs.h"
#include "kvcs_attend_host.h"
#include "kvcs_evict.cuh"

namespace kvcs {
namespace {

constexpr u64 kAttendTimeoutNs = 2000000000ull;  // 2 s per wait

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int element_bytes(int kv_dtype) { return kv_dtype == KVCS_DTYPE_FP8_E4M3 ? 1 : 2; }

PageMap page_map(const kvcs_cache &c, int block_size) {
  PageMap m;
  std::memset(&m, 0, sizeof(m));
  const long long hb = c.head_bytes, heads = c.num_heads;
  const long long page = block_size * heads * hb;
  m.base = static_cast<const unsigned char *>(c.base);
  m.num_blocks = c.num_blocks;
  m.half_stride = c.half_stride ? c.half_stride : c.num_blocks * page;
  m.block_stride = c.block_stride ? c.block_stride : page;
  m.block_size = block_size;
  m.kbs = block_size;
  m.halves = c.layout == KVCS_LAYOUT_LATENT ? 1 : 2;
  m.chunk_stride = 16;
  switch (c.layout) {
    case KVCS_LAYOUT_HND:
      if (c.kernel_block_size > 0) m.kbs = c.kernel_block_size;
      m.sub_stride = heads * m.kbs * hb;
      m.slot_stride = static_cast<int>(hb);
      m.head_stride = m.kbs * hb;
      break;
    case KVCS_LAYOUT_XSPLIT:
      m.slot_stride = 16;
      m.head_stride = block_size * hb;
      m.chunk_stride = block_size * 16;
      break;
    default:  // NHD, latent
      m.slot_stride = static_cast<int>(heads * hb);
      m.head_stride = hb;
      break;
  }
  m.by_block = FastDiv::of(static_cast<u32>(m.block_size));
  m.by_sub = FastDiv::of(static_cast<u32>(m.kbs));
  return m;
}

// Copies of 16 bytes need every piece of every token on a 16-byte boundary.
bool needs_8(const kvcs_cache &c) {
  return !aligned(c.base, 16) || c.half_stride % 16 || c.block_stride % 16 || c.head_bytes % 16;
}

int check_tables(const kvcs_requests *reqs, int64_t total_positions, const uint32_t *status) {
  if (!reqs || total_positions < 0 || reqs->num_requests < 0) return KVCS_EINVAL;
  if (!aligned(reqs->pos_offsets, 8) || !aligned(reqs->first_position, 8) ||
      !aligned(reqs->num_tokens, 8) || !aligned(reqs->block_ids, 4) || !aligned(status, 4))
    return KVCS_EINVAL;
  if (reqs->num_requests == 0) return KVCS_OK;
  if (!reqs->pos_offsets || !reqs->first_position || !reqs->num_tokens) return KVCS_EINVAL;
  if (total_positions > 0 && !reqs->block_ids) return KVCS_EINVAL;
  return KVCS_OK;
}

// Checks shared by attention and attention mass.
int check_attention(const kvcs_cache *cache, int32_t block_size, const kvcs_attention *a) {
  if (!cache || !a) return KVCS_EINVAL;
  kvcs_cache plain = *cache;
  plain.column = 0;
  const int rc = check_caches(&plain, 1, block_size);
  if (rc != KVCS_OK) return rc;
  if (cache->layout == KVCS_LAYOUT_STATE) return KVCS_EINVAL;
  if (a->kv_dtype < KVCS_DTYPE_BF16 || a->kv_dtype > KVCS_DTYPE_FP8_E4M3) return KVCS_EINVAL;
  if (a->q_dtype != KVCS_DTYPE_BF16 && a->q_dtype != KVCS_DTYPE_FP16) return KVCS_EINVAL;
  if (a->kv_dtype != KVCS_DTYPE_FP8_E4M3 && a->kv_dtype != a->q_dtype) return KVCS_EINVAL;
  if (a->q_heads < 1 || a->q_heads % cache->num_heads) return KVCS_EINVAL;
  if (a->total_new < 0 || a->max_new < 0 || a->max_new > a->total_new || a->window < 0 ||
      a->observe < 0 || a->q_stride < 0)
    return KVCS_EINVAL;
  if (!std::isfinite(a->scale) || !std::isfinite(a->k_scale) || !std::isfinite(a->v_scale) ||
      !std::isfinite(a->softcap) || a->softcap < 0.0f)
    return KVCS_EINVAL;
  // (and what is made of them: an infinite factor turns a product of 0 into
  // NaN, and a quotient below the normal numbers has lost bits that a cap this
  // large brings back)
  const float factor = a->scale * a->k_scale, quotient = a->softcap > 0.0f ? factor / a->softcap : 0.0f;
  if (!std::isfinite(factor * kLog2e) || !std::isfinite(a->softcap * kLog2e) ||
      !std::isfinite(quotient) || (a->softcap > 1e18f && factor != 0.0f && !std::isnormal(quotient)))
    return KVCS_EINVAL;
  if (cache->layout == KVCS_LAYOUT_LATENT) return KVCS_EUNSUPPORTED;
  const int es = element_bytes(a->kv_dtype);
  if (cache->head_bytes % (8 * es) || cache->head_bytes / es > 256) return KVCS_EUNSUPPORTED;
  const int64_t dim = cache->head_bytes / es;
  if (a->q_stride && (a->q_stride % 8 || a->q_stride < a->q_heads * dim)) return KVCS_EINVAL;
  if (static_cast<double>(a->total_new) * a->q_heads >= 2147483648.0) return KVCS_EUNSUPPORTED;
  // (a request's positions stay below 2^31: 2^30 cached tokens and fewer new ones)
  if ((a->max_new > 0 ? a->max_new : a->total_new) >= kMaxRequestTokens) return KVCS_EUNSUPPORTED;
  if (static_cast<double>(block_size) * cache->num_heads * cache->head_bytes >= 2147483648.0)
    return KVCS_EUNSUPPORTED;
  return KVCS_OK;
}

AttnParams attn_params(const kvcs_cache *cache, int32_t block_size, const kvcs_requests *reqs,
                       int64_t total_positions, const kvcs_attention *a, uint32_t *status) {
  AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.tab.pos_offsets = reinterpret_cast<const long long *>(reqs->pos_offsets);
  p.tab.first_position = reinterpret_cast<const long long *>(reqs->first_position);
  p.tab.num_tokens = reinterpret_cast<const long long *>(reqs->num_tokens);
  p.tab.block_ids = reinterpret_cast<const int *>(reqs->block_ids);
  p.tab.new_offsets = reinterpret_cast<const long long *>(a->new_offsets);
  p.tab.num_requests = reqs->num_requests;
  p.tab.total_positions = total_positions;
  p.tab.total_new = a->total_new;
  p.tab.max_new = a->max_new > 0 ? a->max_new : a->total_new;
  p.tab.status = status;
  p.map = page_map(*cache, block_size);
  p.head_dim = cache->head_bytes / element_bytes(a->kv_dtype);
  p.q = a->q;
  p.q_stride = a->q_stride ? a->q_stride : static_cast<long long>(a->q_heads) * p.head_dim;
  p.out = a->out;
  p.lse = a->lse;
  p.kv_heads = cache->num_heads;
  p.group = a->q_heads / cache->num_heads;
  p.by_group = FastDiv::of(static_cast<u32>(p.group));
  p.q_bf16 = a->q_dtype == KVCS_DTYPE_BF16;
  p.window = static_cast<int>(a->window < kMaxRequestTokens ? a->window : 0);
  p.observe = static_cast<int>(std::min<int64_t>(a->observe, kMaxRequestTokens));
  p.unit8 = needs_8(*cache) ? 1 : 0;
  p.runs = !p.unit8 && p.map.kbs % 16 == 0 &&
           (p.head_dim == 64 || p.head_dim == 128 || p.head_dim == 256);
  p.row_lo = 1;
  p.row_hi = 0x7fffffff;
  const float s = a->scale * a->k_scale;
  p.scale = s * kLog2e;
  if (a->softcap > 0.0f) {
    p.cap = a->softcap * kLog2e;
    p.inv_cap = s / a->softcap;
  }
  p.v_scale = a->v_scale;
  return p;
}

// Slots a TMA box takes: runs of consecutive slots that lie in one page and
// one tile.  Below 8 the boxes would not start on the swizzle's 1 KiB period.
int tc_box(const kvcs_cache &c, int block_size) {
  const int run = c.layout == KVCS_LAYOUT_HND && c.kernel_block_size > 0 ? c.kernel_block_size
                                                                        : block_size;
  int box = kTcKeys;
  while (run % box) box /= 2;
  return box;
}

// Whether the tensor-memory kernel takes the cache: 16-bit heads of 64 or
// 128 in token rows, everything on 16-byte boundaries, and extents and
// strides a tensor map can hold.
bool tc_takes(const kvcs_cache &c, int block_size, const kvcs_attention &a) {
  const PageMap m = page_map(c, block_size);
  return a.kv_dtype != KVCS_DTYPE_FP8_E4M3 && (c.head_bytes == 128 || c.head_bytes == 256) &&
         (c.layout == KVCS_LAYOUT_NHD || c.layout == KVCS_LAYOUT_HND) && !needs_8(c) &&
         tc_box(c, block_size) >= 8 && c.num_blocks > 0 && c.num_blocks < (1ll << 31) &&
         m.block_stride < (1ll << 40);
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// One half (K or V) of a pool as a tensor [block][group of 8 slots][128-byte
// column][slot of the group][64 elements], read in boxes of `box` slots of one
// head.  NHD: a token's columns run through its heads; HND: a block's groups
// run through its sub-blocks and heads.
bool half_map(CUtensorMap *map, const PageMap &m, int half, int heads, int dim, bool bf16, int box,
              bool heads_in_groups) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const int halves = dim / 64;
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(heads_in_groups ? halves : heads * halves),
                              static_cast<cuuint64_t>(m.block_size / 8) *
                                  (heads_in_groups ? heads : 1),
                              static_cast<cuuint64_t>(m.num_blocks)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(m.slot_stride), 128,
                                 8 * static_cast<cuuint64_t>(m.slot_stride),
                                 static_cast<cuuint64_t>(m.block_stride)};
  const cuuint32_t boxes[5] = {64, 8, static_cast<cuuint32_t>(halves),
                               static_cast<cuuint32_t>(box / 8), 1};
  const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                const_cast<unsigned char *>(m.base) + half * m.half_stride, dims, strides, boxes,
                steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries of one call as a tensor [half][token][head][64 elements], read in
// boxes of one KV head's query group by `tokens` new tokens.
bool query_map(CUtensorMap *map, const AttnParams &p, bool bf16, int tokens) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const int halves = p.head_dim / 64;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(p.kv_heads) * p.group,
                              static_cast<cuuint64_t>(p.tab.total_new),
                              static_cast<cuuint64_t>(halves), 1};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(p.head_dim) * 2,
                                 static_cast<cuuint64_t>(p.q_stride) * 2, 128,
                                 static_cast<cuuint64_t>(p.q_stride) * 2};
  const cuuint32_t boxes[5] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(tokens),
                               1, 1};
  const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                const_cast<void *>(p.q), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The launches of one attention call.  A request's rows are its new tokens
// times the query heads per KV head: up to 16 rows go to the narrow kernel,
// more to the tensor-memory kernel, or to the wide one where that does not
// take the cache.  max_new bounds the rows, so a decode step launches only
// the narrow kernel; when total_new = num_requests * max_new every request
// has max_new tokens and one kernel is enough either way.
//
// 16 rows are one warp's product rows.  Beyond, with 32 query heads to 8 KV
// heads of 128, bf16, the wide kernel against the tensor-memory one: 64
// requests of 2048 tokens, 20 rows 197 and 122 us, 64 rows 247 and 127; one of
// 32,768 tokens 93 and 35, 197 and 38; one of 1024 tokens, 32 rows, 37 and 16.
constexpr int kNarrowRows = 16;
// Observed rows the small mass kernel takes, at most (it against the
// tensor-memory one, 64 requests of 2048 tokens: 16 rows 52 and 107 us, 32
// rows 93 and 107, 40 rows 117 and 107, 64 rows 147 and 110; 4 of 8192: 15 and
// 31, 25 and 31, 32 and 31, 39 and 30).
constexpr int kMassRows = 32;
// Token tiles a part holds, at least (on average).  256 rows over 1024, 512 and
// 2048 tokens: at least 2 tiles 23, 23 and 23 us; 4 tiles 26, 18 and 26; 8
// tiles 23, 18 and 31.
constexpr int kTcMinTiles = 4;

struct AttendPlan {
  bool narrow, wide, tc;
  int narrow_grid, wide_grid;      // wide_grid: the wide or the tensor-memory kernel's
  int splits;                      // tensor-memory kernel: parts per unit
  long long units;                 // and units, at most
  long long part_floats;
};

AttendPlan plan_attend(const AttnParams &p, const kvcs_cache &c, const kvcs_attention &a, int sms) {
  AttendPlan pl;
  std::memset(&pl, 0, sizeof(pl));
  const long long rows = p.tab.max_new * p.group;
  const long long R = p.tab.num_requests;
  const bool alike = p.tab.total_new == R * p.tab.max_new;
  const bool more = rows > kNarrowRows;
  pl.tc = more && tc_takes(c, p.map.block_size, a);
  pl.wide = more && !pl.tc;
  pl.narrow = !more || (!alike && p.group <= kNarrowRows);
  long long nf = 0, wf = 0;
  auto shape = a.kv_dtype == KVCS_DTYPE_BF16   ? &AttendLaunch<kKvBf16>::shape
               : a.kv_dtype == KVCS_DTYPE_FP16 ? &AttendLaunch<kKvFp16>::shape
                                               : &AttendLaunch<kKvFp8>::shape;
  shape(p.head_dim, false, sms, &pl.narrow_grid, &nf);
  shape(p.head_dim, true, sms, &pl.wide_grid, &wf);
  if (pl.tc) {
    const long long tiles = alike ? R * ((rows + kTcRows - 1) / kTcRows)
                                  : p.tab.total_new * p.group / kTcRows + std::min(R, p.tab.total_new);
    const long long units = tiles * p.kv_heads;
    // few units: the token ranges are split, as far as their parts stay long
    pl.units = units;
    const long long key_tiles = p.tab.total_positions * p.map.block_size / std::max(1ll, R) / kTcKeys;
    pl.splits = static_cast<int>(std::max(
        1ll, std::min({sms / std::max(1ll, units), key_tiles / kTcMinTiles,
                       static_cast<long long>(kTcMaxSplits)})));
    pl.wide_grid = static_cast<int>(std::min<long long>(sms, units * pl.splits));
    wf = pl.splits > 1 ? units * pl.splits * kTcRows * (p.head_dim + 4) : 0;
  }
  pl.part_floats = std::max(pl.narrow ? nf : 0, pl.wide || pl.tc ? wf : 0);
  return pl;
}

// Counters first (both launches'), then the partial results.
long long attend_tickets(const AttendPlan &pl) {
  return (pl.narrow ? pl.narrow_grid : 0) + (pl.wide ? pl.wide_grid : 0);
}
int64_t attend_workspace(const AttendPlan &pl) {
  return std::max((attend_tickets(pl) * 4 + 255) / 256 * 256, 256ll) + pl.part_floats * 4;
}

constexpr int kEvictSmemTokens = 49152;   // 192 KiB of scores

// As many caches from `lo` on as one launch holds and its grids can number
// (column groups a row: eight of its halves at most, or as many as its pieces
// need with a thread each; spans only where the rows are few).
struct EvictLaunch {
  int caches;
  long long rows;
};
EvictLaunch evict_launch(const kvcs_cache *caches, int32_t lo, int32_t num_caches,
                         int64_t num_requests) {
  EvictLaunch l = {0, 0};
  double groups = 0.0;
  while (lo + l.caches < num_caches && l.caches < kEvictCaches) {
    const kvcs_cache &c = caches[lo + l.caches];
    const long long rows = l.rows + c.num_heads;
    const int pieces = c.head_bytes / (needs_8(c) ? 8 : 16);
    groups = std::max(groups, 2.0 * std::max(8, (pieces + kEvictThreads - 1) / kEvictThreads));
    if (static_cast<double>(rows) * num_requests * groups >= 2147483648.0) break;
    l.rows = rows;
    ++l.caches;
  }
  return l;
}

// Checks of the caches of an eviction.
int check_evict_caches(const kvcs_cache *caches, int32_t num_caches, int32_t block_size) {
  if (!caches || num_caches < 1) return KVCS_EINVAL;
  std::vector<kvcs_cache> plain(caches, caches + num_caches);
  for (kvcs_cache &c : plain) c.column = 0;
  const int rc = check_caches(plain.data(), num_caches, block_size);
  if (rc != KVCS_OK) return rc;
  for (int32_t i = 0; i < num_caches; ++i) {
    if (caches[i].layout == KVCS_LAYOUT_STATE) return KVCS_EINVAL;
    if (static_cast<double>(block_size) * caches[i].num_heads * caches[i].head_bytes >=
        2147483648.0)
      return KVCS_EUNSUPPORTED;
  }
  return KVCS_OK;
}

// What an eviction's sizes must stay below, whatever its launches: 31-bit token
// and row numbers.
int check_evict_sizes(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                      int64_t num_requests, int64_t total_positions) {
  if (static_cast<double>(total_positions) * block_size >= 2147483648.0) return KVCS_EUNSUPPORTED;
  for (int32_t lo = 0; lo < num_caches;) {
    const EvictLaunch l = evict_launch(caches, lo, num_caches, num_requests);
    if (l.caches == 0) return KVCS_EUNSUPPORTED;
    lo += l.caches;
  }
  return KVCS_OK;
}

// Launches follow one another on the stream and share the space.
int64_t evict_workspace(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                        int64_t num_requests, int64_t total_positions) {
  long long rows = 0;
  for (int32_t lo = 0; lo < num_caches;) {
    const EvictLaunch l = evict_launch(caches, lo, num_caches, num_requests);
    rows = std::max(rows, l.rows);
    lo += l.caches;
  }
  return rows * total_positions * block_size * 4;
}

// The launches over one group of caches; returns how many, or an error code.
template <int kCaches>
int launch_evict(const EvictCall &call, const kvcs_cache *caches, float *const *scores,
                 long long rows, int parts, int64_t average, int sms, cudaStream_t st) {
  EvictParams<kCaches> p;
  static_cast<EvictCall &>(p) = call;
  p.halves_parts = 1;
  long long first = 0;
  for (int n = 0; n < p.num_caches; ++n) {
    const kvcs_cache &c = caches[n];
    EvictCache &e = p.c[n];
    e.map = page_map(c, p.block_size);
    e.scores = scores[n];
    e.m0 = 2ull * (static_cast<u64>(c.layer) * KVCS_MAX_KV_HEADS_PER_LAYER + c.head_offset) + 1;
    e.heads = c.num_heads;
    e.head_bytes = c.head_bytes;
    e.first_row = static_cast<int>(first);
    e.unit = needs_8(c) ? 8 : 16;
    const int pieces = c.head_bytes / e.unit;
    const int least = std::max(1, 32 / e.unit);
    // (at most a thread per piece)
    e.part_pieces = std::min(kEvictThreads, std::max(std::min(least, pieces),
                                                     (pieces + parts - 1) / parts));
    e.parts = (pieces + e.part_pieces - 1) / e.part_pieces;
    p.halves_parts = std::max(p.halves_parts, e.map.halves * e.parts);
    first += c.num_heads;
  }
  const long long units = rows * p.halves_parts;
  // into fresh blocks by runs of kept tokens too (one request, 40,011 tokens to
  // 32,768: 128 us instead of 460; 20,011 to 4096: 61 instead of 95; with 96
  // rows no difference: 130 and 126)
  p.spans = 1;
  if (p.new_block_ids)
    p.spans = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({average / kEvictChunk, 8ll * sms / units, 64})));
  // (short rows need no leave for more than the standard 48 KiB)
  if (p.smem_tokens * 4 > 32768 &&
      cudaFuncSetAttribute(reinterpret_cast<const void *>(kvcs_evict_select_kernel<kCaches>),
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kEvictSmemTokens * 4) != cudaSuccess)
    return KVCS_ECUDA;
  // large CTAs where the rows are few (8 rows of 20,011 tokens: 98 us with 1024
  // threads, 138 with 256; 1024 rows of 512 to 4096: 234 and 203)
  const int threads = rows < 4ll * sms ? kEvictSelectThreads : kEvictSelectThreads / 4;
  kvcs_evict_select_kernel<kCaches>
      <<<static_cast<unsigned>(rows), threads, p.smem_tokens * 4, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KVCS_ECUDA;
  int launches = 1;
  // a launch for the caches of either piece size
  bool has[2] = {false, false};
  for (int n = 0; n < p.num_caches; ++n) has[p.c[n].unit == 16] = true;
  const dim3 grid(static_cast<unsigned>(units * p.spans));
  for (int u = 0; u < 2; ++u) {
    if (!has[u]) continue;
    auto move = p.block_sums ? (u ? kvcs_evict_move_kernel<kCaches, true, true>
                                  : kvcs_evict_move_kernel<kCaches, true, false>)
                             : (u ? kvcs_evict_move_kernel<kCaches, false, true>
                                  : kvcs_evict_move_kernel<kCaches, false, false>);
    move<<<grid, kEvictThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KVCS_ECUDA;
    ++launches;
  }
  return launches;
}

__global__ void __launch_bounds__(1024) kvcs_tickets_kernel(u32 *tickets, int n) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  for (int i = threadIdx.x; i < n; i += blockDim.x) tickets[i] = 0;
}

}  // namespace
}  // namespace kvcs

using namespace kvcs;

extern "C" {

int kvcs_attention_workspace(const kvcs_cache *cache, int32_t block_size, int64_t num_requests,
                             int64_t total_positions, const kvcs_attention *att, int32_t num_sms, int64_t *bytes) {
  if (!bytes || num_requests < 0 || total_positions < 0) return KVCS_EINVAL;
  const int rc = check_attention(cache, block_size, att);
  if (rc != KVCS_OK) return rc;
  int sms = num_sms;
  if (sms <= 0 && device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  kvcs_requests reqs;
  std::memset(&reqs, 0, sizeof(reqs));
  reqs.num_requests = num_requests;
  const AttnParams p = attn_params(cache, block_size, &reqs, total_positions, att, nullptr);
  *bytes = attend_workspace(plan_attend(p, *cache, *att, sms));
  return KVCS_OK;
}

int kvcs_paged_attention(const kvcs_cache *cache, int32_t block_size, const kvcs_requests *reqs,
                         int64_t total_positions, const kvcs_attention *att, uint32_t *status,
                         void *stream) {
  int rc = check_attention(cache, block_size, att);
  if (rc != KVCS_OK) return rc;
  rc = check_tables(reqs, total_positions, status);
  if (rc != KVCS_OK) return rc;
  if (att->total_new == 0 || reqs->num_requests == 0) return KVCS_OK;
  if (!att->q || !att->out || !att->new_offsets || !aligned(att->new_offsets, 8) ||
      !aligned(att->q, 16) || !aligned(att->out, 16) || !aligned(att->lse, 4) || !att->workspace ||
      !aligned(att->workspace, 16))
    return KVCS_EINVAL;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  AttnParams p = attn_params(cache, block_size, reqs, total_positions, att, status);
  const AttendPlan pl = plan_attend(p, *cache, *att, sms);
  if (att->workspace_bytes < attend_workspace(pl)) return KVCS_EINVAL;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  u32 *tickets = static_cast<u32 *>(att->workspace);
  const int n_tickets = static_cast<int>(attend_tickets(pl));
  p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(att->workspace) +
                                     (n_tickets * 4ll + 255) / 256 * 256);
  if (n_tickets > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kvcs_tickets_kernel, tickets, n_tickets) != cudaSuccess)
      return KVCS_ECUDA;
  }
  auto attend = att->kv_dtype == KVCS_DTYPE_BF16   ? &AttendLaunch<kKvBf16>::attend
                : att->kv_dtype == KVCS_DTYPE_FP16 ? &AttendLaunch<kKvFp16>::attend
                                                   : &AttendLaunch<kKvFp8>::attend;
  bool after_zero = true;
  if (pl.narrow) {
    p.row_lo = 1;
    p.row_hi = kNarrowRows;
    p.tickets = tickets;
    if (attend(p, false, pl.narrow_grid, after_zero, st) != cudaSuccess) return KVCS_ECUDA;
    after_zero = false;
  }
  if (pl.wide) {
    p.row_lo = pl.narrow ? kNarrowRows + 1 : 1;
    p.row_hi = 0x7fffffff;
    p.tickets = tickets + (pl.narrow ? pl.narrow_grid : 0);
    if (attend(p, true, pl.wide_grid, after_zero, st) != cudaSuccess) return KVCS_ECUDA;
  }
  if (pl.tc) {
    TcParams t;
    std::memset(&t, 0, sizeof(t));
    t.a = p;
    t.a.row_lo = pl.narrow ? kNarrowRows + 1 : 1;
    t.a.row_hi = 0x7fffffff;
    t.box = tc_box(*cache, block_size);
    t.heads_in_groups = cache->layout == KVCS_LAYOUT_HND;
    t.splits = pl.splits;
    t.most_units = pl.units;
    t.timeout_ns = kAttendTimeoutNs;
    const bool bf16 = att->kv_dtype == KVCS_DTYPE_BF16;
    CUtensorMap mk, mv;
    const bool hig = t.heads_in_groups != 0;
    if (!half_map(&mk, p.map, 0, p.kv_heads, p.head_dim, bf16, t.box, hig) ||
        !half_map(&mv, p.map, 1, p.kv_heads, p.head_dim, bf16, t.box, hig))
      return KVCS_ECUDA;
    auto run = bf16 ? &AttendLaunch<kKvBf16>::attend_tc : &AttendLaunch<kKvFp16>::attend_tc;
    if (run(t, mk, mv, pl.wide_grid, st) != cudaSuccess) return KVCS_ECUDA;
  }
  if (cudaGetLastError() != cudaSuccess) return KVCS_ECUDA;
  count_launches((n_tickets > 0 ? 1 : 0) + (pl.narrow ? 1 : 0) + (pl.wide ? 1 : 0) +
                 (pl.tc ? (pl.splits > 1 ? 2 : 1) : 0));
  return KVCS_OK;
}

int kvcs_attention_mass(const kvcs_cache *cache, int32_t block_size, const kvcs_requests *reqs,
                        int64_t total_positions, const kvcs_attention *att, float *mass,
                        uint32_t *status, void *stream) {
  int rc = check_attention(cache, block_size, att);
  if (rc != KVCS_OK) return rc;
  rc = check_tables(reqs, total_positions, status);
  if (rc != KVCS_OK) return rc;
  if (att->total_new == 0 || reqs->num_requests == 0) return KVCS_OK;
  if (!att->q || !att->lse || !att->new_offsets || !mass || !aligned(att->q, 16) ||
      !aligned(att->new_offsets, 8) || !aligned(att->lse, 4) || !aligned(mass, 4))
    return KVCS_EINVAL;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  AttnParams p = attn_params(cache, block_size, reqs, total_positions, att, status);
  p.mass = mass;
  // rows a request has observed: few go to the small kernel, more to the
  // tensor-memory one, as in the attention
  long long observed = p.tab.max_new;
  if (p.observe > 0) observed = std::min<long long>(observed, p.observe);
  const long long rows = observed * p.group;
  const bool tc = rows > kMassRows && p.group <= 128 && tc_takes(*cache, block_size, *att) &&
                  p.q_stride * 2 < (1ll << 40);
  const bool alike = p.tab.total_new == p.tab.num_requests * p.tab.max_new;
  const bool small = !tc || (!alike && p.group <= kMassRows);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (small) {
    p.row_hi = tc ? kMassRows : 0x7fffffff;
    auto run = att->kv_dtype == KVCS_DTYPE_BF16   ? &AttendLaunch<kKvBf16>::mass
               : att->kv_dtype == KVCS_DTYPE_FP16 ? &AttendLaunch<kKvFp16>::mass
                                                  : &AttendLaunch<kKvFp8>::mass;
    if (run(p, sms, st) != cudaSuccess) return KVCS_ECUDA;
  }
  if (tc) {
    MtParams t;
    std::memset(&t, 0, sizeof(t));
    t.a = p;
    t.a.row_lo = small ? kMassRows + 1 : 1;
    t.a.row_hi = 0x7fffffff;
    t.box = tc_box(*cache, block_size);
    t.heads_in_groups = cache->layout == KVCS_LAYOUT_HND;
    t.tile_tokens = 128 / p.group;
    t.timeout_ns = kAttendTimeoutNs;
    const bool bf16 = att->kv_dtype == KVCS_DTYPE_BF16;
    CUtensorMap mk, mq;
    if (!half_map(&mk, p.map, 0, p.kv_heads, p.head_dim, bf16, t.box, t.heads_in_groups != 0) ||
        !query_map(&mq, p, bf16, t.tile_tokens))
      return KVCS_ECUDA;
    auto run = bf16 ? &AttendLaunch<kKvBf16>::mass_tc : &AttendLaunch<kKvFp16>::mass_tc;
    if (run(t, mk, mq, sms, st) != cudaSuccess) return KVCS_ECUDA;
  }
  count_launches((small ? 1 : 0) + (tc ? 1 : 0));
  return KVCS_OK;
}

int kvcs_eviction_workspace(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                            int64_t num_requests, int64_t total_positions, int64_t *bytes) {
  if (!bytes || num_requests < 0 || total_positions < 0) return KVCS_EINVAL;
  int rc = check_evict_caches(caches, num_caches, block_size);
  if (rc == KVCS_OK)
    rc = check_evict_sizes(caches, num_caches, block_size, num_requests, total_positions);
  if (rc != KVCS_OK) return rc;
  *bytes = evict_workspace(caches, num_caches, block_size, num_requests, total_positions);
  return KVCS_OK;
}

int kvcs_evict(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
               const kvcs_requests *reqs, int64_t total_positions, const kvcs_eviction *ev,
               uint32_t *status, void *stream) {
  if (!ev) return KVCS_EINVAL;
  int rc = check_evict_caches(caches, num_caches, block_size);
  if (rc != KVCS_OK) return rc;
  rc = check_tables(reqs, total_positions, status);
  if (rc != KVCS_OK) return rc;
  if (ev->sinks < 0 || ev->recent < 0 || !ev->scores) return KVCS_EINVAL;
  for (int32_t i = 0; i < num_caches; ++i)
    if (!ev->scores[i] || !aligned(ev->scores[i], 4)) return KVCS_EINVAL;
  if (!aligned(ev->new_block_ids, 4) || !aligned(ev->block_sums, 8)) return KVCS_EINVAL;
  if (reqs->num_requests == 0 || total_positions == 0) return KVCS_OK;
  if (!ev->keep || !aligned(ev->keep, 8)) return KVCS_EINVAL;
  rc = check_evict_sizes(caches, num_caches, block_size, reqs->num_requests, total_positions);
  if (rc != KVCS_OK) return rc;
  if (!ev->workspace || !aligned(ev->workspace, 16) ||
      ev->workspace_bytes <
          evict_workspace(caches, num_caches, block_size, reqs->num_requests, total_positions))
    return KVCS_EINVAL;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  EvictCall p;
  std::memset(&p, 0, sizeof(p));
  p.tab.pos_offsets = reinterpret_cast<const long long *>(reqs->pos_offsets);
  p.tab.first_position = reinterpret_cast<const long long *>(reqs->first_position);
  p.tab.num_tokens = reinterpret_cast<const long long *>(reqs->num_tokens);
  p.tab.block_ids = reinterpret_cast<const int *>(reqs->block_ids);
  p.tab.num_requests = reqs->num_requests;
  p.tab.total_positions = total_positions;
  p.tab.status = status;
  p.keep = reinterpret_cast<const long long *>(ev->keep);
  p.new_block_ids = reinterpret_cast<const int *>(ev->new_block_ids);
  p.block_sums = reinterpret_cast<u64 *>(ev->block_sums);
  p.block_size = block_size;
  p.sinks = static_cast<int>(std::min<int64_t>(ev->sinks, kMaxRequestTokens));
  p.recent = static_cast<int>(std::min<int64_t>(ev->recent, kMaxRequestTokens));
  p.num_blocks = caches[0].num_blocks;
  for (int32_t i = 1; i < num_caches; ++i)
    p.num_blocks = std::min<long long>(p.num_blocks, caches[i].num_blocks);
  int launches = 0;
  p.by_block = FastDiv::of(static_cast<u32>(block_size));
  // scores in shared memory up to twice the average length; longer rows read
  // the rest again in every pass (more would leave room for fewer rows an SM)
  const int64_t tokens = total_positions * block_size;
  const int64_t average = tokens / reqs->num_requests;
  p.smem_tokens = static_cast<int>(
      std::min<int64_t>({tokens, std::max<int64_t>(2 * average, 4096), kEvictSmemTokens}));
  if (p.block_sums) {
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>(reqs->num_requests, 4ll * sms));
    kvcs_evict_zero_kernel<<<grid, 256, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KVCS_ECUDA;
    ++launches;
  }
  for (int32_t lo = 0; lo < num_caches;) {
    const EvictLaunch l = evict_launch(caches, lo, num_caches, reqs->num_requests);
    // few rows: each is split by halves and columns of at least 32 bytes.  (One
    // request, 8 rows, in place: 20,011 tokens to 4096 146 us unsplit, 102 with
    // columns of 128 bytes, 74 of 64, 68 of 32; 131,072 to 65,536 1137, 706, 628
    // from 128 on.  Four requests, 32 rows: 311, 212 of 64, 232 of 32.)
    const long long rows = l.rows * reqs->num_requests;
    int parts = 1;
    while (parts < 8 && rows * 2 * parts < sms) parts *= 2;
    p.num_caches = l.caches;
    p.rows = static_cast<int>(l.rows);
    p.list = static_cast<int *>(ev->workspace);
    const int done = l.caches <= kEvictFewCaches
                         ? launch_evict<kEvictFewCaches>(p, caches + lo, ev->scores + lo, rows, parts,
                                                         average, sms, st)
                         : launch_evict<kEvictCaches>(p, caches + lo, ev->scores + lo, rows, parts,
                                                      average, sms, st);
    if (done < 0) return done;
    launches += done;
    lo += l.caches;
  }
  count_launches(launches);
  return KVCS_OK;
}

}  // extern "C"
