// kvcs_quant.cu -- host side of the operators that write 8-bit caches and read
// cached tokens back (kvcs.h).  As in kvcs.cu, host arguments are checked before
// any CUDA call, nothing is allocated, and all work goes to the caller's stream.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "kvcs.h"
#include "kvcs_attend_host.h"
#include "kvcs_quant.cuh"

namespace kvcs {
namespace {

// Items an SM is given at least, where there is work for as many: tokens and caches
// are taken together into longer items beyond that.
constexpr long long kItems = 64;
// CTAs an SM is given at most (three are there at a time; a CTA's warps go on to
// further items).  32 against 8: a write of 32,768 tokens' 8 layers 314 and 321 us, of
// 8192 tokens' 90 and 88; reads alike (753 and 749, 104 and 103).
constexpr long long kMostCtas = 32;

bool latent(const kvcs_cache &c) { return c.layout == KVCS_LAYOUT_LATENT; }

// Checks shared by both calls; `read`: 16-bit caches too.
int check_quant(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                const kvcs_quantisation *q, bool read) {
  if (!caches || num_caches < 1 || !q) return KVCS_EINVAL;
  std::vector<kvcs_cache> plain(caches, caches + num_caches);
  for (kvcs_cache &c : plain) c.column = 0;
  const int rc = check_caches(plain.data(), num_caches, block_size);
  if (rc != KVCS_OK) return rc;
  if (q->kv_dtype < KVCS_DTYPE_BF16 || q->kv_dtype > KVCS_DTYPE_INT8) return KVCS_EINVAL;
  if (q->dtype != KVCS_DTYPE_BF16 && q->dtype != KVCS_DTYPE_FP16) return KVCS_EINVAL;
  const int es = element_bytes(q->kv_dtype);
  if (es == 2 && (!read || q->k_scales)) return KVCS_EINVAL;
  if (q->kv_dtype == KVCS_DTYPE_INT8 && !q->k_scales) return KVCS_EINVAL;
  if (!q->k_scales && q->v_scales) return KVCS_EINVAL;
  if (!std::isfinite(q->k_scale) || !std::isfinite(q->v_scale)) return KVCS_EINVAL;
  if (!read) {
    if (q->k_scales ? q->k_scale != 1.0f || q->v_scale != 1.0f
                    : !(q->k_scale > 0.0f) || !(q->v_scale > 0.0f) ||
                          !std::isfinite(1.0f / q->k_scale) || !std::isfinite(1.0f / q->v_scale))
      return KVCS_EINVAL;
  }
  if (q->key_stride < 0 || q->value_stride < 0 || q->key_stride % 8 || q->value_stride % 8)
    return KVCS_EINVAL;
  for (int32_t k = 0; k < num_caches; ++k) {
    const kvcs_cache &c = caches[k];
    if (c.layout == KVCS_LAYOUT_STATE) return KVCS_EINVAL;   // states are not per token
    if (q->k_scales) {
      if (!q->k_scales[k] || !aligned(q->k_scales[k], 4)) return KVCS_EINVAL;
      const float *v = q->v_scales ? q->v_scales[k] : nullptr;
      if (latent(c) ? v != nullptr : v == nullptr || !aligned(v, 4)) return KVCS_EINVAL;
    }
    const long long row = static_cast<long long>(c.num_heads) * (c.head_bytes / es);
    if ((q->key_stride && q->key_stride < row) || (!latent(c) && q->value_stride && q->value_stride < row))
      return KVCS_EINVAL;
    if (c.head_bytes % (8 * es) || c.head_bytes / es > kQuantMaxDim) return KVCS_EUNSUPPORTED;
    if (static_cast<double>(block_size) * c.num_heads * c.head_bytes >= 2147483648.0 ||
        row * es >= (1ll << 30))
      return KVCS_EUNSUPPORTED;
  }
  return KVCS_OK;
}

// Pointers of every cache's keys and values.
int check_rows(const kvcs_cache *caches, int32_t num_caches, const void *const *keys,
               const void *const *values) {
  if (!keys) return KVCS_EINVAL;
  for (int32_t k = 0; k < num_caches; ++k) {
    const void *v = values ? values[k] : nullptr;
    if (!keys[k] || !aligned(keys[k], 16) || !aligned(v, 16)) return KVCS_EINVAL;
    if (latent(caches[k]) ? v != nullptr : v == nullptr) return KVCS_EINVAL;
  }
  return KVCS_OK;
}

QuantCache quant_cache(const kvcs_cache &c, int block_size, const kvcs_quantisation &q, int32_t k,
                       const void *key, const void *value) {
  QuantCache d;
  std::memset(&d, 0, sizeof(d));
  d.map = page_map(c, block_size);
  d.key = static_cast<const unsigned char *>(key);
  d.value = static_cast<const unsigned char *>(value);
  if (q.k_scales) {
    d.k_scales = q.k_scales[k];
    d.v_scales = q.v_scales ? q.v_scales[k] : nullptr;
  }
  d.heads = c.num_heads;
  d.dim = c.head_bytes / element_bytes(q.kv_dtype);
  const long long row = static_cast<long long>(d.heads) * d.dim;
  d.key_stride = q.key_stride ? q.key_stride : row;
  d.value_stride = q.value_stride ? q.value_stride : row;
  d.m0 = 2ull * (static_cast<u64>(c.layer) * KVCS_MAX_KV_HEADS_PER_LAYER + c.head_offset) + 1;
  return d;
}

unsigned warp_grid(long long items, int sms) {
  const long long per = kQuantThreads / 32;
  return static_cast<unsigned>(std::max(1ll, std::min((items + per - 1) / per, kMostCtas * sms)));
}

// How a row's pieces go to lanes: 4 or 8 lanes of one piece (heads of up to 64
// and 128 elements; 16-bit caches' pieces are half as long, 8 or 16 lanes), or a
// warp of several.
template <int kCaches>
using WriteKernel = void (*)(QuantWriteParams<kCaches>);
template <int kShift, int kPer, int kCaches>
WriteKernel<kCaches> write_kernel_of(bool int8, bool bf16) {
  return int8 ? (bf16 ? kvcs_write_quantised_kernel<true, true, kShift, kPer, kCaches>
                      : kvcs_write_quantised_kernel<true, false, kShift, kPer, kCaches>)
              : (bf16 ? kvcs_write_quantised_kernel<false, true, kShift, kPer, kCaches>
                      : kvcs_write_quantised_kernel<false, false, kShift, kPer, kCaches>);
}
template <int kCaches>
WriteKernel<kCaches> write_kernel(int dim, bool int8, bool bf16) {
  return dim <= 64    ? write_kernel_of<2, 1, kCaches>(int8, bf16)
         : dim <= 128 ? write_kernel_of<3, 1, kCaches>(int8, bf16)
                      : write_kernel_of<5, 4, kCaches>(int8, bf16);
}

template <int kCaches>
using ReadKernel = void (*)(QuantReadParams<kCaches>);
template <int kCaches>
ReadKernel<kCaches> read_kernel(int dim, int kv_dtype) {
  switch (kv_dtype) {
    case KVCS_DTYPE_INT8:
      return dim <= 64    ? kvcs_read_kernel<KVCS_DTYPE_INT8, 2, 1, kCaches>
             : dim <= 128 ? kvcs_read_kernel<KVCS_DTYPE_INT8, 3, 1, kCaches>
                          : kvcs_read_kernel<KVCS_DTYPE_INT8, 5, 4, kCaches>;
    case KVCS_DTYPE_FP8_E4M3:
      return dim <= 64    ? kvcs_read_kernel<KVCS_DTYPE_FP8_E4M3, 2, 1, kCaches>
             : dim <= 128 ? kvcs_read_kernel<KVCS_DTYPE_FP8_E4M3, 3, 1, kCaches>
                          : kvcs_read_kernel<KVCS_DTYPE_FP8_E4M3, 5, 4, kCaches>;
    default:
      return dim <= 64    ? kvcs_read_kernel<KVCS_DTYPE_BF16, 3, 1, kCaches>
             : dim <= 128 ? kvcs_read_kernel<KVCS_DTYPE_BF16, 4, 1, kCaches>
                          : kvcs_read_kernel<KVCS_DTYPE_BF16, 5, 8, kCaches>;
  }
}

// One launch over caches [lo, lo + n) of a call.
template <int kCaches>
cudaError_t launch_write(const QuantWriteCall &call, const kvcs_cache *caches, int32_t lo, int n,
                         const void *const *keys, const void *const *values,
                         const kvcs_quantisation &q, int dim, int sms, cudaStream_t st) {
  QuantWriteParams<kCaches> w;
  static_cast<QuantWriteCall &>(w) = call;
  w.num_caches = n;
  for (int k = 0; k < n; ++k)
    w.c[k] = quant_cache(caches[lo + k], w.block_size, q, lo + k, keys[lo + k],
                         values ? values[lo + k] : nullptr);
  const long long runs = std::min<long long>(
      n, std::max<long long>(1, (kItems * sms + w.num_tokens - 1) / w.num_tokens));
  w.caches_per_item = static_cast<int>((n + runs - 1) / runs);
  const long long items = w.num_tokens * ((n + w.caches_per_item - 1) / w.caches_per_item);
  return launch_early(write_kernel<kCaches>(dim, q.kv_dtype == KVCS_DTYPE_INT8, q.dtype == KVCS_DTYPE_BF16),
                      warp_grid(items, sms), kQuantThreads, st, w);
}

template <int kCaches>
cudaError_t launch_read(const QuantReadCall &call, const kvcs_cache *caches, int32_t lo, int n,
                        void *const *keys, void *const *values, const kvcs_quantisation &q, int dim,
                        int sms, cudaStream_t st) {
  QuantReadParams<kCaches> p;
  static_cast<QuantReadCall &>(p) = call;
  p.num_caches = n;
  for (int k = 0; k < n; ++k)
    p.c[k] = quant_cache(caches[lo + k], p.block_size, q, lo + k, keys[lo + k],
                         values ? values[lo + k] : nullptr);
  // tokens together, then caches together, as long as there are items enough
  const long long total = p.tab.total_new, want = kItems * sms;
  p.tokens_per_item = static_cast<int>(std::max(1ll, std::min(8ll, total * n / want)));
  const long long groups = (total + p.tokens_per_item - 1) / p.tokens_per_item;
  const long long runs = std::min<long long>(n, std::max(1ll, (want + groups - 1) / groups));
  p.caches_per_item = static_cast<int>((n + runs - 1) / runs);
  const long long items = groups * ((n + p.caches_per_item - 1) / p.caches_per_item);
  return launch_early(read_kernel<kCaches>(dim, q.kv_dtype), warp_grid(items, sms), kQuantThreads, st, p);
}

int largest_dim(const kvcs_cache *caches, int32_t num_caches, const kvcs_quantisation &q) {
  int dim = 0;
  for (int32_t k = 0; k < num_caches; ++k) dim = std::max(dim, caches[k].head_bytes / element_bytes(q.kv_dtype));
  return dim;
}

}  // namespace
}  // namespace kvcs

using namespace kvcs;

extern "C" {

int kvcs_write_kv_quantised(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                            int64_t num_tokens, const void *const *keys, const void *const *values,
                            const int64_t *slot_mapping, const int64_t *positions,
                            const kvcs_quantisation *quant, uint64_t *block_sums, uint32_t *status,
                            void *stream) {
  if (num_tokens < 0) return KVCS_EINVAL;
  int rc = check_quant(caches, num_caches, block_size, quant, false);
  if (rc != KVCS_OK) return rc;
  if (!aligned(block_sums, 8) || !aligned(status, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 8))
    return KVCS_EINVAL;
  if (num_tokens == 0) return KVCS_OK;
  if (!slot_mapping || !positions) return KVCS_EINVAL;
  rc = check_rows(caches, num_caches, keys, values);
  if (rc != KVCS_OK) return rc;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  QuantWriteCall w;
  std::memset(&w, 0, sizeof(w));
  w.slots = reinterpret_cast<const long long *>(slot_mapping);
  w.positions = reinterpret_cast<const long long *>(positions);
  w.block_sums = reinterpret_cast<u64 *>(block_sums);
  w.status = status;
  w.num_tokens = num_tokens;
  w.num_blocks = caches[0].num_blocks;
  w.block_size = block_size;
  w.k_inv = 1.0f / quant->k_scale;
  w.v_inv = 1.0f / quant->v_scale;
  for (int32_t k = 0; k < num_caches; ++k) {
    w.num_blocks = std::min<long long>(w.num_blocks, caches[k].num_blocks);
    w.store8 |= needs_8(caches[k]) ? 1 : 0;
  }
  const int dim = largest_dim(caches, num_caches, *quant);
  for (int32_t lo = 0; lo < num_caches; lo += kQuantCaches) {
    const int n = std::min(kQuantCaches, num_caches - lo);
    auto launch = n <= kQuantFewCaches ? launch_write<kQuantFewCaches> : launch_write<kQuantCaches>;
    if (launch(w, caches, lo, n, keys, values, *quant, dim, sms, st) != cudaSuccess) return KVCS_ECUDA;
    count_launches(1);
  }
  return KVCS_OK;
}

int kvcs_read_kv(const kvcs_cache *caches, int32_t num_caches, int32_t block_size,
                 const kvcs_requests *reqs, int64_t total_positions, const int64_t *token_offsets,
                 int64_t total_tokens, void *const *keys, void *const *values,
                 const kvcs_quantisation *quant, uint32_t *status, void *stream) {
  if (total_tokens < 0) return KVCS_EINVAL;
  int rc = check_quant(caches, num_caches, block_size, quant, true);
  if (rc != KVCS_OK) return rc;
  rc = check_tables(reqs, total_positions, status);
  if (rc != KVCS_OK) return rc;
  if (!aligned(token_offsets, 8)) return KVCS_EINVAL;
  if (total_tokens >= (1ll << 31)) return KVCS_EUNSUPPORTED;
  if (total_tokens == 0 || reqs->num_requests == 0) return KVCS_OK;
  if (!token_offsets) return KVCS_EINVAL;
  rc = check_rows(caches, num_caches, keys, values);
  if (rc != KVCS_OK) return rc;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return KVCS_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  QuantReadCall p;
  std::memset(&p, 0, sizeof(p));
  p.tab.pos_offsets = reinterpret_cast<const long long *>(reqs->pos_offsets);
  p.tab.first_position = reinterpret_cast<const long long *>(reqs->first_position);
  p.tab.num_tokens = reinterpret_cast<const long long *>(reqs->num_tokens);
  p.tab.block_ids = reinterpret_cast<const int *>(reqs->block_ids);
  p.tab.new_offsets = reinterpret_cast<const long long *>(token_offsets);
  p.tab.num_requests = reqs->num_requests;
  p.tab.total_positions = total_positions;
  p.tab.total_new = total_tokens;
  p.tab.max_new = total_tokens;
  p.tab.status = status;
  p.block_size = block_size;
  p.by_block = FastDiv::of(static_cast<u32>(block_size));
  p.stored_bf16 = quant->kv_dtype == KVCS_DTYPE_BF16;
  p.out_bf16 = quant->dtype == KVCS_DTYPE_BF16;
  p.k_scale = quant->k_scale;
  p.v_scale = quant->v_scale;
  for (int32_t k = 0; k < num_caches; ++k) p.load8 |= needs_8(caches[k]) ? 1 : 0;
  const int dim = largest_dim(caches, num_caches, *quant);
  for (int32_t lo = 0; lo < num_caches; lo += kQuantCaches) {
    const int n = std::min(kQuantCaches, num_caches - lo);
    auto launch = n <= kQuantFewCaches ? launch_read<kQuantFewCaches> : launch_read<kQuantCaches>;
    if (launch(p, caches, lo, n, keys, values, *quant, dim, sms, st) != cudaSuccess) return KVCS_ECUDA;
    count_launches(1);
  }
  return KVCS_OK;
}

}  // extern "C"
