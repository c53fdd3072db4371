// kvcs_attend_type.cu -- the attention and attention-mass kernels of one
// cache type (KVCS_KV_TYPE), compiled once per type.

#include <atomic>

#include "kvcs_attend_host.h"

namespace kvcs {

constexpr int kThisType = KVCS_KV_TYPE;

// Lets a kernel use `bytes` of shared memory, once per device and kernel (a
// failure is not remembered).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<u64> *done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done->load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// Everything is a template over the type: the three objects share one
// namespace.
template <int kType>
struct TypeLaunch {
  // Heads narrower than the compiled width are filled up with zeros.
  static int width_of(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

  // CTAs per SM by shared memory (228 KB an SM, 1 KB of it reserved per CTA).
  template <int kDim>
  static constexpr int ctas_per_sm() {
    return 228 * 1024 / (AttendShape<kType, kDim>::kSmemBytes + 2048) >= 2 ? 2 : 1;
  }

  template <int kDim, bool kWide>
  static cudaError_t attend(const AttnParams &p, int grid, bool after_zero, cudaStream_t st) {
    constexpr int smem = AttendShape<kType, kDim>::kSmemBytes;
    static std::atomic<u64> done{0};
    const cudaError_t e = allow_smem(kvcs_attend_kernel<kType, kDim, kWide>, smem, &done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_zero ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kvcs_attend_kernel<kType, kDim, kWide>, p);
  }

  template <int kDim, int kScores>
  static cudaError_t attend_tc(const TcParams &p, const CUtensorMap &k, const CUtensorMap &v,
                               int grid, cudaStream_t st) {
    if constexpr (kType == kKvFp8) {
      return cudaErrorNotSupported;
    } else {
      auto kernel = kvcs_attend_tc_kernel<kType == kKvBf16, kDim, kScores>;
      constexpr int smem = TcShape<kDim>::kSmemBytes;
      static std::atomic<u64> done{0};
      const cudaError_t e = allow_smem(kernel, smem, &done);
      if (e != cudaSuccess) return e;
      kernel<<<static_cast<unsigned>(grid), kTcThreads, smem, st>>>(p, k, v);
      if (p.splits == 1) return cudaGetLastError();
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(p.most_units * (kTcRows / kTcJoinRows)));
      cfg.blockDim = dim3(kTcJoinThreads);
      cfg.stream = st;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, kvcs_attend_join_kernel<kType == kKvBf16, kDim>, p);
    }
  }

  template <int kDim>
  static cudaError_t mass(const AttnParams &p, int sms, cudaStream_t st) {
    using S = MassShape<kType, kDim>;
    static std::atomic<u64> done{0};
    const cudaError_t e = allow_smem(kvcs_mass_kernel<kType, kDim>, S::kSmemBytes, &done);
    if (e != cudaSuccess) return e;
    kvcs_mass_kernel<kType, kDim>
        <<<static_cast<unsigned>(S::kCtas * sms), kMassThreads, S::kSmemBytes, st>>>(p);
    return cudaGetLastError();
  }

  template <int kDim, int kScores>
  static cudaError_t mass_tc(const MtParams &p, const CUtensorMap &k, const CUtensorMap &q, int grid,
                             cudaStream_t st) {
    if constexpr (kType == kKvFp8) {
      return cudaErrorNotSupported;
    } else {
      auto kernel = kvcs_mass_tc_kernel<kType == kKvBf16, kDim, kScores>;
      constexpr int smem = MtShape<kDim>::kSmemBytes;
      static std::atomic<u64> done{0};
      const cudaError_t e = allow_smem(kernel, smem, &done);
      if (e != cudaSuccess) return e;
      kernel<<<static_cast<unsigned>(grid), kMtThreads, smem, st>>>(p, k, q);
      return cudaGetLastError();
    }
  }
};

using This = TypeLaunch<kThisType>;

template <>
void AttendLaunch<kThisType>::shape(int dim, bool wide, int sms, int *grid, long long *part_floats) {
  const int w = This::width_of(dim);
  const int per = w == 64 ? This::ctas_per_sm<64>() : w == 128 ? This::ctas_per_sm<128>() : This::ctas_per_sm<256>();
  *grid = per * sms;
  *part_floats = static_cast<long long>(*grid) * 2 * attend_rows(wide) * (w + 2);
}

template <>
cudaError_t AttendLaunch<kThisType>::attend(const AttnParams &p, bool wide, int grid, bool after_zero,
                                        cudaStream_t st) {
  switch (This::width_of(p.head_dim)) {
    case 64:
      return wide ? This::attend<64, true>(p, grid, after_zero, st)
                  : This::attend<64, false>(p, grid, after_zero, st);
    case 128:
      return wide ? This::attend<128, true>(p, grid, after_zero, st)
                  : This::attend<128, false>(p, grid, after_zero, st);
    default:
      return wide ? This::attend<256, true>(p, grid, after_zero, st)
                  : This::attend<256, false>(p, grid, after_zero, st);
  }
}

template <>
cudaError_t AttendLaunch<kThisType>::attend_tc(const TcParams &p, const CUtensorMap &k,
                                               const CUtensorMap &v, int grid, cudaStream_t st) {
  static constexpr decltype(&This::attend_tc<64, kPlain>) run[2][3] = {
      {&This::attend_tc<64, kPlain>, &This::attend_tc<64, kCapped>, &This::attend_tc<64, kFarCapped>},
      {&This::attend_tc<128, kPlain>, &This::attend_tc<128, kCapped>, &This::attend_tc<128, kFarCapped>}};
  return run[p.a.head_dim == 128][scores_kind(p.a)](p, k, v, grid, st);
}

template <>
cudaError_t AttendLaunch<kThisType>::mass_tc(const MtParams &p, const CUtensorMap &k,
                                             const CUtensorMap &q, int grid, cudaStream_t st) {
  static constexpr decltype(&This::mass_tc<64, kPlain>) run[2][3] = {
      {&This::mass_tc<64, kPlain>, &This::mass_tc<64, kCapped>, &This::mass_tc<64, kFarCapped>},
      {&This::mass_tc<128, kPlain>, &This::mass_tc<128, kCapped>, &This::mass_tc<128, kFarCapped>}};
  return run[p.a.head_dim == 128][scores_kind(p.a)](p, k, q, grid, st);
}

template <>
cudaError_t AttendLaunch<kThisType>::mass(const AttnParams &p, int sms, cudaStream_t st) {
  switch (This::width_of(p.head_dim)) {
    case 64: return This::mass<64>(p, sms, st);
    case 128: return This::mass<128>(p, sms, st);
    default: return This::mass<256>(p, sms, st);
  }
}

}  // namespace kvcs
