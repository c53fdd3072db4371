// kvcs_attend_host.h -- host-side seams between the library's translation
// units: shared argument checks, device setup, the launch counter, and the
// launchers of each cache type's attention kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kvcs.h"
#include "kvcs_attend_cols.cuh"
#include "kvcs_mass_tc.cuh"

namespace kvcs {

// kvcs.cu
int check_caches(const kvcs_cache *caches, int32_t num_caches, int32_t block_size);
cudaError_t device_sms(int *sms);
void count_launches(int n);

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int element_bytes(int kv_dtype) {
  return kv_dtype == KVCS_DTYPE_FP8_E4M3 || kv_dtype == KVCS_DTYPE_INT8 ? 1 : 2;
}

// kvcs_attend.cu
PageMap page_map(const kvcs_cache &c, int block_size);
bool needs_8(const kvcs_cache &c);
int check_tables(const kvcs_requests *reqs, int64_t total_positions, const uint32_t *status);

// A launch that may begin while the kernel before it ends.
template <typename Params>
cudaError_t launch_early(void (*kernel)(Params), unsigned grid, unsigned threads, cudaStream_t st,
                         const Params &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// kvcs_attend_type.cu, once per cache type; kExt: for extended views (no mass)
template <int kType, bool kExt>
struct AttendLaunch {
  // floats of workspace a launch's partial results take, and its grid; kind:
  // narrow (0) or wide (1), in extended views the row tile's products (1, 2, 4)
  static void shape(int dim, int kind, int sms, int *grid, long long *part_floats);
  static cudaError_t attend(const AttnParams &p, int kind, int grid, bool after_zero,
                            cudaStream_t st);
  // the tensor-memory kernel (heads of 64 or 128; 16-bit caches, in extended views
  // 8-bit ones of bf16 queries as well, without the maps), and the joining of its parts
  static cudaError_t attend_tc(const TcParams &p, const CUtensorMap &k, const CUtensorMap &v,
                               int grid, bool early, cudaStream_t st);
  static cudaError_t mass(const AttnParams &p, int sms, cudaStream_t st);
  static cudaError_t mass_tc(const MtParams &p, const CUtensorMap &k, const CUtensorMap &q, int grid,
                             cudaStream_t st);
};

}  // namespace kvcs
