// kvcs_attend_host.h -- host-side seams between the library's translation
// units: shared argument checks, device setup, the launch counter, and the
// launchers of each cache type's attention kernels.
#pragma once

#include <cuda_runtime.h>

#include "kvcs.h"
#include "kvcs_mass_tc.cuh"

namespace kvcs {

// kvcs.cu
int check_caches(const kvcs_cache *caches, int32_t num_caches, int32_t block_size);
cudaError_t device_sms(int *sms);
void count_launches(int n);

// kvcs_attend_type.cu, once per cache type
template <int kType>
struct AttendLaunch {
  // floats of workspace a launch's partial results take, and its grid
  static void shape(int dim, bool wide, int sms, int *grid, long long *part_floats);
  static cudaError_t attend(const AttnParams &p, bool wide, int grid, bool after_zero,
                            cudaStream_t st);
  // the tensor-memory kernel (16-bit caches, heads of 64 or 128), and the
  // joining of its parts
  static cudaError_t attend_tc(const TcParams &p, const CUtensorMap &k, const CUtensorMap &v,
                               int grid, cudaStream_t st);
  static cudaError_t mass(const AttnParams &p, int sms, cudaStream_t st);
  static cudaError_t mass_tc(const MtParams &p, const CUtensorMap &k, const CUtensorMap &q, int grid,
                             cudaStream_t st);
};

}  // namespace kvcs
