// kvcs_tree.cuh -- what the new tokens of a drafted tree see of one another.
//
// Token i of a request's tree has the parent up[i] < i, or -1: it follows the
// cached text.  Its depth d_i is the number of its ancestors, its position that
// of the first new token plus d_i, and it sees itself, its ancestors, and the
// cached tokens before the tree; of the ancestors, with a window, those at most
// window - 1 steps up or at positions below the sinks.
//
// One thread follows a token's parents, in shared memory, and gathers the bits
// of a mask word in a register: an ancestor's index is below its child's, so the
// words come in falling order.  A CTA takes a request at a time.  Latency is all
// there is to it: 4 to 7 us, for one tree of 7 tokens as for 64 of 16.  The attention kernels are launched as its programmatic
// dependents and wait for it only before they read the masks.
#pragma once

#include "kvcs_attn_common.cuh"

namespace kvcs {

constexpr int kTreeThreads = 128;
constexpr int kMaxTree = 1024;   // new tokens of a request's tree, at most

struct TreeParams {
  Tables tab;
  const int *parents;   // [total_new]
  int *place;           // [total_new]: depths, or -1
  u32 *kin;             // [total_new][kin_words]
  int kin_words;
  int block_size;
  int window;
  long long sinks;
  u32 *tickets;         // zeroed on the way
  int n_tickets;
};

__global__ void __launch_bounds__(kTreeThreads) kvcs_tree_kernel(const __grid_constant__ TreeParams p) {
  __shared__ int up[kMaxTree];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0)
    for (int i = tid; i < p.n_tickets; i += kTreeThreads) p.tickets[i] = 0;
  for (long long r = blockIdx.x; r < p.tab.num_requests; r += gridDim.x) {
    const Request q = read_request(p.tab, r, p.block_size, false);
    const int n = min(q.n, kMaxTree);
    bool odd = false;
    for (int i = tid; i < n; i += kTreeThreads) {
      const int u = p.parents[q.q0 + i];
      up[i] = u;
      odd |= u < -1 || u >= i;
    }
    const bool bad = __syncthreads_or(odd);
    if (bad && tid == 0) raise(p.tab, kStatusBadRequests);
    const long long root = q.at + q.base;   // position of a token of depth 0
    for (int i = tid; i < n; i += kTreeThreads) {
      u32 *const row = p.kin + (q.q0 + i) * p.kin_words;
      int depth = 0;
      if (bad) {
        depth = -1;
      } else if (p.window > 0) {
        for (int j = up[i]; j >= 0; j = up[j]) ++depth;
      }
      p.place[q.q0 + i] = depth;
      for (int w = p.kin_words - 1; w > i >> 5; --w) row[w] = 0;
      int w = i >> 5, k = 0;
      u32 bits = 0;
      for (int j = bad ? -1 : i; j >= 0; j = up[j], ++k) {
        for (; w > j >> 5; --w) {
          row[w] = bits;
          bits = 0;
        }
        if (p.window == 0 || k < p.window || root + depth - k < p.sinks) bits |= 1u << (j & 31);
      }
      for (; w >= 0; --w) {
        row[w] = bits;
        bits = 0;
      }
    }
    __syncthreads();   // `up` is free again
  }
}

}  // namespace kvcs
