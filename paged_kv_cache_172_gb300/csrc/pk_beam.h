// pk_beam.h -- declarations shared between the C-ABI layer and the kernels of beam
// search (host side), and the device wrappers that only these kernels use.
#pragma once

#include "pk_internal.h"
#ifdef __CUDACC__
#include <string.h>

#include "pk_common.cuh"
#endif

namespace pk {

constexpr int kMaxBeams = 32;

// Beam selection (beam_select.cu).
struct BeamSelectArgs {
  const void* logits;  // rows of V, row_stride elements apart
  long long row_stride;
  const float* scores;  // [B, W]
  int32_t* tokens;      // [B, W] the chosen continuations, best first
  int32_t* parents;
  float* new_scores;
  float* ended;  // [B, W] by beam
  int32_t* status;
  int B, W, V, eos, pad, dtype;
  int ranks, groups;  // CTAs of a cluster, clusters of a request
  // With groups > 1, per beam: its best keys and the logarithm of its sum.
  unsigned long long* ws_top;  // [B * W][W]
  double* ws_lse;              // [B * W]
};
// How many clusters of `ranks` CTAs the current device holds at once, an SM to each CTA (its
// processing clusters have SMs left over); kept per device.
int clusters_at_once(int ranks);
void beam_select_shape(int B, int W, int V, int* groups, int* ranks);
cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t stream);

// Block tables that follow the beams (beam_tables.cu).
struct BeamReorderArgs {
  const int32_t* parents;       // [B, W]
  const int32_t* block_tables;  // [B * W, M]
  const int32_t* context_lens;  // [B * W]
  const int32_t* shared_lens;   // [B] or null
  int32_t* ring;                // [num_blocks]
  const int64_t* free_state;    // [2]
  int32_t* tables_out;
  int32_t* lens_out;
  int64_t* free_state_out;
  int64_t* pairs;   // [B * W, 2]
  // Workspace of the launches by requests, or null: [B + 1, 2] blocks that each request
  // takes and gives back, then the ring's state; [B, M] beams whose entry goes back.
  int64_t* counts;
  uint32_t* masks;
  int32_t* status;
  int B, W, M, bs_log2, num_blocks;
};
bool beam_reorder_in_one(int B, int W, int M);
cudaError_t launch_beam_reorder(const BeamReorderArgs& a, cudaStream_t stream);

struct BeamBacktrackArgs {
  const int32_t* tokens;   // [S, B, W]
  const int32_t* parents;  // [S, B, W]
  const int32_t* lengths;  // [B, K]
  const int32_t* beams;    // [B, K]
  int32_t* out;            // [B, K, S]
  int32_t* status;
  int S, B, W, K, pad;
};
cudaError_t launch_beam_backtrack(const BeamBacktrackArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
// The cluster's barrier in two halves, for all threads of all CTAs: what was written to
// shared memory before the first is seen behind the second.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores 8 bytes to what p is in the shared memory of the cluster's CTA `rank`.
template <typename X>
__device__ __forceinline__ void store_cluster(X* p, int rank, X x) {
  static_assert(sizeof(X) == 8, "one store");
  uint32_t at;
  unsigned long long y;
  memcpy(&y, &x, 8);
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(y) : "memory");
}
__device__ __forceinline__ void store_cluster_byte(uint8_t* p, int rank, int x) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
#endif

}  // namespace pk
