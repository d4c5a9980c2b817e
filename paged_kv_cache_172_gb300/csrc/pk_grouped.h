// pk_grouped.h -- declarations shared between the C-ABI layer and the kernels of a
// serving step with grouped K/V heads (host side), and the device wrappers that
// only these kernels use.
#pragma once

#include "pk_internal.h"
#ifdef __CUDACC__
#include "pk_tcgen05.cuh"
#endif

namespace pk {

// 4-D tiled tensor map over 16-bit data: dims innermost first, byte strides of
// dims 1 and up, box extents; swizzle128 as for make_map_3d.
cudaError_t make_map_4d(CUtensorMap* map, const void* base, const unsigned long long dims[4],
                        const unsigned long long strides[3], const unsigned box[4],
                        bool swizzle128);

struct StepPlanArgs {
  const int32_t* cached_lens;
  const int32_t* new_lens;
  const int32_t* free_blocks;  // ring of num_blocks ids
  const int64_t* free_state;   // [2] blocks taken and put so far
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* q_offsets;
  int64_t* slot_mapping;
  int32_t* positions;
  int64_t* free_state_out;
  int32_t* status;
  int B, T_max, bs_log2, num_blocks, max_blocks;
};
int step_plan_max_batch();
cudaError_t launch_step_plan(const StepPlanArgs& a, cudaStream_t stream);

struct RopeArgs {
  const void* q;  // [T, H, D] and [T, Hkv, D] rows, strides in elements between tokens
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const int32_t* positions;        // [n_axes, T]
  const unsigned long long* table;  // [R / 2] turns per position, axis in the low two bits
  const int64_t* slots;
  void* q_out;
  void* k_out;    // may be null
  void* k_cache;  // both null: rotation only
  void* v_cache;
  int32_t* status;
  long long n_slots;
  int T, H, Hkv, D, R, n_axes;
  bool bf16, interleaved;
};
cudaError_t launch_rope_write(const RopeArgs& a, cudaStream_t stream);

// x / n for 0 <= x < 2^31 by a product with 2^(31 + s) / n rounded up, 2^s the power
// of two from n on: the excess, x * 2^s at most, stays below 2^(31 + s) / n * n.
struct DivBy {
  unsigned m;
  int s;
};
inline DivBy div_by(int n) {
  int s = 0;
  while ((1ll << s) < n) ++s;
  return {(unsigned)(((1ull << (31 + s)) + n - 1) / n), s};
}

// Attention of packed new tokens (grouped_prompt.cu): prompts over their own
// rows (block_tables and kv_starts null), chunks over the paged cache, or queries over
// rows of another array.
struct GroupedArgs {
  const int32_t* q_offsets;     // [B + 1]
  const int32_t* context_lens;  // [B], paged and cross
  const int32_t* kv_starts;     // [B], cross: first row of a request's keys
  const int32_t* block_tables;  // [B, max_blocks], paged
  void* out;                    // [T, H, D]
  float* ws;                    // parts of split units, split * T * H * (D + 2) floats
  int32_t* status;
  int B, T, H, Hkv, G, D;
  int span;       // tokens of a unit (two tiles)
  int g_magic;    // 2^16 / G, rounded up: r * g_magic >> 16 = r / G for r < 128
  int max_units;  // units of a K/V head, at most
  int max_tiles;  // key tiles of a unit, at most
  int split;      // parts of a unit, at most
  DivBy by_span, by_split, by_hkv;
  int block_size, num_blocks, max_blocks, max_context;
  int max_q, Tk;  // cross: queries of a request, at most; rows of the keys
  float scale_log2;
  bool bf16;
};
constexpr int kGroupedMinPartTiles = 4;  // key tiles of a part, at least
constexpr int kGroupedMaxSplit = 32;     // parts of a unit, at most
int grouped_span(int G);  // tokens of a work unit; 0: unsupported
int grouped_split(int B, int T, int H, int Hkv, int max_context);
size_t grouped_workspace_bytes(int B, int T, int H, int Hkv, int D, int max_context);
cudaError_t launch_grouped(const GroupedArgs& a, const void* q, const void* k, const void* v,
                           long long q_stride, long long k_stride, long long v_stride,
                           cudaStream_t stream);

// Grouped decode (grouped_decode.cu): one query token per sequence over the paged cache,
// or few queries a request over rows of another array (kv_starts set).
struct GroupedDecodeArgs {
  const void* q;  // [B, H, D], cross: [T, H, D]
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  float* ws_o;   // [B, H, num_parts, D] unnormalised outputs of the parts (cross: T for B)
  float* ws_ml;  // [B, H, num_parts, 2] their (max, normaliser), log2 domain
  int32_t* status;
  int B, H, Hkv, G, D, block_size, num_blocks, max_blocks, max_context;
  int part_tokens, num_parts;
  // cross: requests' rows and keys; a request's max_q * G columns at most
  const int32_t* q_offsets;
  const int32_t* kv_starts;
  long long q_stride, k_stride, v_stride;
  int T, Tk, max_q;
  float scale_log2;
  bool bf16;
};
// (query, head) pairs of a request and K/V head that the kernel of single tokens serves in
// cross attention: always, and for one or two requests where its CTAs run at once.
constexpr int kCrossFew = 16, kCrossFewMost = 48;
int grouped_decode_partition(int B, int H, int Hkv, int D, int max_context);
// Whether that many partitions merge inside the launch, without a workspace.
bool grouped_decode_in_cluster(int B, int H, int Hkv, long long parts);
cudaError_t launch_grouped_decode(const GroupedDecodeArgs& a, const void* k_cache,
                                  const void* v_cache, cudaStream_t stream);

#ifdef __CUDACC__
// One lane of a converged warp, the same each time.  (elect.sync and not lane == 0:
// the compiler then knows that one thread issues the copies and products behind it
// and does not wrap each in a loop over the lanes that might.)
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// 4-D tiled TMA load (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, int c0,
                                            int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_u32(bar))
      : "memory");
}

namespace tc {
// Registers -> tensor memory, 32 lanes x 16 columns, from the first 16 registers of r.
__device__ __forceinline__ void st_32x16(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
}  // namespace tc
#endif

}  // namespace pk
