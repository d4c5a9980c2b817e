// pk_internal.h -- declarations shared between the C-ABI layer and the kernel
// translation units (host side only).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "pagedkv.h"

namespace pk {

// Sets Kern's dynamic shared-memory limit on the current device the first
// time it is launched there.  The attribute belongs to the function as loaded
// on one device, so it is tracked per device; two threads that race on a
// device's first launch may both set it, which is harmless.
template <auto Kern>
cudaError_t ensure_dynamic_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};  // bit d: set on device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Multiprocessor count of the current device (cached per device; 0 when the
// query fails).
int sm_count();

// Makes `e` the value pa_last_cuda_error() reports on this thread.
void record_cuda_error(cudaError_t e);

struct DecodeArgs {
  const __half* q;
  const __half* k_new;  // [B, H, D] token appended at position ctx-1, or null
  const __half* v_new;
  __half* k_cache;      // pools, written only when appending
  __half* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  __half* out;
  float* ws_o;    // [B, H, num_parts, D] unnormalised partition outputs
  float* ws_ml;   // [B, H, num_parts, 2] partition (max, normaliser), log2 domain
  int32_t* status;
  int B, H, D, block_size, num_blocks, max_blocks, max_context_len;
  int part_tokens, num_parts;
  float scale_log2;  // scale * log2(e)
  // Shared-prefix decode (null otherwise): group of each sequence (-1: none),
  // and per group the tokens its members share; partitions lying entirely
  // inside the shared prefix are computed once per group by the prefix kernel.
  const int32_t* seq_group;
  const int32_t* group_prefix_len;
  const int32_t* group_offsets;  // [G+1] into group_seqs
  const int32_t* group_seqs;     // member sequence indices, the first one's table is read
  int num_groups, max_group_size, max_prefix_parts;
  // FP8 (e4m3) pools: per-(token, head) fp32 scales laid out [num_blocks, H, bs].
  bool fp8;
  const float* k_scale;
  const float* v_scale;
};

// The four tensor maps of a decode launch (scale maps used by FP8 pools only).
struct DecodeMaps {
  CUtensorMap k, v, ks, vs;
  CUtensorMap ksw, vsw;  // 64-dim halves, 128-byte swizzle (grouped calls' shared prefix)
};

// Encodes the [num_blocks * block_size, H, D] view of a cache pool as a 3-D
// TMA tensor map with a box of (D, box_heads, box_tokens).
cudaError_t make_pool_map(CUtensorMap* map, const void* base, long long rows, int H, int D,
                          int box_heads, int box_tokens);

// General 3-D tiled tensor map over fp16 data: dims innermost first, byte
// strides of dims 1 and 2, box extents; swizzle128 selects the 128-byte
// shared-memory swizzle (the inner box must then be 64 fp16 = 128 bytes).
cudaError_t make_map_3d(CUtensorMap* map, const void* base, const unsigned long long dims[3],
                        const unsigned long long strides[2], const unsigned box[3],
                        bool swizzle128,
                        CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_FLOAT16);

// 4-D and 5-D tiled tensor maps over 16-bit data (same conventions, strides of dims 1 and
// up in bytes, in any order).
cudaError_t make_map_4d(CUtensorMap* map, const void* base, const unsigned long long dims[4],
                        const unsigned long long strides[3], const unsigned box[4],
                        bool swizzle128);
cudaError_t make_map_5d(CUtensorMap* map, const void* base, const unsigned long long dims[5],
                        const unsigned long long strides[4], const unsigned box[5],
                        bool swizzle128);

// Launch the partition kernel then the combine kernel on `stream`.  When
// a.seq_group is set, the partition grid also computes the groups' shared-
// prefix partitions (multi-query, from maps.ksw / maps.vsw).
cudaError_t launch_decode(const DecodeArgs& a, const DecodeMaps& maps, cudaStream_t stream);
bool decode_supported(int D, int block_size);
// Heads per warp of the decode partition kernel (2: e4m3 pools with an even
// head count, whose K/V and scale boxes then span two adjacent heads).
int decode_heads_per_warp(bool fp8, int H);
// Tokens per TMA box of the decode partition kernel's stages (the box of the
// K/V and scale maps must match it).
int decode_box_tokens(bool fp8, int block_size, int heads_per_warp);
bool prefix_supported(int D, int block_size, int max_group_size);

cudaError_t launch_kv_cache_write(const __half* k, const __half* v, const int64_t* slots, int T,
                                  int H, int D, long long n_slots, __half* kc, __half* vc,
                                  int32_t* status, cudaStream_t stream);

cudaError_t launch_kv_cache_write_fp8(const __half* k, const __half* v, const int64_t* slots,
                                      int T, int H, int D, int block_size, long long n_slots,
                                      uint8_t* k8, uint8_t* v8, float* k_scale, float* v_scale,
                                      int32_t* status, cudaStream_t stream);

cudaError_t launch_block_copy(__half* kc, __half* vc, const int64_t* pairs, int N,
                              long long block_elems, int num_blocks, int32_t* status,
                              cudaStream_t stream);

struct PrefillArgs {
  const __half* q;
  // Tail split (set by launch_prefill): CTAs [0, full_units) are whole units
  // (one per (sequence, head, 256-query pair), in that order, units gx * H * B);
  // each later unit's key tiles are split into `split` parts whose partials
  // (D + 4 floats per query row: o[D], m, l, pad) go to ws and are merged by
  // a combine kernel.
  float* ws;
  size_t ws_floats;
  int gx, full_units, split;
  const __half* k_cache;  // the pools (set by launch_prefill; read directly by
  const __half* v_cache;  // the cp.async gather of blocks under 8 tokens)
  const int32_t* block_tables;
  const int32_t* context_lens;
  // [B] new queries per sequence (<= Lq; rows past it are written as zeros),
  // or null: Lq for every sequence
  const int32_t* q_lens;
  __half* out;
  int32_t* status;
  int B, H, Lq, D, block_size, num_blocks, max_blocks;
  float scale_log2;
};
bool prefill_supported(int D, int block_size);
// Bytes of workspace the tail split needs on the current device (0: none).
size_t prefill_workspace_bytes(int B, int H, int Lq, int D);
cudaError_t launch_prefill(const PrefillArgs& a, const void* k_cache, const void* v_cache,
                           cudaStream_t stream);

// ---- one serving step with grouped K/V heads --------------------------------

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

// Attention of packed new tokens (grouped_prompt.cu): prompts over their own
// rows (block_tables null) or chunks over the paged cache.
struct GroupedArgs {
  const int32_t* q_offsets;     // [B + 1]
  const int32_t* context_lens;  // [B], paged
  const int32_t* block_tables;  // [B, max_blocks], paged
  void* out;                    // [T, H, D]
  float* ws;                    // parts of split units, split * T * H * (D + 2) floats
  int32_t* status;
  int B, T, H, Hkv, G, D;
  int span;       // tokens of a unit (two tiles)
  unsigned long long span_magic;  // 2^40 / span, rounded up
  int g_magic;    // 2^16 / G, rounded up: r * g_magic >> 16 = r / G for r < 128
  int max_units;  // units of a K/V head, at most
  int max_tiles;  // key tiles of a unit, at most
  int split, min_part_tiles;
  int block_size, num_blocks, max_blocks, max_context;
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

// Grouped decode (grouped_decode.cu): one query token per sequence.
struct GroupedDecodeArgs {
  const void* q;  // [B, H, D]
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  float* ws_o;   // [B, H, num_parts, D] unnormalised outputs of the parts
  float* ws_ml;  // [B, H, num_parts, 2] their (max, normaliser), log2 domain
  int32_t* status;
  int B, H, Hkv, G, D, block_size, num_blocks, max_blocks, max_context;
  int part_tokens, num_parts;
  float scale_log2;
  bool bf16;
};
int grouped_decode_partition(int B, int H, int Hkv, int D, int max_context);
// Whether that many partitions merge inside the launch, without a workspace.
bool grouped_decode_in_cluster(int B, int H, int Hkv, long long parts);
cudaError_t launch_grouped_decode(const GroupedDecodeArgs& a, const void* k_cache,
                                  const void* v_cache, cudaStream_t stream);

}  // namespace pk
