// api_grouped.cu -- the extern "C" entry points of a serving step with grouped
// K/V heads (declared in include/pagedkv.h): argument validation and launches.
// No entry point allocates memory or synchronises.
#include <math.h>

#include "pk_grouped.h"

namespace {

pa_status launched(cudaError_t e) {
  if (e == cudaSuccess) return PA_OK;
  pk::record_cuda_error(e);
  return PA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool heads_ok(int H, int Hkv) { return H > 0 && Hkv > 0 && H <= 65535 && H % Hkv == 0; }

bool dtype_ok(int t) { return t == PA_F16 || t == PA_BF16; }

// A token's heads * D elements, `stride` elements apart, 16-byte aligned rows.
bool rows_ok(const void* p, int64_t stride, int heads, int D) {
  return p != nullptr && aligned16(p) && stride % 8 == 0 && stride >= (int64_t)heads * D &&
         stride < (1LL << 36);
}

// Tokens of a call or of a context: the kernels round them up to tiles and step
// past them by their threads in 32 bits.
constexpr int kMaxCount = INT32_MAX - 32768;

int log2_block(int bs) { return bs == 4 ? 2 : bs == 8 ? 3 : bs == 16 ? 4 : bs == 32 ? 5 : -1; }

bool pool_ok(int num_blocks, int block_size, int Hkv) {
  // (slot, head) rows, one block more than the pool has, in 32-bit coordinates
  return num_blocks > 0 && ((long long)num_blocks + 1) * block_size * Hkv < (1LL << 31);
}

}  // namespace

extern "C" {

pa_status pa_step_plan(const int32_t* cached_lens, const int32_t* new_lens, int B, int block_size,
                       int num_blocks, int max_blocks_per_seq, int T_max,
                       const int32_t* free_blocks, const int64_t* free_state,
                       int32_t* block_tables, int32_t* context_lens, int32_t* q_offsets,
                       int64_t* slot_mapping, int32_t* positions, int64_t* free_state_out,
                       int32_t* status, pa_stream_t stream) {
  if (B < 0 || T_max < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID;
  if (T_max > kMaxCount) return PA_ERR_INVALID;
  const int lg = log2_block(block_size);
  if (lg < 0 || B > pk::step_plan_max_batch()) return PA_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * block_size >= (1LL << 31) - 64) return PA_ERR_INVALID;
  if (!free_blocks || !free_state || !q_offsets || !free_state_out) return PA_ERR_INVALID;
  if (B > 0 && (!cached_lens || !new_lens || !block_tables || !context_lens))
    return PA_ERR_INVALID;
  if (T_max > 0 && (!slot_mapping || !positions)) return PA_ERR_INVALID;
  pk::StepPlanArgs a;
  a.cached_lens = cached_lens;
  a.new_lens = new_lens;
  a.free_blocks = free_blocks;
  a.free_state = free_state;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.q_offsets = q_offsets;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.free_state_out = free_state_out;
  a.status = status;
  a.B = B;
  a.T_max = T_max;
  a.bs_log2 = lg;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  return launched(pk::launch_step_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

pa_status pa_rope_table(const double* inv_freq, const int32_t* axes, int n, uint64_t* table) {
  if (n < 0 || (n > 0 && (!inv_freq || !table))) return PA_ERR_INVALID;
  for (int i = 0; i < n; ++i) {
    if (!isfinite(inv_freq[i]) || (axes && (axes[i] < 0 || axes[i] > 3))) return PA_ERR_INVALID;
    // inv_freq / 2 pi as an unevaluated sum: 1 / 2 pi in two doubles, and the
    // first product's rounding error recovered by a fused multiply-add.
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double f0 = fabs(inv_freq[i]);
    double hi = f0 * kHi;
    const double lo = fma(f0, kHi, -hi) + f0 * kLo;
    hi -= floor(hi);  // exact, as hi >= 0; whole turns drop out
    // 2^62 steps (the two low bits stay free), modulo one turn; |lo| is far
    // below one turn for any inv_freq below 2^50
    if (f0 >= 1125899906842624.0) return PA_ERR_INVALID;
    constexpr double kSteps = 4611686018427387904.0;
    uint64_t f = ((uint64_t)(hi * kSteps) + (uint64_t)llrint(lo * kSteps)) << 2;
    if (inv_freq[i] < 0.0) f = 0 - f;  // the other way round (its low bits stay zero)
    table[i] = f | (uint64_t)(axes ? axes[i] : 0);
  }
  return PA_OK;
}

pa_status pa_rope_cache_write(const void* q, const void* k, const void* v,
                              const int32_t* positions, const uint64_t* table,
                              const int64_t* slot_mapping, int T, int H, int Hkv, int D,
                              int rotary_dim, int n_axes, int interleaved, pa_dtype dtype,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              int block_size, int num_blocks, void* q_out, int64_t q_out_stride,
                              void* k_out, int64_t k_out_stride, void* k_cache, void* v_cache,
                              int32_t* status, pa_stream_t stream) {
  if (T < 0 || T > kMaxCount || !heads_ok(H, Hkv) || !dtype_ok(dtype) || n_axes < 1 ||
      n_axes > 4)
    return PA_ERR_INVALID;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  const bool cache = k_cache != nullptr || v_cache != nullptr;
  if (cache && log2_block(block_size) < 0) return PA_ERR_UNSUPPORTED;
  if (T == 0) return PA_OK;
  if (!rows_ok(q, q_stride, H, D) || !rows_ok(k, k_stride, Hkv, D) || !positions || !table ||
      !rows_ok(q_out, q_out_stride, H, D))
    return PA_ERR_INVALID;
  if (k_out != nullptr ? !rows_ok(k_out, k_out_stride, Hkv, D) : !cache) return PA_ERR_INVALID;
  if (cache && (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache) ||
                !slot_mapping || !rows_ok(v, v_stride, Hkv, D) ||
                !pool_ok(num_blocks, block_size, Hkv)))
    return PA_ERR_INVALID;
  // in place only onto itself
  if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride))
    return PA_ERR_INVALID;
  pk::RopeArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.positions = positions;
  a.table = reinterpret_cast<const unsigned long long*>(table);
  a.slots = slot_mapping;
  a.q_out = q_out;
  a.k_out = k_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.status = status;
  a.n_slots = cache ? (long long)num_blocks * block_size : 0;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.R = rotary_dim;
  a.n_axes = n_axes;
  a.bf16 = dtype == PA_BF16;
  a.interleaved = interleaved != 0;
  return launched(pk::launch_rope_write(a, reinterpret_cast<cudaStream_t>(stream)));
}

// Shared checks of the attention calls; PA_OK to go on.
static pa_status attention_args(int B, int H, int Hkv, int D, int dtype) {
  if (B < 0 || !heads_ok(H, Hkv) || !dtype_ok(dtype)) return PA_ERR_INVALID;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

static pa_status cache_args(const void* k_cache, const void* v_cache, const int32_t* block_tables,
                            const int32_t* context_lens, int Hkv, int block_size, int num_blocks,
                            int max_blocks, int max_context) {
  if (!k_cache || !v_cache || !block_tables || !context_lens || !aligned16(k_cache) ||
      !aligned16(v_cache) || !pool_ok(num_blocks, block_size, Hkv) || max_blocks <= 0 ||
      max_context < 0 || max_context > kMaxCount ||
      (long long)max_context > (long long)max_blocks * block_size)
    return PA_ERR_INVALID;
  return PA_OK;
}

static bool paged_block(int bs) { return bs == 8 || bs == 16 || bs == 32; }

// Prompts (block_tables null) and chunks.
static pa_status packed_impl(pk::GroupedArgs& a, const void* q, const void* k, const void* v,
                             int64_t qs, int64_t ks, int64_t vs, float scale, int max_keys,
                             pa_stream_t stream) {
  if (!isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID;
  a.G = a.H / a.Hkv;
  a.span = pk::grouped_span(a.G);
  if (a.span == 0) return PA_ERR_UNSUPPORTED;
  a.by_span = pk::div_by(a.span);
  a.by_split = pk::div_by(a.split);
  a.by_hkv = pk::div_by(a.Hkv);
  a.g_magic = (65536 + a.G - 1) / a.G;
  if (a.B == 0 || a.T == 0) return PA_OK;
  if (!a.q_offsets || !a.out || !aligned16(a.out) || !rows_ok(q, qs, a.H, a.D))
    return PA_ERR_INVALID;
  // A sequence whose context is bad still has its ql <= T rows in the plan.
  a.max_tiles = (int)(((long long)(max_keys > a.T ? max_keys : a.T) + 127) / 128);
  const long long units = (long long)a.T / a.span + a.B;
  if (units * a.Hkv * a.split >= (1LL << 31)) return PA_ERR_INVALID;
  a.max_units = (int)units;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  const cudaError_t e =
      pk::launch_grouped(a, q, k, v, qs, ks, vs, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaErrorInvalidValue ? PA_ERR_INVALID : launched(e);
}

pa_status pa_prompt_attention(const void* q, const void* k, const void* v,
                              const int32_t* q_offsets, int B, int T, int H, int Hkv, int D,
                              pa_dtype dtype, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, float scale, void* out, int32_t* status,
                              pa_stream_t stream) {
  const pa_status st = attention_args(B, H, Hkv, D, dtype);
  if (st != PA_OK) return st;
  if (T < 0 || T > kMaxCount) return PA_ERR_INVALID;
  if (B > 0 && T > 0 && (!rows_ok(k, k_stride, Hkv, D) || !rows_ok(v, v_stride, Hkv, D)))
    return PA_ERR_INVALID;
  pk::GroupedArgs a = {};
  a.q_offsets = q_offsets;
  a.out = out;
  a.status = status;
  a.B = B;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.split = 1;
  a.bf16 = dtype == PA_BF16;
  return packed_impl(a, q, k, v, q_stride, k_stride, v_stride, scale, T, stream);
}

size_t pa_chunk_attention_workspace_size(int B, int T, int H, int Hkv, int D,
                                         int max_context_len) {
  if (B <= 0 || T <= 0 || T > kMaxCount || !heads_ok(H, Hkv) || (D != 64 && D != 128) ||
      max_context_len <= 0 || max_context_len > kMaxCount)
    return 0;
  return pk::grouped_workspace_bytes(B, T, H, Hkv, D, max_context_len);
}

pa_status pa_chunk_attention(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* q_offsets, int B, int T, int H, int Hkv, int D,
                             pa_dtype dtype, int64_t q_stride, int block_size, int num_blocks,
                             int max_blocks_per_seq, int max_context_len, float scale, void* out,
                             void* workspace, size_t workspace_bytes, int32_t* status,
                             pa_stream_t stream) {
  pa_status st = attention_args(B, H, Hkv, D, dtype);
  if (st != PA_OK) return st;
  if (!paged_block(block_size)) return PA_ERR_UNSUPPORTED;
  if (T < 0 || T > kMaxCount) return PA_ERR_INVALID;
  pk::GroupedArgs a = {};
  a.split = 1;
  if (B > 0 && T > 0) {
    st = cache_args(k_cache, v_cache, block_tables, context_lens, Hkv, block_size, num_blocks,
                    max_blocks_per_seq, max_context_len);
    if (st != PA_OK) return st;
    if (workspace != nullptr) {
      if (!aligned16(workspace)) return PA_ERR_INVALID;
      if (workspace_bytes <
          pk::grouped_workspace_bytes(B, T, H, Hkv, D, max_context_len))
        return PA_ERR_WORKSPACE;
      a.split = pk::grouped_split(B, T, H, Hkv, max_context_len);
    }
  }
  a.q_offsets = q_offsets;
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.out = out;
  a.ws = static_cast<float*>(workspace);
  a.status = status;
  a.B = B;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_context = max_context_len;
  a.bf16 = dtype == PA_BF16;
  return packed_impl(a, q, k_cache, v_cache, q_stride, 0, 0, scale, max_context_len, stream);
}

static int decode_partition(int B, int H, int Hkv, int D, int max_context,
                            int partition_tokens) {
  if (max_context < 1) max_context = 1;  // every row is empty: one partition
  return partition_tokens > 0 ? partition_tokens
                              : pk::grouped_decode_partition(B, H, Hkv, D, max_context);
}

size_t pa_decode_grouped_workspace_size(int B, int H, int Hkv, int D, int block_size,
                                        int max_context_len, int partition_tokens) {
  if (B <= 0 || !heads_ok(H, Hkv) || (D != 64 && D != 128) || !paged_block(block_size) ||
      max_context_len <= 0 || max_context_len > kMaxCount || partition_tokens < 0)
    return 0;
  const int pt = decode_partition(B, H, Hkv, D, max_context_len, partition_tokens);
  const long long parts = ((long long)max_context_len + pt - 1) / pt;
  return pk::grouped_decode_in_cluster(B, H, Hkv, parts)
             ? 0
             : (size_t)B * H * parts * (D + 2) * sizeof(float);
}

pa_status pa_decode_grouped(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens, int B,
                            int H, int Hkv, int D, pa_dtype dtype, int block_size, int num_blocks,
                            int max_blocks_per_seq, int max_context_len, int partition_tokens,
                            float scale, void* out, void* workspace, size_t workspace_bytes,
                            int32_t* status, pa_stream_t stream) {
  pa_status st = attention_args(B, H, Hkv, D, dtype);
  if (st != PA_OK) return st;
  if (!paged_block(block_size)) return PA_ERR_UNSUPPORTED;
  if (B > 65535 || !isfinite(scale) || partition_tokens < 0 || partition_tokens % 64 != 0 ||
      partition_tokens > 2048)
    return PA_ERR_INVALID;
  if (B == 0) return PA_OK;
  st = cache_args(k_cache, v_cache, block_tables, context_lens, Hkv, block_size, num_blocks,
                  max_blocks_per_seq, max_context_len);
  if (st != PA_OK) return st;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return PA_ERR_INVALID;
  pk::GroupedDecodeArgs a = {};
  a.part_tokens = decode_partition(B, H, Hkv, D, max_context_len, partition_tokens);
  const long long parts =
      ((long long)(max_context_len > 0 ? max_context_len : 1) + a.part_tokens - 1) /
      a.part_tokens;
  if (parts > 65535) return PA_ERR_INVALID;
  a.num_parts = (int)parts;
  if (!pk::grouped_decode_in_cluster(B, H, Hkv, parts)) {
    const size_t need = (size_t)B * H * parts * (D + 2) * sizeof(float);
    if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_INVALID;
    a.ws_o = static_cast<float*>(workspace);
    a.ws_ml = a.ws_o + (size_t)B * H * parts * D;
  }
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.out = out;
  a.status = status;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.D = D;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_context = max_context_len;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.bf16 = dtype == PA_BF16;
  const cudaError_t e = pk::launch_grouped_decode(a, k_cache, v_cache,
                                                  reinterpret_cast<cudaStream_t>(stream));
  return e == cudaErrorInvalidValue ? PA_ERR_INVALID : launched(e);
}

}  // extern "C"
