// api_grouped.cu -- the extern "C" entry points of a serving step with grouped
// K/V heads (declared in include/pagedkv.h): argument validation and launches.
// No entry point allocates memory or synchronises.
#include <math.h>

#include "pk_internal.h"

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
    double hi = inv_freq[i] * kHi;
    const double lo = fma(inv_freq[i], kHi, -hi) + inv_freq[i] * kLo;
    hi -= floor(hi);  // exact; whole turns drop out
    // 2^62 steps (the two low bits stay free), modulo one turn; |lo| is far
    // below one turn for any inv_freq below 2^50
    if (fabs(inv_freq[i]) >= 1125899906842624.0) return PA_ERR_INVALID;
    constexpr double kSteps = 4611686018427387904.0;
    const uint64_t f = ((uint64_t)(hi * kSteps) + (uint64_t)llrint(lo * kSteps)) << 2;
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
  if (T < 0 || !heads_ok(H, Hkv) || !dtype_ok(dtype) || n_axes < 1 || n_axes > 4)
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

}  // extern "C"
