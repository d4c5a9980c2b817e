// api_beam.cu -- the extern "C" entry points of beam search (declared in
// include/pagedkv.h): argument validation and launches.  No entry point allocates
// memory or synchronises.
#include "pk_beam.h"

namespace {

pa_status launched(cudaError_t e) {
  if (e == cudaSuccess) return PA_OK;
  pk::record_cuda_error(e);
  return PA_ERR_CUDA;
}

constexpr int kMaxCount = INT32_MAX - 32768;
constexpr int kMaxRows = 1 << 20;  // beams of a call
constexpr int kMaxVocabulary = 1 << 28;  // (a row's bytes in 31 bits)

bool beams_ok(int B, int W) { return B >= 0 && W > 0 && (long long)B * W <= kMaxRows; }

int log2_block(int bs) { return bs == 4 ? 2 : bs == 8 ? 3 : bs == 16 ? 4 : bs == 32 ? 5 : -1; }

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace

extern "C" {

size_t pa_beam_select_workspace_size(int B, int W, int V) {
  if (B <= 0 || !beams_ok(B, W) || W > pk::kMaxBeams || V <= 0 || V > kMaxVocabulary) return 0;
  int groups, ranks;
  pk::beam_select_shape(B, W, V, &groups, &ranks);
  return groups == 1 ? 0 : (size_t)B * W * (W * 8 + 8);
}

pa_status pa_beam_select(const void* logits, pa_dtype dtype, int64_t row_stride,
                         const float* scores, int B, int W, int V, int eos_token, int pad_token,
                         int32_t* tokens, int32_t* parents, float* new_scores,
                         float* ended_scores, void* workspace, size_t workspace_bytes,
                         int32_t* status, pa_stream_t stream) {
  if (!beams_ok(B, W) || V <= 0 || V > kMaxVocabulary || eos_token < -1 || eos_token >= V ||
      row_stride < V || row_stride >= (1LL << 40))
    return PA_ERR_INVALID;
  if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32) return PA_ERR_INVALID;
  if (W > pk::kMaxBeams) return PA_ERR_UNSUPPORTED;
  if (B == 0) return PA_OK;
  if (!logits || !scores || !tokens || !parents || !new_scores || !ended_scores ||
      !aligned(logits, dtype == PA_F32 ? 4 : 2))
    return PA_ERR_INVALID;
  const size_t need = pa_beam_select_workspace_size(B, W, V);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PA_ERR_INVALID;
  }
  pk::BeamSelectArgs a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.tokens = tokens;
  a.parents = parents;
  a.new_scores = new_scores;
  a.ended = ended_scores;
  a.status = status;
  a.B = B;
  a.W = W;
  a.V = V;
  a.eos = eos_token;
  a.pad = pad_token;
  a.dtype = dtype;
  pk::beam_select_shape(B, W, V, &a.groups, &a.ranks);
  a.ws_top = static_cast<unsigned long long*>(workspace);
  a.ws_lse = reinterpret_cast<double*>(a.ws_top + (size_t)B * W * W);
  return launched(pk::launch_beam_select(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pa_beam_reorder_workspace_size(int B, int W, int max_blocks_per_seq) {
  if (B <= 0 || !beams_ok(B, W) || max_blocks_per_seq <= 0 ||
      pk::beam_reorder_in_one(B, W, max_blocks_per_seq))
    return 0;
  return ((size_t)B + 2) * 16 + (size_t)B * max_blocks_per_seq * 4;
}

pa_status pa_beam_reorder(const int32_t* parents, const int32_t* block_tables,
                          const int32_t* context_lens, const int32_t* shared_lens, int B, int W,
                          int block_size, int num_blocks, int max_blocks_per_seq,
                          int32_t* free_blocks, const int64_t* free_state, int32_t* tables_out,
                          int32_t* context_lens_out, int64_t* free_state_out,
                          int64_t* copy_pairs, void* workspace, size_t workspace_bytes,
                          int32_t* status, pa_stream_t stream) {
  if (!beams_ok(B, W) || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
      max_blocks_per_seq > kMaxCount)
    return PA_ERR_INVALID;
  const int lg = log2_block(block_size);
  if (lg < 0 || W > pk::kMaxBeams) return PA_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * block_size >= (1LL << 31) - 64) return PA_ERR_INVALID;
  if (!free_blocks || !free_state || !free_state_out) return PA_ERR_INVALID;
  if (B > 0 && (!parents || !block_tables || !context_lens || !tables_out || !context_lens_out ||
                !copy_pairs))
    return PA_ERR_INVALID;
  const size_t need = pa_beam_reorder_workspace_size(B, W, max_blocks_per_seq);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PA_ERR_INVALID;
  }
  pk::BeamReorderArgs a;
  a.parents = parents;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.shared_lens = shared_lens;
  a.ring = free_blocks;
  a.free_state = free_state;
  a.tables_out = tables_out;
  a.lens_out = context_lens_out;
  a.free_state_out = free_state_out;
  a.pairs = copy_pairs;
  a.counts = need > 0 ? static_cast<int64_t*>(workspace) : nullptr;
  a.masks = need > 0 ? reinterpret_cast<uint32_t*>(a.counts + 2 * ((size_t)B + 2)) : nullptr;
  a.status = status;
  a.B = B;
  a.W = W;
  a.M = max_blocks_per_seq;
  a.bs_log2 = lg;
  a.num_blocks = num_blocks;
  return launched(pk::launch_beam_reorder(a, reinterpret_cast<cudaStream_t>(stream)));
}

pa_status pa_beam_backtrack(const int32_t* tokens, const int32_t* parents,
                            const int32_t* lengths, const int32_t* beams, int S, int B, int W,
                            int K, int pad_token, int32_t* out, int32_t* status,
                            pa_stream_t stream) {
  if (!beams_ok(B, W) || S < 0 || K < 0 || S > kMaxCount / pk::kMaxBeams) return PA_ERR_INVALID;
  if (W > pk::kMaxBeams || K > pk::kMaxBeams) return PA_ERR_UNSUPPORTED;
  if (S == 0 || B == 0 || K == 0) return PA_OK;
  if (!tokens || !parents || !lengths || !beams || !out) return PA_ERR_INVALID;
  pk::BeamBacktrackArgs a;
  a.tokens = tokens;
  a.parents = parents;
  a.lengths = lengths;
  a.beams = beams;
  a.out = out;
  a.status = status;
  a.S = S;
  a.B = B;
  a.W = W;
  a.K = K;
  a.pad = pad_token;
  return launched(pk::launch_beam_backtrack(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
