// step_plan.cu -- block tables, slots and positions of one serving step, built
// on the GPU from the sequences' lengths.
//
// With c = cached_lens[b], n = new_lens[b], bs the block size:
//   have(b) = ceil(c / bs), want(b) = ceil((c + n) / bs), need = want - have;
//   before(b) = sum of need over the sequences before b, offs(b) likewise of n;
//   block_tables[b][have + k] = ring[(head + before(b) + k) mod num_blocks];
//   token t of the packed step belongs to the sequence b with
//   offs(b) <= t < offs(b + 1), sits at position c + t - offs(b), and its slot
//   is block_tables[b][position / bs] * bs + position % bs.
// Blocks leave the ring first in, first out and in the order of the
// sequences, so equal inputs give equal tables.
//
// One launch of one CTA or of one cluster of eight.  Every CTA scans all B
// lengths itself (8 bytes a sequence) and keeps both prefix sums in shared
// memory, so no CTA waits for another before it can place its share of the
// tokens and of the fresh table entries by binary search; a token in a fresh
// block takes the id from the ring, not from the table another CTA may still
// be writing.  The ring's state is written behind a cluster barrier, as the
// lengths are, so both may be updated in place.  The work is a few hundred
// kilobytes at most: the call is bound by its launch and by two trips to memory
// (lengths, then ring entries), and one launch instead of a scan and a fill is
// what counts.
// Measured (GB300): 38 single tokens 3.4 us, 200 sequences with 11,000 new tokens
// 6.1 us, of which the launch of an empty kernel is about two thirds.
#include <cooperative_groups.h>

#include "pk_common.cuh"
#include "pk_grouped.h"

namespace pk {

namespace {

constexpr unsigned kFullMask = 0xffffffffu;

// Two running sums carried together: new tokens and fresh blocks.
struct Pair {
  long long tok, blk;
};

__device__ __forceinline__ Pair add(Pair a, Pair b) { return {a.tok + b.tok, a.blk + b.blk}; }

// Largest b with sums[b] <= x, sums being B + 1 prefix sums from 0 and
// x < sums[B]: where sequences are empty, the one that holds x.
__device__ __forceinline__ int owner(const int32_t* sums, int B, int x) {
  int lo = 0, hi = B;  // sums[lo] <= x < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const StepPlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* s_tok = plan_smem;              // [B + 1] prefix sums of the new tokens
  int32_t* s_blk = plan_smem + (a.B + 1);  // [B + 1] ... of the fresh blocks
  __shared__ Pair s_warp[kPlanThreads / 32];
  __shared__ Pair s_total;

  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << a.bs_log2;
  const long long cap = (long long)a.max_blocks << a.bs_log2;

  pdl_wait();
  pdl_launch_dependents();
  const long long head = a.free_state[0], tail = a.free_state[1];
  // A state that no ring of this size can have holds nothing.
  const long long held =
      (head >= 0 && tail >= head && tail - head <= a.num_blocks) ? tail - head : 0;

  // ---- both prefix sums, kPlanThreads sequences a round
  if (tid == 0) s_total = {0, 0};
  __syncthreads();
  for (int base = 0; base < a.B; base += kPlanThreads) {
    const int b = base + tid;
    Pair v = {0, 0};
    if (b < a.B) {
      const long long c = a.cached_lens[b], n = a.new_lens[b];
      if (c < 0 || n < 0 || c + n > cap) {
        if (rank == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
      } else {
        v.tok = n;
        v.blk = ((c + n + bs - 1) >> a.bs_log2) - ((c + bs - 1) >> a.bs_log2);
      }
    }
    Pair x = v;  // inclusive scan of the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Pair y = {__shfl_up_sync(kFullMask, x.tok, d), __shfl_up_sync(kFullMask, x.blk, d)};
      if (lane >= d) x = add(x, y);
    }
    if (lane == 31) s_warp[warp] = x;
    const Pair carried = s_total;
    __syncthreads();
    if (warp == 0) {
      Pair w = lane < kPlanThreads / 32 ? s_warp[lane] : Pair{0, 0};
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Pair y = {__shfl_up_sync(kFullMask, w.tok, d), __shfl_up_sync(kFullMask, w.blk, d)};
        if (lane >= d) w = add(w, y);
      }
      if (lane < kPlanThreads / 32) s_warp[lane] = w;
    }
    __syncthreads();
    Pair before = add(carried, {x.tok - v.tok, x.blk - v.blk});
    if (warp > 0) before = add(before, s_warp[warp - 1]);
    if (b < a.B) {  // (sums past 2^31 belong to a step that is refused below)
      s_tok[b] = (int32_t)before.tok;
      s_blk[b] = (int32_t)before.blk;
    }
    if (tid == 0) s_total = add(carried, s_warp[kPlanThreads / 32 - 1]);
    __syncthreads();
  }
  const Pair total = s_total;
  // All or nothing: a step that does not fit takes no block and plans no token.
  const bool room = total.blk <= held, fits = room && total.tok <= a.T_max;
  const int T = fits ? (int)total.tok : 0;
  const int fresh = fits ? (int)total.blk : 0;
  if (!fits && rank == 0 && tid == 0)
    flag_status(a.status, room ? PA_DEV_BAD_CONTEXT : PA_DEV_NO_BLOCKS);
  if (tid == 0) {
    s_tok[a.B] = T;
    s_blk[a.B] = fresh;
  }
  __syncthreads();

  const int first = rank * kPlanThreads + tid, step = ranks * kPlanThreads;
  // ---- per sequence
  for (int b = first; b <= a.B; b += step) a.q_offsets[b] = fits ? s_tok[b] : 0;
  const unsigned h0 = held > 0 ? (unsigned)(head % a.num_blocks) : 0;
  auto ring_id = [&](int i) {  // i-th fresh block of the step; -1 if the entry is bad
    unsigned at = h0 + (unsigned)i;  // h0, i < num_blocks, their sum below 2^32
    if (at >= (unsigned)a.num_blocks) at -= (unsigned)a.num_blocks;
    const int id = a.free_blocks[at];
    if (id >= 0 && id < a.num_blocks) return id;
    flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
    return -1;
  };
  // ---- fresh table entries
  for (int i = first; i < fresh; i += step) {
    const int b = owner(s_blk, a.B, i);
    const int have = (a.cached_lens[b] + bs - 1) >> a.bs_log2;
    a.block_tables[(size_t)b * a.max_blocks + have + (i - s_blk[b])] = ring_id(i);
  }
  // ---- tokens
  for (int t = first; t < a.T_max; t += step) {
    long long slot = -1;
    int pos = 0;
    if (t < T) {
      const int b = owner(s_tok, a.B, t);
      const int c = a.cached_lens[b];
      pos = c + (t - s_tok[b]);
      const int have = (int)(((long long)c + bs - 1) >> a.bs_log2), blk = pos >> a.bs_log2;
      int id;
      if (blk >= have) {
        id = ring_id(s_blk[b] + blk - have);
      } else {  // the cached part of a block that new tokens continue
        id = a.block_tables[(size_t)b * a.max_blocks + blk];
        if (id < 0 || id >= a.num_blocks) {
          flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
          id = -1;
        }
      }
      if (id >= 0) slot = ((long long)id << a.bs_log2) + (pos & (bs - 1));
    }
    a.slot_mapping[t] = slot;
    a.positions[t] = pos;
  }
  // Every CTA has read the ring's state and the other sequences' lengths: both may
  // be replaced, in place too (context_lens over cached_lens, an entry by the one
  // thread that still reads it).
  if (ranks > 1)
    cluster.sync();
  else
    __syncthreads();
  for (int b = first; b < a.B; b += step) {
    const long long c = a.cached_lens[b], n = a.new_lens[b];
    const bool bad = c < 0 || n < 0 || c + n > cap;
    // (In place a bad sequence keeps its length: as 0 it would be a new sequence to the
    // next step, which would fill its row with fresh blocks and flag nothing.)
    if (!bad || a.context_lens != a.cached_lens)
      a.context_lens[b] = bad ? 0 : (int32_t)(fits ? c + n : c);
  }
  if (rank == 0 && tid == 0) {
    a.free_state_out[0] = head + fresh;
    a.free_state_out[1] = tail;
  }
}

}  // namespace

int step_plan_max_batch() { return 16384; }

template <int kPlanThreads>
static cudaError_t launch_t(const StepPlanArgs& a, int ranks, cudaStream_t stream) {
  const int smem = 2 * (a.B + 1) * (int)sizeof(int32_t);
  if (smem > 40 * 1024) {
    const cudaError_t e = ensure_dynamic_smem<step_plan_kernel<kPlanThreads>>(
        2 * (step_plan_max_batch() + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, step_plan_kernel<kPlanThreads>, a);
}

// Threads and blocks of the cluster, by the sequences and the tokens to place.  Up to 256 of
// each a block of 256 threads does it in one round, and its barriers cost less than those of
// 1024 (38 sequences with a token each 3.5 us against 3.9, 200 sequences 3.8 against 4.1; 1000
// sequences would take 7.0 against 4.8).  Up to 1024 one block of 1024 is as quick as eight
// (1000 sequences 4.8 against 5.0, one chunk of 500 tokens 3.3 against 3.6), and above that
// the tokens are what takes the time and eight blocks share them (2304 tokens 4.1 us against
// 4.8, 16,512 tokens 5.8 against 16.5).
cudaError_t launch_step_plan(const StepPlanArgs& a, cudaStream_t stream) {
  const int n = a.T_max > a.B ? a.T_max : a.B;
  if (n <= 256) return launch_t<256>(a, 1, stream);
  return launch_t<1024>(a, n <= 1024 ? 1 : 8, stream);
}

}  // namespace pk
