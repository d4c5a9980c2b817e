// beam_tables.cu -- what follows the beams: block tables, and the way back to a
// hypothesis' tokens.
//
// Reorder.  Beam w of a request goes on from beam p = parents[w]: its new row is p's,
// its length p's.  A last block that is half full and that an earlier beam of the request
// goes on writing in is replaced by one from the ring, and the pair (old, new) is the
// copy to make (all or nothing: the blocks needed are counted before anything is
// written).  A block that beams of the request held, at a place in their rows, and that
// none holds there any more goes back to the ring.  Requests in order, in each one the
// rows' columns in order, in each one the beams: equal inputs give equal tables.
//
// A CTA brings its requests' rows to shared memory while it reads parents and lengths, so
// that a table may be its own output.  Its threads look at a column each for the blocks
// that go back, and its warps write a new row each.  What a request needs and gives back
// has to be known before, for the places in the ring: a small batch is one cluster, whose
// CTAs share out the requests and tell each other their numbers; a larger one takes a CTA
// to a request and two launches, the first to count, the second to add up the counts
// before its request and write.  Rows that do not fit shared memory are read where they
// are, and written by column, every entry of which a thread then holds.
//
// Bound: the launches, and the trips to memory (entries, then the ring).  Measured (GB300,
// in a replayed graph): 32 requests of 4 beams with 64-512 tokens 5.3 us; 256 of 8 with
// 500-8,000, tables of 4.1 MB, 10.5 us in two launches.  (Before tables went through shared
// memory the first took 13 us by one CTA of 1,024 threads.)
//
// Backtrack.  Tokens of hypothesis k: beam(n - 1) = beams[k], token(s) = tokens[s][beam(s)],
// beam(s - 1) = parents[s][beam(s)].  A walk of S steps is a chain of S loads, so a
// request's CTAs, a cluster that shares out the steps, keep parents and tokens in shared
// memory, cut the steps into pieces of 32 and walk all pieces from all W beams at once; a
// walk over the pieces' results then gives each piece's beam, and all pieces are walked
// again for their beams.  That makes three walks of 32 steps and one of S / 32 out of one
// of S.  Bound: those chains, and the trips to parents and tokens, W words a step.
// Measured: the best hypothesis of 32 requests of 4 beams over 100 steps 5.3 us; 8
// hypotheses each of 64 requests of 8 beams over 2,048 steps 10.9 us (14.4 by a CTA to a
// request, 22 with tokens fetched from memory by the walks).
#include <algorithm>

#include "pk_beam.h"
#include "pk_common.cuh"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- reorder
// The beams of a request whose entry at a column goes back: those that are no beam's
// parent, hold one there that no parent holds, and no earlier one of them.  at: the column
// in the request's first row; had: blocks of the old rows; parents: the beams that are one.
template <int WM>
__device__ __forceinline__ uint32_t given_back(const BeamReorderArgs& a, const int32_t* at,
                                               int col, const int* had, uint32_t parents) {
  const int W = a.W;
  uint32_t held = 0, drop = 0;
  int old[WM];
#pragma unroll
  for (int w = 0; w < WM; ++w) {
    old[w] = -1;
    if (w < W && col < had[w]) {
      old[w] = at[(size_t)w * a.M];
      held |= 1u << w;
    }
  }
#pragma unroll 1
  for (uint32_t left = held & ~parents; left != 0; left &= left - 1) {
    const int w = __ffs(left) - 1, id = at[(size_t)w * a.M];
    const uint32_t others = (held & parents) | (held & ((1u << w) - 1));
    bool keep = false;
#pragma unroll
    for (int u = 0; u < WM; ++u) keep |= (others >> u & 1) && old[u] == id;
    if (keep) continue;
    if (id >= 0 && id < a.num_blocks)
      drop |= 1u << w;
    else
      flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
  }
  return drop;
}

// Blocks in the ring; -1 for a state that no ring of this size can have.
__device__ __forceinline__ long long blocks_held(long long head, long long tail, int NB) {
  return head >= 0 && tail >= head && tail - head <= NB ? tail - head : -1;
}

// Exclusive sum over the block's threads and its total.
template <int kThreads>
__device__ __forceinline__ int block_scan(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_scan = [&](int y) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(kAll, y, d);
      if (lane >= d) y += z;
    }
    return y;
  };
  const int y = warp_scan(x);
  if (lane == 31) s_warp[warp] = y;
  __syncthreads();
  const int w = warp_scan(lane < kThreads / 32 ? s_warp[lane] : 0);
  __syncthreads();
  total = __shfl_sync(kAll, w, 31);
  const int before = __shfl_sync(kAll, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + y - x;
}

constexpr int kThreads = 512;
constexpr int kMaxRanks = 8;              // CTAs of a small batch
constexpr int kRounds = 2;                // columns of a thread there
constexpr int kStageBytes = 160 * 1024;   // rows that are brought to shared memory

constexpr int kScanFrom = 4096;           // requests whose counts are summed up once

enum Pass { kCluster, kCount, kWrite };

// A CTA's shared memory: its requests' rows (STAGED), then for each beam its parent, its
// old and its new blocks, its new length and the last block where it is to be copied, and
// for each request the beams that need a copy, the blocks taken before it, the beams that
// are a parent and its first column of its own (-1: a request that stays as it is).
int reorder_bytes(int nb, int W, int M, bool staged) {
  return (staged ? nb * W * M * 4 : 0) + nb * W * 20 + nb * 16;
}

template <int WM, Pass P, bool STAGED>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const BeamReorderArgs a) {
  extern __shared__ __align__(16) int s_dyn[];
  __shared__ int s_warp[kThreads / 32];
  __shared__ long long s_sum[3][kThreads / 32];
  __shared__ int2 s_rank[kMaxRanks];  // blocks that a CTA's requests take and give back
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W, M = a.M, bs = 1 << a.bs_log2;
  const int rank = blockIdx.x, ranks = gridDim.x;
  const int b0 = P == kCluster ? rank * a.B / ranks : rank;
  const int nb = P == kCluster ? (rank + 1) * a.B / ranks - b0 : 1;
  int* s_tab = s_dyn;
  int* s_parent = s_tab + (STAGED ? nb * W * M : 0);  // [nb][W]
  int* s_had = s_parent + nb * W;
  int* s_has = s_had + nb * W;
  int* s_len = s_has + nb * W;
  int* s_tail = s_len + nb * W;
  int* s_need = s_tail + nb * W;  // [nb]
  int* s_before = s_need + nb;
  int* s_used = s_before + nb;
  int* s_first = s_used + nb;
  if (P == kCluster) cluster_arrive();  // (nobody stores to a CTA that has not begun)
  pdl_wait();
  pdl_launch_dependents();
  // ---- everything from memory at once
  const int32_t* from = a.block_tables + (size_t)b0 * W * M;
  if (STAGED) {
    const int n = nb * W * M;
    const int n4 = (reinterpret_cast<uintptr_t>(from) & 15) == 0 ? n / 4 : 0;
#pragma unroll 4
    for (int i = tid; i < n4; i += kThreads)
      reinterpret_cast<int4*>(s_tab)[i] = reinterpret_cast<const int4*>(from)[i];
#pragma unroll 4
    for (int i = 4 * n4 + tid; i < n; i += kThreads) s_tab[i] = from[i];
  }
  // (By requests the second launch may replace the state while others still read it.)
  const int64_t* state = P == kWrite ? a.counts + 2 * a.B : a.free_state;
  const long long head = state[0], tail = state[1];
#pragma unroll 1
  for (int i = tid; i < nb * W; i += kThreads) {
    s_parent[i] = a.parents[b0 * W + i];
    s_had[i] = a.context_lens[b0 * W + i];  // (the length, for now)
  }
#pragma unroll 1
  for (int i = tid; i < nb; i += kThreads)
    s_first[i] = a.shared_lens != nullptr ? a.shared_lens[b0 + i] : 0;
  long long t = 0, d = 0, ta = 0, da = 0;  // kWrite: before this request and in all
  uint32_t first_mask = 0;                 // ... and of the thread's first column
  if (P == kWrite) {
    if (tid < M) first_mask = a.masks[(size_t)b0 * M + tid];
    if (a.B >= kScanFrom && tid == 0) {  // (summed up: see beam_scan_kernel)
      t = a.counts[2 * b0];
      d = a.counts[2 * b0 + 1];
      ta = a.counts[2 * a.B + 2];
      da = a.counts[2 * a.B + 3];
    }
#pragma unroll 1
    for (int b = tid; b < a.B && a.B < kScanFrom; b += kThreads) {
      const long long x = a.counts[2 * b], y = a.counts[2 * b + 1];
      ta += x;
      da += y;
      if (b < b0) {
        t += x;
        d += y;
      }
    }
  }
  __syncthreads();
  const long long held = blocks_held(head, tail, a.num_blocks);
  const int32_t* tab = STAGED ? s_tab : from;
  // ---- the requests, a warp to each, a lane to a beam
#pragma unroll 1
  for (int i = warp; i < nb; i += kThreads / 32) {
    const bool here = lane < W;
    const int p = here ? s_parent[i * W + lane] : -1, l = here ? s_had[i * W + lane] : 0;
    const int shared = s_first[i];
    const bool lost = p < -1 || p >= W;
    const bool off = l < 0 || (int)(((long long)l + bs - 1) >> a.bs_log2) > M || shared < 0;
    int flags = (lost ? PA_DEV_BAD_BEAM : 0) | (off ? PA_DEV_BAD_CONTEXT : 0);
    const bool bad = __any_sync(kAll, flags != 0);
    const int src = p >= 0 && p < W ? p : lane;
    const int l_src = __shfl_sync(kAll, l, src);
    const int len = bad ? l : p >= 0 ? l_src : 0;
    const int had = bad ? 0 : (int)(((long long)l + bs - 1) >> a.bs_log2);
    const int has = bad ? 0 : (int)(((long long)len + bs - 1) >> a.bs_log2);
    int col = -1, id = -1;  // of the last block, half full and an entry of the pool
    if (here && has > 0 && (len & (bs - 1)) != 0) {
      id = tab[((size_t)i * W + src) * M + has - 1];
      if (id >= 0 && id < a.num_blocks)
        col = has - 1;
      else
        flags |= PA_DEV_BAD_BLOCK_ID;
    }
    // An earlier beam holds it as its last block.
    const unsigned same =
        __match_any_sync(kAll, (unsigned long long)(unsigned)col << 32 | (unsigned)id);
    const uint32_t need =
        __ballot_sync(kAll, col >= 0 && (same & ((1u << lane) - 1)) != 0);
    const uint32_t used = __reduce_or_sync(kAll, here && p >= 0 && !bad ? 1u << p : 0u);
    if (here) {
      s_parent[i * W + lane] = bad ? lane : p;
      s_had[i * W + lane] = had;
      s_has[i * W + lane] = has;
      s_len[i * W + lane] = len;
      s_tail[i * W + lane] = id;
    }
    if (lane == 0) {
      s_need[i] = (int)need;
      s_used[i] = (int)used;
      s_first[i] = bad ? -1 : shared >> a.bs_log2;
    }
    if (P != kWrite && flags != 0) flag_status(a.status, flags);
  }
  __syncthreads();
  // ---- the blocks that go back, a thread to a column
  const int items = nb * M;
  auto column = [&](int i, int& q, int& col) {  // item i: a column of request q
    q = P == kCluster ? i / M : 0;
    col = i - q * M;
  };
  auto drops = [&](int i) -> uint32_t {
    if (i >= items) return 0u;
    int q, col;
    column(i, q, col);
    const int first = s_first[q];
    const uint32_t used = (uint32_t)s_used[q];
    if (first < 0 || col < first || used == (1u << (W - 1) << 1) - 1) return 0u;
    return given_back<WM>(a, tab + (size_t)q * W * M + col, col, s_had + q * W, used);
  };
  uint32_t drop[kRounds];  // (kCluster)
  int mine = 0;
  if constexpr (P == kCluster) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      drop[r] = drops(r * kThreads + tid);
      mine += __popc(drop[r]);
    }
  }
  if constexpr (P == kCount) {
#pragma unroll 1
    for (int i = tid; i < items; i += kThreads) {
      const uint32_t x = drops(i);
      a.masks[(size_t)b0 * M + i] = x;
      mine += __popc(x);
    }
  }
  // ---- what is taken and given back before this CTA's requests, and in all
  long long taken = 0, dropped = 0, all_dropped = 0;
  if constexpr (P == kCluster) {
    int total, needs = 0;
    block_scan<kThreads>(mine, s_warp, total);
    if (warp == 0) {
#pragma unroll 1
      for (int base = 0; base < nb; base += 32) {
        const int i = base + lane, x = i < nb ? __popc(s_need[i]) : 0;
        int y = x;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const int z = __shfl_up_sync(kAll, y, k);
          if (lane >= k) y += z;
        }
        if (i < nb) s_before[i] = needs + y - x;
        needs += __shfl_sync(kAll, y, 31);
      }
    }
    cluster_wait();
    if (warp == 0 && lane < ranks) store_cluster(&s_rank[rank], lane, make_int2(needs, total));
    cluster_arrive();
    cluster_wait();
    int before = 0;
#pragma unroll 1
    for (int r = 0; r < ranks; ++r) {
      const int2 x = s_rank[r];
      taken += x.x;
      all_dropped += x.y;
      if (r < rank) {
        before += x.x;
        dropped += x.y;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < nb; i += kThreads) s_before[i] += before;
    __syncthreads();
  }
  if constexpr (P == kCount) {
    int total;
    block_scan<kThreads>(mine, s_warp, total);
    if (tid == 0) {
      a.counts[2 * b0] = __popc(s_need[0]);
      a.counts[2 * b0 + 1] = total;
      if (b0 == 0) {
        a.counts[2 * a.B] = head;
        a.counts[2 * a.B + 1] = tail;
      }
    }
    return;
  }
  if constexpr (P == kWrite) {
    // Three sums at once: of the warps, then of all by every warp.
    long long x[3] = {t << 32 | ta, d, da};  // (at most 2^20 taken)
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1)
#pragma unroll
      for (int e = 0; e < 3; ++e) x[e] += __shfl_xor_sync(kAll, x[e], k);
    if (lane == 0)
#pragma unroll
      for (int e = 0; e < 3; ++e) s_sum[e][warp] = x[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 3; ++e) x[e] = s_sum[e][lane % (kThreads / 32)];
#pragma unroll
    for (int k = kThreads / 64; k >= 1; k >>= 1)
#pragma unroll
      for (int e = 0; e < 3; ++e) x[e] += __shfl_xor_sync(kAll, x[e], k);
    const long long takes = x[0];
    dropped = x[1];
    all_dropped = x[2];
    taken = takes & 0xffffffffll;
    if (tid == 0) s_before[0] = (int)(takes >> 32);
    __syncthreads();
  }
  const bool fits = taken <= held;
  // Places in the ring, less than num_blocks past these (a ring that does not fit is left).
  const unsigned NB = (unsigned)a.num_blocks;
  const unsigned head0 = fits ? (unsigned)((unsigned long long)head % NB) : 0;
  const unsigned tail0 = fits ? (unsigned)((unsigned long long)tail % NB) : 0;
  if (rank == 0 && tid == 0) {
    if (!fits) flag_status(a.status, PA_DEV_NO_BLOCKS);
    const long long room = a.num_blocks - held;
    a.free_state_out[0] = head + (fits ? taken : 0);
    a.free_state_out[1] = tail + (!fits ? 0 : all_dropped < room ? all_dropped : room);
  }
  // ---- the ring
  if (fits) {
    long long put = dropped;
#pragma unroll
    for (int r = 0; r < (P == kCluster ? kRounds : 1); ++r) {
#pragma unroll 1
      for (int base = r * kThreads; base < items; base += kThreads) {
        const int i = base + tid;
        uint32_t left = P == kCluster ? drop[r]
                        : base == 0 ? first_mask
                        : i < items ? a.masks[(size_t)b0 * M + i]
                                    : 0u;
        int total, q, col;
        long long at = put + block_scan<kThreads>(__popc(left), s_warp, total);
        put += total;
        column(i, q, col);
#pragma unroll 1
        for (; left != 0; left &= left - 1, ++at) {
          // (a ring that would hold more than there are: its state was wrong)
          if (held + at < NB) {
            unsigned to = tail0 + (unsigned)at;
            if (to >= NB) to -= NB;
            a.ring[to] = tab[((size_t)q * W + __ffs(left) - 1) * M + col];
          } else {
            flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
          }
        }
        if (P == kCluster) break;
      }
    }
  }
  // A fresh block for beam w of a request, -1 where the ring's entry is none; its pair.
  auto fresh = [&](int q, int w) {
    const uint32_t need = (uint32_t)s_need[q];
    unsigned at = head0 + (unsigned)(s_before[q] + __popc(need & ((1u << w) - 1)));
    if (at >= NB) at -= NB;
    const int id = a.ring[at];
    return id >= 0 && id < a.num_blocks ? id : -1;
  };
  // ---- rows (by warp), lengths and pairs
#pragma unroll 1
  for (int i = warp; i < nb * W; i += kThreads / 32) {
    const int q = P == kCluster ? i / W : 0, w = i - q * W;
    const size_t o = (size_t)b0 * W + i;
    const bool moves = fits && s_first[q] >= 0;
    int id = -2;  // of a last block that is new
    if (moves && ((uint32_t)s_need[q] >> w & 1)) id = fresh(q, w);
    if (lane == 0) {
      // (what was not moved keeps the length that it came with; of one that was, s_len's)
      a.lens_out[o] = moves || s_first[q] < 0 ? s_len[i] : a.context_lens[o];
      a.pairs[2 * o] = id >= 0 ? s_tail[i] : 0;
      a.pairs[2 * o + 1] = id >= 0 ? id : 0;
      if (id == -1) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
    }
    if (!STAGED || (!moves && a.tables_out == a.block_tables)) continue;
    const int has = moves ? s_has[i] : M, p = moves ? s_parent[i] : w;
    const int32_t* src = tab + (q * W + (p >= 0 ? p : 0)) * M;
    int32_t* out = a.tables_out + o * M;
#pragma unroll 4
    for (int col = lane; col < M; col += 32)
      out[col] = col < has ? (id != -2 && col == has - 1 ? id : src[col]) : -1;
  }
  // ---- rows that were not staged, a thread to a column
  if constexpr (!STAGED) {
    const bool moves = fits && s_first[0] >= 0;
    if (!moves && a.tables_out == a.block_tables) return;
    const uint32_t need = moves ? (uint32_t)s_need[0] : 0u;
#pragma unroll 1
    for (int col = tid; col < M; col += kThreads) {
      int now[WM];
#pragma unroll
      for (int w = 0; w < WM; ++w) {
        now[w] = -1;
        if (w < W && (!moves || col < s_has[w]))
          now[w] = tab[(size_t)(moves ? s_parent[w] : w) * M + col];
      }
      int32_t* out = a.tables_out + (size_t)b0 * W * M + col;
#pragma unroll
      for (int w = 0; w < WM; ++w)
        if (w < W) out[(size_t)w * M] = now[w];
#pragma unroll 1
      for (uint32_t left = need; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1;
        if (col == s_has[w] - 1) out[(size_t)w * M] = fresh(0, w);
      }
    }
  }
}

// Many requests' counts to those of the requests before each, and of all behind the state;
// neighbouring requests to a thread.  (Every CTA of the second launch adding them up took
// 69.4 us for 4,096 requests of 8 beams, this 67.5, and 4,054 and 836 us for 65,536 of one;
// for fewer the launch costs 1.5 us more than it gives.)
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamReorderArgs a) {
  __shared__ long long s_sum[2][kScanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int each = (a.B + kScanThreads - 1) / kScanThreads;
  const int b0 = min(tid * each, a.B), b1 = min(b0 + each, a.B);
  long long own[2] = {0, 0}, x[2];
#pragma unroll 4
  for (int b = b0; b < b1; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) own[e] += a.counts[2 * (size_t)b + e];
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // of the threads up to this one, then of the warps before
    x[e] = own[e];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(kAll, x[e], k);
      if (lane >= k) x[e] += y;
    }
    if (lane == 31) s_sum[e][warp] = x[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    long long y = lane < warp ? s_sum[e][lane] : 0;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) y += __shfl_xor_sync(kAll, y, k);
    x[e] += y;
    if (tid == kScanThreads - 1) a.counts[2 * (size_t)a.B + 2 + e] = x[e];
    x[e] -= own[e];
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long y = a.counts[2 * (size_t)b + e];
      a.counts[2 * (size_t)b + e] = x[e];
      x[e] += y;
    }
}

template <int WM>
cudaError_t launch_reorder_t(const BeamReorderArgs& a, cudaStream_t stream) {
  constexpr int kMost = 224 * 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.counts == nullptr) {
    constexpr auto kern = beam_reorder_kernel<WM, kCluster, true>;
    const int ranks = a.B < kMaxRanks ? std::max(a.B, 1) : kMaxRanks;
    cfg.gridDim = dim3(ranks);
    cfg.dynamicSmemBytes = reorder_bytes((a.B + ranks - 1) / ranks, a.W, a.M, true);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
    cfg.numAttrs = 2;
    const cudaError_t e = ensure_dynamic_smem<kern>(kMost);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, a);
  }
  cfg.gridDim = dim3(a.B);
  auto both = [&](auto count, auto write) {
    cudaError_t e = cudaLaunchKernelEx(&cfg, count, a);
    if (e == cudaSuccess && a.B >= kScanFrom) {
      cudaLaunchConfig_t one = cfg;
      one.gridDim = dim3(1);
      one.blockDim = dim3(kScanThreads);
      one.dynamicSmemBytes = 0;
      e = cudaLaunchKernelEx(&one, beam_scan_kernel, a);
    }
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, write, a);
  };
  const bool staged = (long long)a.W * a.M * 4 <= kStageBytes;
  cfg.dynamicSmemBytes = reorder_bytes(1, a.W, a.M, staged);
  if (!staged)
    return both(beam_reorder_kernel<WM, kCount, false>, beam_reorder_kernel<WM, kWrite, false>);
  constexpr auto count = beam_reorder_kernel<WM, kCount, true>;
  constexpr auto write = beam_reorder_kernel<WM, kWrite, true>;
  cudaError_t e = ensure_dynamic_smem<count>(kMost);
  if (e == cudaSuccess) e = ensure_dynamic_smem<write>(kMost);
  return e != cudaSuccess ? e : both(count, write);
}

// ---------------------------------------------------------------- backtrack
constexpr int kBackThreads = 1024;
constexpr int kPiece = 32;              // steps of a piece, a lane to each in the end
constexpr int kBackBytes = 160 * 1024;  // parents and beams of the steps held at a time
constexpr int kBatch = 8;               // loads of a thread in flight

// Bytes of a step's parents: one for each beam and one for "none", which W stands for and
// which is its own parent, so that a walk asks nothing.
__host__ __device__ constexpr int step_bytes(int W) { return W + 1; }

// A CTA's shared memory for `steps` steps: tokens; the hypotheses' beams, four steps to a
// word; parents; the hypotheses' beams at its pieces' last steps; and, of all the cluster's
// pieces, the beam below each from each of its last step's.
int back_bytes(int steps, int ranks, int W, int K) {
  return steps * (4 * W + step_bytes(W) + K) + steps / kPiece * (ranks * step_bytes(W) + K);
}

// Copies 4 bytes to shared memory, not awaited.
__device__ __forceinline__ void copy_word(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from)
               : "memory");
}

__global__ void __launch_bounds__(kBackThreads)
    beam_backtrack_kernel(const BeamBacktrackArgs a, int steps, int ranks) {
  extern __shared__ __align__(16) uint8_t s_back[];
  const int W = a.W, K = a.K, SW = step_bytes(W);
  const int b = blockIdx.x / ranks, rank = blockIdx.x - b * ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = steps / kPiece;
  // [K][piece of steps / 4][pieces]: neighbouring pieces in neighbouring words
  int32_t* s_token = reinterpret_cast<int32_t*>(s_back);  // [steps][W]
  uint32_t* s_beam = reinterpret_cast<uint32_t*>(s_token + steps * W);
  uint8_t* s_parent = s_back + 4 * steps * W + K * steps;  // [steps][SW]
  uint8_t* s_at = s_parent + steps * SW;                   // [K][pieces]
  uint8_t* s_map = s_at + K * pieces;                      // [ranks * pieces][SW]
  __shared__ int s_n[kMaxBeams];         // the hypotheses' lengths
  __shared__ uint8_t s_cur[kMaxBeams];   // their beam at the last step still to walk
  __shared__ uint8_t s_part[kMaxBeams];  // ... and below the piece that they begin in
  __shared__ int s_most;
  cluster_arrive();  // (nobody stores to a CTA that has not begun)
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) s_most = 0;
  __syncthreads();
  if (tid < K) {
    int n = a.lengths[b * K + tid];
    const int w = a.beams[b * K + tid];
    if (n < 0 || n > a.S || (n > 0 && (w < 0 || w >= W))) {
      flag_status(a.status, PA_DEV_BAD_BEAM);
      n = 0;
    }
    s_n[tid] = n;
    s_cur[tid] = n > 0 ? (uint8_t)w : (uint8_t)W;
    atomicMax(&s_most, n);
  }
  __syncthreads();
  const size_t plane = (size_t)a.B * W;
  int32_t* out = a.out + (size_t)b * K * a.S;
#pragma unroll 1
  for (int k = 0; k < K; ++k)  // behind all of them
#pragma unroll 1
    for (int s = s_most + rank * kBackThreads + tid; s < a.S; s += ranks * kBackThreads)
      out[(size_t)k * a.S + s] = a.pad;
  // (a thread's parents: of one beam, every `rows`-th step)
  const int rows = kBackThreads / W, my_s = tid / W, my_w = tid - my_s * W;
  // Steps lo .. hi - 1 in the cluster, base .. base + n - 1 in this CTA.
#pragma unroll 1
  for (int hi = s_most, lo; hi > 0; hi = lo) {
    lo = max(0, hi - ranks * steps);
    const int base = lo + rank * steps, n = min(max(hi - base, 0), steps);
    const int np = (n + kPiece - 1) / kPiece, p0 = rank * pieces;
    if (my_s < rows) {
      const size_t at = (size_t)(base + my_s) * plane + (size_t)b * W + my_w;
      const size_t next = rows * plane;
      const int32_t* from = a.tokens + at;
#pragma unroll 4
      for (int s = my_s; s < n; s += rows, from += next)  // (awaited at the end)
        copy_word(s_token + s * W + my_w, from);
      from = a.parents + at;
#pragma unroll 1
      for (int s = my_s; s < n; s += kBatch * rows, from += kBatch * next) {
        int p[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) p[j] = s + j * rows < n ? from[j * next] : -1;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s + j * rows < n)
            s_parent[(s + j * rows) * SW + my_w] = (uint8_t)min((unsigned)p[j], (unsigned)W);
      }
    }
#pragma unroll 1
    for (int s = tid; s < n; s += kBackThreads) s_parent[s * SW + W] = (uint8_t)W;
    __syncthreads();
    cluster_wait();  // (the other CTAs are done with their last maps)
    // ---- the beam below each piece from each of its last step's, and below the piece
    // that a hypothesis begins in from its own: told to all CTAs
#pragma unroll 1
    for (int i = tid; i < np * SW + K; i += kBackThreads) {
      uint8_t* to;
      int p, w, last;  // piece of this CTA, beam at the last of so many steps of it
      if (i < np * SW) {
        p = i / SW;
        w = i - p * SW;
        last = min(n - p * kPiece, kPiece);
        to = s_map + p0 * SW + i;
      } else {
        const int k = i - np * SW, end = min(s_n[k], hi) - base;  // its steps from base on
        if (end <= 0 || end > n) continue;
        p = (end - 1) / kPiece;
        w = s_cur[k];
        last = end - p * kPiece;
        to = s_part + k;
      }
      const uint8_t* at = s_parent + (p * kPiece + last - 1) * SW;
#pragma unroll 4
      for (int s = last; s > 0; --s, at -= SW) w = at[w];
#pragma unroll 1
      for (int r = 0; r < ranks; ++r) store_cluster_byte(to, r, w);
    }
    cluster_arrive();
    cluster_wait();
    // ---- each hypothesis over the cluster's pieces
    if (tid < K) {
      const int end = min(s_n[tid], hi) - lo;
      int w = s_cur[tid];
      if (end > 0) {
        int p = (end - 1) / kPiece;
        uint8_t* at = s_at + tid * pieces - p0;  // (of this CTA's pieces only)
        if (p >= p0 && p < p0 + pieces) at[p] = (uint8_t)w;
        w = s_part[tid];
#pragma unroll 4
        for (--p; p >= 0; --p) {
          if (p >= p0 && p < p0 + pieces) at[p] = (uint8_t)w;
          w = s_map[p * SW + w];
        }
        s_cur[tid] = (uint8_t)w;
      }
    }
    __syncthreads();
    cluster_arrive();
    // ---- all pieces of all hypotheses: their beams, W where there is no token
#pragma unroll 1
    for (int i = tid; i < K * np; i += kBackThreads) {
      const int k = i / np, p = i - k * np;
      const int end = min(s_n[k], hi) - base - p * kPiece;  // steps of it from this piece on
      int w = end > 0 ? s_at[k * pieces + p] : W;
      const uint8_t* at = s_parent + p * kPiece * SW;
      uint32_t* to = s_beam + k * (kPiece / 4) * pieces + p;
      bool off = false;
#pragma unroll 1
      for (int q = kPiece / 4 - 1; q >= 0; --q) {
        uint32_t four = 0;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const int s = 4 * q + e;
          const bool in = s < end;
          four |= (uint32_t)(in ? w : W) << (8 * e);
          const int below = in ? at[s * SW + w] : w;
          off |= below == W && w != W && base + p * kPiece + s > 0;
          w = below;
        }
        to[q * pieces] = four;
      }
      if (off) flag_status(a.status, PA_DEV_BAD_BEAM);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // ---- the tokens, a warp to a piece of a hypothesis, a lane to a step
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
      const uint32_t* fours = s_beam + (k * (kPiece / 4) + (lane >> 2)) * pieces;
      int32_t* to = out + (size_t)k * a.S + base + lane;
#pragma unroll 2
      for (int p = warp; p < np; p += kBackThreads / 32) {
        const int s = p * kPiece + lane;
        if (s >= n) continue;
        const int w = fours[p] >> (8 * (lane & 3)) & 255;
        to[p * kPiece] = w < W ? s_token[s * W + w] : a.pad;
      }
    }
    __syncthreads();
  }
  cluster_wait();
}

}  // namespace

// One cluster, or a CTA to a request and two launches (6 to 7 us): the cluster is quicker
// while a CTA has at most 32 rows of 4,096 entries in all (a batch of 32 requests of 4 beams
// 4.9 us in one and 5.9 in two, of 64 5.8 and 6.1, of 80 7.3 and 6.1; 16 of 8 beams in 256
// columns 5.8 and 6.9, 24 7.7 and 6.9).
bool beam_reorder_in_one(int B, int W, int M) {
  const long long each = (B + kMaxRanks - 1) / kMaxRanks;  // requests of a CTA
  return each * M <= kRounds * kThreads && each * W <= 32 && each * W * M <= 4096;
}

cudaError_t launch_beam_reorder(const BeamReorderArgs& a, cudaStream_t stream) {
  if (a.W <= 4) return launch_reorder_t<4>(a, stream);
  if (a.W <= 8) return launch_reorder_t<8>(a, stream);
  return launch_reorder_t<kMaxBeams>(a, stream);
}

cudaError_t launch_beam_backtrack(const BeamBacktrackArgs& a, cudaStream_t stream) {
  // CTAs of a request: as many as find an SM each, 256 steps each at least.  (An SM has
  // some 500 of its pieces of a step under way at a time, whatever their size.)
  int ranks = std::min(kMaxRanks, (a.S + 255) / 256);
  while (ranks > 1 && clusters_at_once(ranks) < a.B) --ranks;
  // Their steps: what fits shared memory.
  const int each = 4 * a.W + 2 * step_bytes(a.W) + 2 * a.K;  // (a bound: ranks <= kPiece)
  int steps = kBackBytes / each / kPiece * kPiece;
  steps = std::min(steps, ((a.S + ranks - 1) / ranks + kPiece - 1) / kPiece * kPiece);
  const cudaError_t e = ensure_dynamic_smem<beam_backtrack_kernel>(kBackBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * ranks);
  cfg.blockDim = dim3(kBackThreads);
  cfg.dynamicSmemBytes = back_bytes(steps, ranks, a.W, a.K);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, beam_backtrack_kernel, a, steps, ranks);
}

}  // namespace pk
