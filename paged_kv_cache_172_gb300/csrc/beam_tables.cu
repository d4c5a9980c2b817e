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
// Every thread takes a column of a request, reads its W entries and writes the new ones,
// so that a table may be its own output; what a request needs and gives back has to be
// known before, for the places in the ring.  Few entries: one CTA takes all requests and
// its scan over the columns carries the places along.  Many: one CTA to a request counts,
// a second launch adds up the counts before its request and writes.
//
// Bound: the launches and the trips parents, lengths, last blocks, entries.
//
// Backtrack.  Tokens of hypothesis k: beam(n - 1) = beams[k], token(s) = tokens[s][beam(s)],
// beam(s - 1) = parents[s][beam(s)].  A walk of S steps is a chain of S loads, so each
// request's CTA keeps its parents in shared memory, cuts the steps into pieces of 32 and
// walks all pieces from all W beams at once; a walk over the pieces' results then gives
// each piece's beam, and all pieces are walked again for their beams.  That makes three
// walks of 32 steps and one of S / 32 out of one of S.
#include <algorithm>

#include "pk_beam.h"
#include "pk_common.cuh"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- reorder
// What a warp finds out about a request, a lane to a beam.
struct Request {
  int p;         // parent of the lane's beam, -1: none
  int had, has;  // blocks of the old and of the new row
  int len;       // new length
  int tail;      // column of the last block, half full and an entry of the pool; -1: none
  int tail_id;
  uint32_t need;  // beams that get a copy of their last block
  bool bad;       // left as it is
  int flags;      // what is wrong with it, for the status
};

__device__ __forceinline__ Request look_at(const BeamReorderArgs& a, int b) {
  const int lane = threadIdx.x & 31, W = a.W, bs = 1 << a.bs_log2;
  Request r;
  const bool here = lane < W;
  r.p = here ? a.parents[b * W + lane] : -1;
  const int old_len = here ? a.context_lens[b * W + lane] : 0;
  const int shared = a.shared_lens != nullptr ? a.shared_lens[b] : 0;
  const bool lost = here && (r.p < -1 || r.p >= W);
  const bool off = here && (old_len < 0 || ((long long)old_len + bs - 1) >> a.bs_log2 > a.M);
  r.flags = (lost ? PA_DEV_BAD_BEAM : 0) | (off || shared < 0 ? PA_DEV_BAD_CONTEXT : 0);
  r.bad = __any_sync(kAll, r.flags != 0);
  const int src = r.p >= 0 && r.p < W ? r.p : lane;
  const int l = __shfl_sync(kAll, old_len, src);
  r.len = r.p >= 0 ? l : 0;
  r.had = r.bad ? 0 : (int)(((long long)old_len + bs - 1) >> a.bs_log2);
  r.has = r.bad ? 0 : (int)(((long long)r.len + bs - 1) >> a.bs_log2);
  r.tail = -1;
  r.tail_id = -1;
  if (!r.bad && here && r.has > 0 && (r.len & (bs - 1)) != 0) {
    r.tail_id = a.block_tables[((size_t)b * W + src) * a.M + r.has - 1];
    if (r.tail_id >= 0 && r.tail_id < a.num_blocks)
      r.tail = r.has - 1;
    else
      r.flags |= PA_DEV_BAD_BLOCK_ID;
  }
  bool again = false;  // an earlier beam holds it as its last block
#pragma unroll 1
  for (int u = 0; u < W; ++u) {
    const int t = __shfl_sync(kAll, r.tail, u), id = __shfl_sync(kAll, r.tail_id, u);
    again |= u < lane && t >= 0 && t == r.tail && id == r.tail_id;
  }
  r.need = __ballot_sync(kAll, again);
  return r;
}

// A request as the columns' threads see it.
struct Rows {
  int b, first;  // first: the first column whose blocks are the request's own
  uint32_t need;
  int before;  // blocks that requests before it take
  bool bad;
};

template <int WM>
struct Column {
  int old[WM];          // entries; meaningful for beams that hold one
  uint32_t held, used;  // beams that hold an entry here; of those, the parents of one
  uint32_t drop;        // beams whose entry goes back

  // had: blocks of the old rows
  __device__ __forceinline__ void read(const BeamReorderArgs& a, const Rows& r, int col,
                                       const int* had, const int* parent) {
    const int W = a.W;
    held = used = drop = 0;
    const int32_t* at = a.block_tables + (size_t)r.b * W * a.M + col;
#pragma unroll
    for (int w = 0; w < WM; ++w) {
      old[w] = -1;
      if (w < W && col < had[w]) {
        old[w] = at[(size_t)w * a.M];
        held |= 1u << w;
      }
    }
    if (held == 0) return;
#pragma unroll 1
    for (int w = 0; w < W; ++w)
      if (parent[w] >= 0) used |= 1u << parent[w];
    used &= held;
    if (col < r.first || used == held) return;
#pragma unroll 1
    for (uint32_t left = held & ~used; left != 0; left &= left - 1) {
      const int w = __ffs(left) - 1, id = at[(size_t)w * a.M];
      // held by a parent, or given back by an earlier beam
      const uint32_t others = used | (held & ((1u << w) - 1));
      bool keep = false;
#pragma unroll
      for (int u = 0; u < WM; ++u) keep |= (others >> u & 1) && old[u] == id;
      if (keep) continue;
      if (id >= 0 && id < a.num_blocks)
        drop |= 1u << w;
      else
        flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
    }
  }
};

constexpr int kMaxInOne = 1024;  // requests of the launch by one CTA

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

enum Pass { kInOne, kCount, kWrite };

template <int WM, Pass P, int kThreads>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const BeamReorderArgs a) {
  // parents and blocks of a CTA's requests: one, or all of them
  extern __shared__ int s_rows[];
  __shared__ int s_warp[kThreads / 32];
  __shared__ long long s_sum[kThreads / 32];
  __shared__ uint32_t s_bits[P == kInOne ? kMaxInOne : 1];  // need
  __shared__ int s_before[P == kInOne ? kMaxInOne : 1];
  __shared__ uint8_t s_bad[P == kInOne ? kMaxInOne : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W;
  const int b0 = P == kInOne ? 0 : blockIdx.x, nb = P == kInOne ? a.B : 1;
  int* s_parent = s_rows;        // [nb][W]
  int* s_had = s_rows + nb * W;  // [nb][W]
  int* s_has = s_had + nb * W;   // [nb][W]
  int* s_tail = s_has + nb * W;  // [nb][W] id of a last block to copy
  pdl_wait();
  pdl_launch_dependents();
  // (By requests the second launch may replace the state while others still read it.)
  const int64_t* state = P == kWrite ? a.counts + 2 * a.B : a.free_state;
  const long long head = state[0], tail = state[1];
  const long long held = blocks_held(head, tail, a.num_blocks);
  // ---- the requests: parents, lengths, last blocks
#pragma unroll 1
  for (int i = warp; i < nb; i += kThreads / 32) {
    const Request r = look_at(a, b0 + i);
    if (lane < W) {
      s_parent[i * W + lane] = r.bad ? lane : r.p;
      s_had[i * W + lane] = r.had;
      s_has[i * W + lane] = r.has;
      s_tail[i * W + lane] = r.tail_id;
    }
    if (lane == 0) {
      s_bits[i] = r.need;
      s_bad[i] = r.bad;
    }
    if (P != kWrite && r.flags != 0) flag_status(a.status, r.flags);
  }
  __syncthreads();
  // ---- blocks to take: before each request, and in all
  long long taken = 0, dropped = 0;  // dropped: those of requests before (kWrite)
  if constexpr (P == kInOne) {
    int done = 0;
#pragma unroll 1
    for (int base = 0; base < nb; base += kThreads) {
      const int i = base + tid;
      int total;
      const int x = i < nb ? __popc(s_bits[i]) : 0;
      const int at = block_scan<kThreads>(x, s_warp, total);
      if (i < nb) s_before[i] = done + at;
      done += total;
    }
    taken = done;
    __syncthreads();
  }
  long long before = 0, all_dropped = 0;
  if constexpr (P == kWrite) {
    long long t = 0, d = 0, ta = 0, da = 0;
#pragma unroll 1
    for (int b = tid; b < a.B; b += kThreads) {
      const long long x = a.counts[2 * b], y = a.counts[2 * b + 1];
      ta += x;
      da += y;
      if (b < b0) {
        t += x;
        d += y;
      }
    }
    auto sum = [&](long long x) {
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) x += __shfl_xor_sync(kAll, x, k);
      if (lane == 0) s_sum[warp] = x;
      __syncthreads();
      long long y = 0;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) y += s_sum[w];
      __syncthreads();
      return y;
    };
    before = sum(t);
    dropped = sum(d);
    taken = sum(ta);
    all_dropped = sum(da);
  }
  const bool fits = P == kCount || taken <= held;
  // Places in the ring, less than num_blocks past these (a ring that does not fit is left).
  const unsigned NB = (unsigned)a.num_blocks;
  const unsigned head0 = fits && held >= 0 ? (unsigned)((unsigned long long)head % NB) : 0;
  const unsigned tail0 = fits && held >= 0 ? (unsigned)((unsigned long long)tail % NB) : 0;
  if (P != kCount && !fits && tid == 0 && blockIdx.x == 0)
    flag_status(a.status, PA_DEV_NO_BLOCKS);
  // ---- the columns
  const int items = nb * a.M;  // (one CTA: few; one request: M)
  long long put = dropped;     // blocks given back so far
  int mine = 0;                // (kCount)
#pragma unroll 1
  for (int base = 0; base < items; base += kThreads) {
    const int i = base + tid, q = i / a.M, col = i - q * a.M;
    Column<WM> c;
    c.held = c.used = c.drop = 0;
    Rows r = {b0 + q, 0, 0, 0, true};
    if (i < items) {
      r.bad = s_bad[q];
      r.need = s_bits[q];
      r.before = P == kInOne ? s_before[q] : (int)before;
      r.first = a.shared_lens != nullptr && !r.bad ? a.shared_lens[r.b] >> a.bs_log2 : 0;
      if (!r.bad && fits) c.read(a, r, col, s_had + q * W, s_parent + q * W);
    }
    if constexpr (P == kCount) {
      mine += __popc(c.drop);
      continue;
    }
    int total;
    long long at = put + block_scan<kThreads>(__popc(c.drop), s_warp, total);
    put += total;
    if (i >= items) continue;
    const size_t row0 = (size_t)r.b * W * a.M + col;
#pragma unroll 1
    for (uint32_t left = c.drop; left != 0; left &= left - 1, ++at) {
      // (a ring that would hold more than there are: its state was wrong)
      if (held + at < NB) {
        unsigned to = tail0 + (unsigned)at;
        if (to >= NB) to -= NB;
        a.ring[to] = a.block_tables[row0 + (size_t)(__ffs(left) - 1) * a.M];
      } else {
        flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
      }
    }
    if (r.bad || !fits) {
      if (a.tables_out != a.block_tables)
#pragma unroll 1
        for (int w = 0; w < W; ++w)
          a.tables_out[row0 + (size_t)w * a.M] = a.block_tables[row0 + (size_t)w * a.M];
      continue;
    }
    int now[WM];
#pragma unroll
    for (int w = 0; w < WM; ++w) {
      now[w] = -1;
      if (w < W && col < s_has[q * W + w])
        now[w] = a.block_tables[row0 + (size_t)s_parent[q * W + w] * a.M];
    }
#pragma unroll
    for (int w = 0; w < WM; ++w)
      if (w < W) a.tables_out[row0 + (size_t)w * a.M] = now[w];
#pragma unroll 1
    for (uint32_t left = r.need; left != 0; left &= left - 1) {
      const int w = __ffs(left) - 1;
      if (col != s_has[q * W + w] - 1) continue;
      unsigned from = head0 + (unsigned)(r.before + __popc(r.need & ((1u << w) - 1)));
      if (from >= NB) from -= NB;
      const int id = a.ring[from];
      const bool ok = id >= 0 && id < a.num_blocks;
      if (!ok) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
      a.tables_out[row0 + (size_t)w * a.M] = ok ? id : -1;
      int64_t* pair = a.pairs + 2 * ((size_t)r.b * W + w);
      pair[0] = ok ? s_tail[q * W + w] : 0;
      pair[1] = ok ? id : 0;
    }
  }
  if constexpr (P == kCount) {
    int total;
    block_scan<kThreads>(mine, s_warp, total);
    if (tid == 0) {
      a.counts[2 * b0] = __popc(s_bits[0]);
      a.counts[2 * b0 + 1] = total;
      if (b0 == 0) {
        a.counts[2 * a.B] = head;
        a.counts[2 * a.B + 1] = tail;
      }
    }
  } else {
    // ---- the pairs of beams that need no copy, and the lengths
#pragma unroll 1
    for (int i = tid; i < nb * W; i += kThreads) {
      const int q = i / W, w = i - q * W;
      const size_t o = (size_t)b0 * W + i;
      const bool moved = fits && !s_bad[q];
      if (!moved || !(s_bits[q] >> w & 1)) a.pairs[2 * o] = a.pairs[2 * o + 1] = 0;
    }
    // (in place: a parent's length is read by the warp that replaces it)
#pragma unroll 1
    for (int i = warp; i < nb; i += kThreads / 32) {
      const size_t o = (size_t)(b0 + i) * W + lane;
      const int l = lane < W ? a.context_lens[o] : 0;
      const int p = lane < W ? s_parent[i * W + lane] : lane;
      const int from = __shfl_sync(kAll, l, p >= 0 ? p : lane);
      if (lane < W) a.lens_out[o] = !fits || s_bad[i] ? l : p >= 0 ? from : 0;
    }
    if (tid == 0 && blockIdx.x == 0) {
      const long long gave = P == kInOne ? put : all_dropped;
      const long long room = a.num_blocks - held;
      a.free_state_out[0] = head + (fits ? taken : 0);
      a.free_state_out[1] = tail + (!fits ? 0 : gave < room ? gave : room);
    }
  }
}

template <int WM>
cudaError_t launch_reorder_t(const BeamReorderArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.counts == nullptr) {
    constexpr auto kern = beam_reorder_kernel<WM, kInOne, 1024>;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = 16 * a.B * a.W;
    if (cfg.dynamicSmemBytes > 32 * 1024) {
      const cudaError_t e = ensure_dynamic_smem<kern>(200 * 1024);
      if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
  }
  constexpr int kThreads = 256;
  cfg.gridDim = dim3(a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 16 * a.W;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, beam_reorder_kernel<WM, kCount, kThreads>, a);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, beam_reorder_kernel<WM, kWrite, kThreads>, a);
}

// ---------------------------------------------------------------- backtrack
constexpr int kBackThreads = 512;
constexpr int kPiece = 32;              // steps of a piece
constexpr int kBackBytes = 160 * 1024;  // parents and beams of the steps held at a time
constexpr uint8_t kOff = 255;           // a parent that is none of the beams

__global__ void __launch_bounds__(kBackThreads)
    beam_backtrack_kernel(const BeamBacktrackArgs a, int steps) {
  extern __shared__ uint8_t s_back[];
  const int W = a.W, K = a.K, b = blockIdx.x, tid = threadIdx.x;
  const int pieces = (steps + kPiece - 1) / kPiece;
  uint8_t* s_parent = s_back;                   // [steps][W]
  uint8_t* s_beam = s_parent + steps * W;       // [K][steps], kOff: no token
  uint8_t* s_map = s_beam + (size_t)K * steps;  // [pieces][W] beam below a piece
  uint8_t* s_at = s_map + pieces * W;           // [K][pieces] beam at a piece's last step
  __shared__ int s_n[kMaxBeams];        // the hypotheses' lengths
  __shared__ uint8_t s_cur[kMaxBeams];  // their beam at the last step still to walk
  __shared__ int s_most;
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
    s_cur[tid] = n > 0 ? (uint8_t)w : kOff;
    atomicMax(&s_most, n);
  }
  __syncthreads();
  const size_t plane = (size_t)a.B * W;
  int32_t* out = a.out + (size_t)b * K * a.S;
#pragma unroll 1
  for (int i = tid; i < K * (a.S - s_most); i += kBackThreads) {  // behind all of them
    const int k = i / (a.S - s_most);
    out[(size_t)k * a.S + s_most + (i - k * (a.S - s_most))] = a.pad;
  }
  for (int hi = s_most; hi > 0; hi -= steps) {  // steps lo .. hi - 1
    const int lo = hi > steps ? hi - steps : 0, n = hi - lo;
    const int np = (n + kPiece - 1) / kPiece;
#pragma unroll 4
    for (int i = tid; i < n * W; i += kBackThreads) {
      const int s = i / W, w = i - s * W;
      const int p = a.parents[(size_t)(lo + s) * plane + (size_t)b * W + w];
      s_parent[i] = p >= 0 && p < W ? (uint8_t)p : kOff;
    }
    __syncthreads();
    // the beam below each piece, from each of its last step's
#pragma unroll 1
    for (int i = tid; i < np * W; i += kBackThreads) {
      const int p = i / W;
      int w = i - p * W;
#pragma unroll 1
      for (int s = min(n, (p + 1) * kPiece) - 1; s >= p * kPiece && w != kOff; --s)
        w = s_parent[s * W + w];
      s_map[i] = (uint8_t)w;
    }
    __syncthreads();
    // each hypothesis over the pieces (it may begin inside one)
    if (tid < K) {
      const int end = min(s_n[tid] - lo, n);  // its steps here
      int w = s_cur[tid];
      if (end > 0) {
        int p = (end - 1) / kPiece;
        s_at[tid * pieces + p] = (uint8_t)w;
#pragma unroll 1
        for (int s = end - 1; s >= p * kPiece && w != kOff; --s) w = s_parent[s * W + w];
#pragma unroll 1
        for (--p; p >= 0; --p) {
          s_at[tid * pieces + p] = (uint8_t)w;
          if (w != kOff) w = s_map[p * W + w];
        }
        s_cur[tid] = (uint8_t)w;
      }
    }
    __syncthreads();
    // all pieces of all hypotheses
#pragma unroll 1
    for (int i = tid; i < K * np; i += kBackThreads) {
      const int k = i / np, p = i - k * np;
      const int end = min(s_n[k] - lo, n), last = min(n, (p + 1) * kPiece) - 1;
      int w = p * kPiece < end ? s_at[k * pieces + p] : kOff;
#pragma unroll 1
      for (int s = last; s >= p * kPiece; --s) {
        const bool in = s < end && w != kOff;
        s_beam[(size_t)k * steps + s] = in ? (uint8_t)w : kOff;
        if (in) w = s_parent[s * W + w];
        if (in && w == kOff && lo + s > 0) flag_status(a.status, PA_DEV_BAD_BEAM);
      }
    }
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < K * n; i += kBackThreads) {
      const int k = i / n, s = i - k * n, w = s_beam[(size_t)k * steps + s];
      out[(size_t)k * a.S + lo + s] =
          w != kOff ? a.tokens[(size_t)(lo + s) * plane + (size_t)b * W + w] : a.pad;
    }
    __syncthreads();
  }
}

}  // namespace

// One CTA or one to a request: its rounds over 1,024 columns against a second launch.
bool beam_reorder_in_one(int B, int W, int M) {
  return B <= kMaxInOne && (long long)B * W <= 8192 && (long long)B * M <= 4096;
}

cudaError_t launch_beam_reorder(const BeamReorderArgs& a, cudaStream_t stream) {
  if (a.W <= 4) return launch_reorder_t<4>(a, stream);
  if (a.W <= 8) return launch_reorder_t<8>(a, stream);
  return launch_reorder_t<kMaxBeams>(a, stream);
}

cudaError_t launch_beam_backtrack(const BeamBacktrackArgs& a, cudaStream_t stream) {
  // steps whose parents and beams (and the pieces' of 32) fit shared memory
  int steps = kBackBytes / (a.W + a.K) / kPiece * kPiece;
  steps = std::min(steps, (a.S + kPiece - 1) / kPiece * kPiece);
  const int smem = steps * (a.W + a.K) + steps / kPiece * (a.W + a.K);
  const cudaError_t e = ensure_dynamic_smem<beam_backtrack_kernel>(kBackBytes * 33 / 32);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B);
  cfg.blockDim = dim3(kBackThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_backtrack_kernel, a, steps);
}

}  // namespace pk
