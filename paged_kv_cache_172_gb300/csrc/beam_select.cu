// beam_select.cu -- the best continuations of a request's beams over the vocabulary.
//
// With x = logits of beam w and lse_w = log sum_v exp(x[v]), candidate (w, v) has
//     c(w, v) = scores[w] + (x[v] - lse_w);
// the W largest with v != eos are chosen, best first, ties to the lowest (w, v).
//
// Only a row's own W best can be among them, and they are found while the row's sum is:
// one pass over the logits.  A CTA takes a row, or one of its `splits` ranges, in chunks
// of 8,192 that its threads hold in registers, with the next chunk's loads in flight.
// Every thread keeps a running maximum and sum of its own.  Of the first chunk the W-th
// largest of 64 groups' maxima is a threshold that W values reach and few others; values
// that reach it go to a list in shared memory as (ordered value, ~index) keys, of which
// the W best are kept by counting for each how many are above it.  The W-th of them is
// the threshold of the chunks behind.  Where a chunk has more values over it than the
// list holds (logits that rise along the row) its own threshold is taken, and where that
// does not help (equal values) W rounds of the largest key below the last one.  A second
// launch, one CTA to a request, merges the ranges' lists and then the beams', both in
// order, by as many rounds as there are beams.
//
// Rounding: sums in fp32 by thread and in 64 bits from there, candidates in 64 bits (two
// beams' can be nearer than fp32 tells apart), the scores once to fp32.  A sum goes by
// the values' index and not by the row's alignment, so equal rows have equal sums.
//
// Bound: HBM, or the trip from the logits to the threshold to the list and the second
// launch, for few rows.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "pk_beam.h"
#include "pk_common.cuh"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kEach = 16;                 // values of a thread and chunk
constexpr int kChunk = kThreads * kEach;  // values of a chunk
constexpr int kGroups = kThreads / 8;     // lanes whose maxima make the threshold
constexpr int kList = 2048;               // keys that reached the threshold, at most
constexpr int kSlack = 64;                // keys past the W best before they are sorted out
constexpr int kMaxSplits = 32;
constexpr float kLog2e = 1.4426950408889634f;
using Key = unsigned long long;

// Order of floats as unsigned numbers.  (-0 is taken as +0 before: equal values tie.)
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Larger values first, then lower indices; 0 stands for none.
__device__ __forceinline__ Key key_of(float x, int i) {
  return ((Key)ordered(x) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(Key k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int index_of(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key warp_max(Key k) {
  const uint32_t hi = (uint32_t)(k >> 32), top = __reduce_max_sync(kAll, hi);
  const uint32_t lo = __reduce_max_sync(kAll, hi == top ? (uint32_t)k : 0u);
  return ((Key)top << 32) | lo;
}

// The warp's sums l relative to maxima m, relative to M, added in 64 bits.  (A lane
// without values has m = -inf and l = 0; a NaN among l stays one.)
__device__ __forceinline__ double add_up(float l, float m, float M) {
  double x = l != 0.f ? l * ex2_approx((m - M) * kLog2e) : 0.f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  if constexpr (std::is_same<T, float>::value)
    return x;
  else if constexpr (std::is_same<T, __half>::value)
    return __half2float(x);
  else
    return __bfloat162float(x);
}

// A thread's values of a chunk as they come from memory.  VEC: 16-byte pieces, every row
// being aligned; otherwise one value after the other, neighbours in neighbouring lanes.
template <typename T, bool VEC>
struct Raw {
  static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;  // values of a piece
  static constexpr int P = kEach / N;
  using Piece = typename std::conditional<
      VEC, uint4, typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type>::type;
  Piece p[P];

  static __device__ __forceinline__ int index(int base, int k, int j) {  // of value j, piece k
    return base + (k * kThreads + (int)threadIdx.x) * N + j;
  }
  __device__ __forceinline__ void load(const T* row, int base, int end) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int i = index(base, k, 0);
      if (VEC ? i + N <= end : i < end)
        p[k] = __ldcs(reinterpret_cast<const Piece*>(row + i));
    }
  }
  // (values past the end read as -inf)
  __device__ __forceinline__ void get(const T* row, int base, int end, float (&x)[kEach]) const {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int i = index(base, k, 0);
      if constexpr (VEC) {
        T v[N];
        *reinterpret_cast<uint4*>(v) = p[k];
#pragma unroll
        for (int j = 0; j < N; ++j) x[k * N + j] = to_float<T>(v[j]) + 0.f;
        if (i + N > end) {  // the row's last piece, or none of it
#pragma unroll
          for (int j = 0; j < N; ++j)
            x[k * N + j] = i + j < end ? to_float<T>(row[i + j]) + 0.f : -INFINITY;
        }
      } else {
        T v;
        *reinterpret_cast<Piece*>(&v) = p[k];
        x[k] = i < end ? to_float<T>(v) + 0.f : -INFINITY;
      }
    }
  }
};

struct Shared {
  Key list[kList];
  Key sorted[kMaxBeams];
  uint32_t group[kGroups];
  float sum[kThreads / 32];
  float max[kThreads / 32];
  Key best[kThreads / 32];
  int count;
  uint32_t threshold;  // ordered
};

// The W best of the list's n keys, in order, to its front and to `sorted`; all threads.
// Keys differ, so that each one's place is the number of those above it.
__device__ __forceinline__ int sort_out(Shared& s, int n, int W) {
  const int keep = min(n, W);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key k = s.list[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += s.list[j] > k;
    if (above < W) s.sorted[above] = k;
  }
  __syncthreads();
  if (threadIdx.x < keep) s.list[threadIdx.x] = s.sorted[threadIdx.x];
  if (threadIdx.x == 0) {
    s.count = keep;
    // below any value until there are W
    s.threshold = keep == W ? (uint32_t)(s.sorted[W - 1] >> 32) : 0u;
  }
  __syncthreads();
  return keep;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) beam_rows_kernel(const BeamSelectArgs a) {
  __shared__ Shared s;
  const int row = blockIdx.x, split = blockIdx.y, W = a.W;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  if (!isfinite(a.scores[row])) return;  // a dead beam: the second launch knows it
  const T* x0 = static_cast<const T*>(a.logits) + (long long)row * a.row_stride;
  const int chunks = (a.V - 1) / kChunk + 1;
  const int c0 = (int)((long long)split * chunks / a.splits);
  const int c1 = (int)((long long)(split + 1) * chunks / a.splits);

  Raw<T, VEC> raw;
  if (c0 < c1) raw.load(x0, c0 * kChunk, a.V);
  if (tid == 0) {
    s.count = 0;
    s.threshold = 0;
  }
  float m = -INFINITY, l = 0.f;
  int kept = 0;  // of the list's keys, those that were sorted out
  int held = 0;  // keys of the chunks before
  constexpr uint32_t kNone = 0x007fffffu;  // ordered(-inf): no candidate
  for (int c = c0; c < c1; ++c) {
    const int base = c * kChunk;
    float x[kEach];
    raw.get(x0, base, a.V, x);
    if (c + 1 < c1) raw.load(x0, base + kChunk, a.V);
    // ---- running maximum and sum
    float mt = x[0];
#pragma unroll
    for (int i = 1; i < kEach; ++i) mt = fmaxf(mt, x[i]);
    if (mt > m) {
      l *= ex2_approx((m - mt) * kLog2e);  // (m = -inf: l is 0)
      m = mt;
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kEach; ++i) l += ex2_approx((x[i] - ref) * kLog2e);
    // ---- candidates: the end is none
    constexpr int N = Raw<T, VEC>::N;
    if (a.eos >= base && a.eos - base < kChunk) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (Raw<T, VEC>::index(base, i / N, i % N) == a.eos) x[i] = -INFINITY;
      mt = x[0];
#pragma unroll
      for (int i = 1; i < kEach; ++i) mt = fmaxf(mt, x[i]);
    }
    const uint32_t top = ordered(mt);
    // Keys from `t` on (behind the first chunk: above it, an equal one comes too late).
    auto push = [&](uint32_t t) {
      if (top < t || top <= kNone) return;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint32_t o = ordered(x[i]);
        if (o >= t && o > kNone && !isnan(x[i])) {
          const int at = atomicAdd(&s.count, 1);
          if (at < kList) s.list[at] = key_of(x[i], Raw<T, VEC>::index(base, i / N, i % N));
        }
      }
    };
    // The W-th largest of the groups' maxima, which W of this chunk's values reach.
    auto own_threshold = [&]() {
      uint32_t g = top;
      g = max(g, __shfl_xor_sync(kAll, g, 1));
      g = max(g, __shfl_xor_sync(kAll, g, 2));
      g = max(g, __shfl_xor_sync(kAll, g, 4));
      if ((lane & 7) == 0) s.group[tid >> 3] = g;
      __syncthreads();
      if (tid < kGroups) {
        const uint32_t mine = s.group[tid];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < kGroups; ++j) {
          const uint32_t o = s.group[j];
          above += o > mine || (o == mine && j < tid);
        }
        if (above == W - 1) s.threshold = mine;
      }
      __syncthreads();
      return s.threshold;
    };
    if (c == c0) {
      push(own_threshold());
    } else {
      const uint32_t t = s.threshold;
      push(kept == W ? t + 1 : t);
    }
    __syncthreads();
    int n = s.count;
    __syncthreads();
    const bool full = n > kList;
    if (full) {
      if (tid == 0) s.count = held;
      const uint32_t before = kept == W ? s.threshold + 1 : 0u;
      const uint32_t mine = own_threshold();
      push(max(mine, before));
      __syncthreads();
      n = s.count;
      if (n > kList) {
        Key last = ~0ull;
        for (int r = 0; r < W; ++r) {
          Key k = 0;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const Key o = key_of(x[i], Raw<T, VEC>::index(base, i / N, i % N));
            if (ordered(x[i]) > kNone && !isnan(x[i]) && o < last && o > k) k = o;
          }
          k = warp_max(k);
          if (lane == 0) s.best[warp] = k;
          __syncthreads();
          k = warp_max(lane < kThreads / 32 ? s.best[lane] : 0);
          if (tid == 0) s.list[held + r] = k;
          last = k;
          __syncthreads();
        }
        n = held + W;  // (0 where there was none: below every key)
        while (n > held && s.list[n - 1] == 0) --n;
      }
      __syncthreads();
    }
    if (c == c0 || full || n > W + kSlack || c + 1 == c1) n = kept = sort_out(s, n, W);
    held = n;
  }
  // ---- the row's (or range's) keys, maximum and sum
  const size_t at = (size_t)row * a.splits + split;
  if (tid < W) a.ws_keys[at * W + tid] = tid < kept ? s.sorted[tid] : 0ull;
  const float mw = unordered(__reduce_max_sync(kAll, ordered(m)));
  l *= ex2_approx((m == -INFINITY ? -INFINITY : m - mw) * kLog2e);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(kAll, l, d);
  if (lane == 0) {
    s.max[warp] = mw;
    s.sum[warp] = l;
  }
  __syncthreads();
  if (warp > 0) return;
  m = lane < kThreads / 32 ? s.max[lane] : -INFINITY;
  l = lane < kThreads / 32 ? s.sum[lane] : 0.f;
  const float M = unordered(__reduce_max_sync(kAll, ordered(m)));
  const double L = add_up(l, m, M);
  if (lane == 0) {
    a.ws_max[at] = M;
    a.ws_sum[at] = (float)L;
  }
}

// Order of doubles as unsigned numbers.
__device__ __forceinline__ double unordered(Key o) {
  return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}
__device__ __forceinline__ Key ordered(double x) {
  const Key u = (Key)__double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

// One CTA to a request, a warp to a beam.
template <typename T>
__global__ void beam_merge_kernel(const BeamSelectArgs a) {
  extern __shared__ Key s_keys[];  // [W][splits * W], then [W][W] sorted
  __shared__ double s_lse[kMaxBeams];
  const int W = a.W, S = a.splits, b = blockIdx.x;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Key* s_top = s_keys + (size_t)W * S * W;
  pdl_wait();
  pdl_launch_dependents();
  const int row = b * W + w;
  const float score = a.scores[row];
  const bool alive = isfinite(score);
  // ---- a warp's beam: its log-sum-exp, and its W best in order
  double lse = -INFINITY;
  if (alive) {
    const Key* keys = a.ws_keys + (size_t)row * S * W;
    for (int i = lane; i < S * W; i += 32) s_keys[(size_t)w * S * W + i] = keys[i];
    const float m = lane < S ? a.ws_max[(size_t)row * S + lane] : -INFINITY;
    const float part = lane < S ? a.ws_sum[(size_t)row * S + lane] : 0.f;
    const float M = unordered(__reduce_max_sync(kAll, ordered(m)));
    const double l = add_up(part, m, M);
    // Nothing allowed (l = 0) gives no candidate; NaN or +inf among the logits neither.
    if (isnan(l)) {
      if (lane == 0) flag_status(a.status, PA_DEV_BAD_LOGITS);
    } else if (l > 0.0) {
      lse = (double)M + log(l);
    }
  }
  __syncwarp();
  const bool some = lse > -INFINITY;
  int at = 0;  // the lane's place in its range's list
  Key head = some && lane < S ? s_keys[((size_t)w * S + lane) * W] : 0;
  for (int r = 0; r < W; ++r) {
    const Key k = warp_max(head);
    if (lane == 0) s_top[w * W + r] = k;
    if (k != 0 && head == k) {
      ++at;
      head = at < W ? s_keys[((size_t)w * S + lane) * W + at] : 0;
    }
  }
  if (lane == 0) s_lse[w] = lse;
  __syncthreads();
  if (w > 0) return;
  // ---- all beams: lane i holds the next candidate of beam i
  const float sc = lane < W ? a.scores[b * W + lane] : -INFINITY;
  const double ls = lane < W ? s_lse[lane] : -INFINITY;
  const bool here = ls > -INFINITY;
  auto candidate = [&](float x) { return (double)sc + ((double)x - ls) + 0.0; };
  at = 0;
  Key k = here ? s_top[lane * W] : 0;
  // (0: none; what a finite number is ordered as is not)
  Key c = k != 0 ? ordered(candidate(value_of(k))) : 0;
  Key my_key = 0;  // of place `lane`
  int my_beam = lane;
  Key my_c = 0, last_c = 0, last_key = 0;
  int last_beam = 0;
  for (int r = 0; r < W; ++r) {
    const Key best = warp_max(c);
    last_c = best;
    if (best == 0) break;
    last_beam = __ffs(__ballot_sync(kAll, c == best)) - 1;
    last_key = __shfl_sync(kAll, k, last_beam);
    if (lane == r) {
      my_c = best;
      my_beam = last_beam;
      my_key = last_key;
    }
    if (lane == last_beam) {
      ++at;
      k = at < W ? s_top[lane * W + at] : 0;
      c = k != 0 ? ordered(candidate(value_of(k))) : 0;
    }
  }
  if (lane >= W) return;
  const int o = b * W + lane;
  a.tokens[o] = my_key != 0 ? index_of(my_key) : a.pad;
  a.parents[o] = my_beam;
  a.new_scores[o] = my_c != 0 ? (float)unordered(my_c) : -INFINITY;
  // ---- ends that are better than the last one chosen
  float ended = -INFINITY;
  if (here && a.eos >= 0) {
    const float x = to_float<T>(
        static_cast<const T*>(a.logits)[(long long)o * a.row_stride + a.eos]) + 0.f;
    const Key e = ordered(candidate(x));
    const bool ahead = last_c != 0 && lane == last_beam
                           ? key_of(x, a.eos) > last_key
                           : e > last_c || (e == last_c && lane < last_beam);
    if (x > -INFINITY && ahead) ended = (float)unordered(e);
  }
  a.ended[o] = ended;
}

template <typename T>
cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 &&
                   (a.B * a.W == 1 || a.row_stride * (int)sizeof(T) % 16 == 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * a.W, a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, beam_rows_kernel<T, true>, a)
                      : cudaLaunchKernelEx(&cfg, beam_rows_kernel<T, false>, a);
  if (e != cudaSuccess) return e;
  const int smem = (a.W * a.splits * a.W + a.W * a.W) * (int)sizeof(Key);
  constexpr auto merge = beam_merge_kernel<T>;
  if (smem > 40 * 1024) {
    e = ensure_dynamic_smem<merge>(80 * 1024);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(a.B);
  cfg.blockDim = dim3(32 * a.W);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, merge, a);
}

}  // namespace

// Ranges of a row: as many as fill two CTAs to an SM, a chunk each at least, and no more
// than the second launch can hold the keys of (64 KB).
int beam_select_splits(int B, int W, int V) {
  const long long rows = (long long)B * W;
  const int nsm = sm_count() > 0 ? sm_count() : 152;
  const int chunks = (V - 1) / kChunk + 1;
  long long s = (2LL * nsm + rows - 1) / rows;
  if (s > chunks) s = chunks;
  if (s > kMaxSplits) s = kMaxSplits;
  if (s > 8192 / (W * W)) s = 8192 / (W * W);
  return s > 1 ? (int)s : 1;
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t stream) {
  return a.dtype == PA_F32    ? launch_t<float>(a, stream)
         : a.dtype == PA_BF16 ? launch_t<__nv_bfloat16>(a, stream)
                              : launch_t<__half>(a, stream);
}

}  // namespace pk
