// beam_select.cu -- the best continuations of a request's beams over the vocabulary.
//
// With x = logits of beam w and lse_w = log sum_v exp(x[v]), candidate (w, v) has
//     c(w, v) = scores[w] + (x[v] - lse_w);
// the W largest with v != eos are chosen, best first, ties to the lowest (w, v).
//
// Only a row's own W best can be among them, and they are found while the row's sum is:
// one pass over the logits, one launch.  A request is a cluster of CTAs whose warps share
// out its live beams' rows, a piece of a row to each; no warp waits for another until all
// pieces are done.  A warp takes its piece in chunks of 512 values that its lanes hold in
// registers, with the next chunk's loads in flight, and keeps a running maximum and sum in
// every lane.  Of the first chunk the W-th largest of the lanes' maxima is a threshold that
// W values reach and few others.  Values that reach it go to a list in shared memory as
// (ordered value, ~index) keys; when the list is full, its W best are kept by counting for
// each key how many are above it, and the W-th becomes the threshold, of the other warps
// of the CTA on that row too.  The cluster's first CTA then merges the pieces' lists by
// beam and the beams' lists, in order, by as many rounds of a maximum over the lanes as
// there are beams.
//
// Rounding: sums in fp32, candidates in 64 bits (two beams' can be nearer than fp32 tells
// apart), the scores once to fp32.  A sum goes by the values' index and not by the row's
// alignment, so equal rows have equal sums.
//
// Bound: HBM, or the trip from the logits to the lists to the merge, for few rows, where
// the code itself comes from memory: it is kept short.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "pk_beam.h"
#include "pk_common.cuh"

namespace pk {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kEach = 16;           // values of a lane and chunk
constexpr int kChunk = 32 * kEach;  // values of a warp's chunk
constexpr int kList = 128;          // keys of a warp's list
constexpr int kSlack = 8;           // keys past the W best before they are sorted out
constexpr int kMaxPieces = 64;      // of a row: two lists to a lane of the merge
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;
using Key = unsigned long long;

// Order of floats and doubles as unsigned numbers.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ Key ordered(double x) {
  const Key u = (Key)__double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered(Key o) {
  return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}
// Larger values first, then lower indices; 0 stands for none.  (-0 is +0: they tie.)
__device__ __forceinline__ Key key_of(float x, int i) {
  return ((Key)ordered(x + 0.f) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(Key k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int index_of(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key warp_max(Key k) {
  const uint32_t hi = (uint32_t)(k >> 32), top = __reduce_max_sync(kAll, hi);
  const uint32_t lo = __reduce_max_sync(kAll, hi == top ? (uint32_t)k : 0u);
  return ((Key)top << 32) | lo;
}

__device__ __forceinline__ void mul_f32x2(float& d0, float& d1, float a0, float a1, float b0,
                                          float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// The warp's sums l relative to its maxima m, relative to M.  (A lane without values has
// m = -inf and l = 0; a NaN among l stays one.)
__device__ __forceinline__ float add_up(float l, float m, float M) {
  float x = l != 0.f ? l * ex2_approx((m - M) * kLog2e) : 0.f;
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

// A lane's values of a chunk as they come from memory.  VEC: 16-byte pieces, every row
// being aligned; otherwise one value after the other, neighbours in neighbouring lanes.
template <typename T, bool VEC>
struct Raw {
  static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;  // values of a piece
  static constexpr int P = kEach / N;
  using Piece = typename std::conditional<
      VEC, uint4, typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type>::type;
  Piece p[P];

  static __device__ __forceinline__ int index(int base, int i) {  // of value i of the lane
    return base + (i / N * 32 + (int)(threadIdx.x & 31)) * N + i % N;
  }
  __device__ __forceinline__ void load(const T* row, int base, int end) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int i = index(base, k * N);
      if (VEC ? i + N <= end : i < end)
        p[k] = __ldcs(reinterpret_cast<const Piece*>(row + i));
    }
  }
  // (values past the end read as -inf)
  __device__ __forceinline__ void get(const T* row, int base, int end, float (&x)[kEach]) const {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      T v[N];
      *reinterpret_cast<Piece*>(v) = p[k];
#pragma unroll
      for (int j = 0; j < N; ++j) x[k * N + j] = to_float<T>(v[j]);
    }
    if (base + kChunk > end) {  // a piece's last chunk
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int at = index(base, i);
        if (at >= end)
          x[i] = -INFINITY;
        else if (VEC && at - i % N + N > end)
          x[i] = to_float<T>(row[at]);
      }
    }
  }
};

// The W best of a warp's n <= kList keys, in order, to the list's front (by way of `room`).
// Keys differ, so that each one's place is the number of those above it.
__device__ __forceinline__ int sort_out(Key* list, Key* room, int n, int W) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
    const Key k = i < n ? list[i] : ~0ull;
    int above = 0;
#pragma unroll 4
    for (int q = 0; q < n; ++q) above += list[q] > k;
    if (i < n && above < W) room[above] = k;
  }
  __syncwarp();
  n = min(n, W);
  if (lane < n) list[lane] = room[lane];
  __syncwarp();
  return n;
}

// x[i] for an i known at run time only, without a trip through memory.
__device__ __forceinline__ float pick(const float (&x)[kEach], int i) {
  float y[kEach / 2];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = i & 8 ? x[j + 8] : x[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = i & 4 ? y[j + 4] : y[j];
  y[0] = i & 2 ? y[2] : y[0];
  y[1] = i & 2 ? y[3] : y[1];
  return i & 1 ? y[1] : y[0];
}

// The W-th largest of the lanes' x: a bitonic sort over the lanes, largest first.
__device__ __forceinline__ uint32_t nth_largest(uint32_t x, int W) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t y = __shfl_xor_sync(kAll, x, j);
      x = ((lane & k) == 0) == ((lane & j) == 0) ? max(x, y) : min(x, y);
    }
  return __shfl_sync(kAll, x, W - 1);
}

// A warp's piece [begin, end) of a row: its W best to the list (0 behind the last), its
// maximum and sum returned.  shared: a threshold that W values of the row reach.
template <typename T, bool VEC>
__device__ __forceinline__ float2 scan(const T* row, int begin, int end, int eos, int W,
                                       Key* list, Key* room, uint32_t* shared) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
  float t = -FLT_MAX;  // values from it on are candidates (-inf and NaN never)
  int n = 0;
  Raw<T, VEC> raw;
  raw.load(row, begin, end);
#pragma unroll 1
  for (int base = begin; base < end; base += kChunk) {
    const bool last = base + kChunk >= end;
    float x[kEach];
    raw.get(row, base, end, x);
    if (!last) raw.load(row, base + kChunk, end);
    float mt = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < kEach; i += 2) mt = max3f(mt, x[i], x[i + 1]);
    if (mt > m) {
      l *= ex2_approx((m - mt) * kLog2e);  // (m = -inf: l is 0)
      m = mt;
    }
    const float ref = m == -INFINITY ? 0.f : -m;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
      float a, b;
      add_f32x2(a, b, x[i], x[i + 1], ref, ref);
      mul_f32x2(a, b, a, b, kLog2e, kLog2e);
      add_f32x2(s0, s1, s0, s1, ex2_approx(a), ex2_approx(b));
    }
    l += s0 + s1;
    if (eos >= base && eos - base < kChunk) {  // the end is no candidate
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (Raw<T, VEC>::index(base, i) == eos) x[i] = -INFINITY;
      mt = x[0];
#pragma unroll
      for (int i = 1; i < kEach; ++i) mt = fmaxf(mt, x[i]);
    }
    if (base == begin) {
      // The W-th largest of the lanes' maxima is reached by W values (an order of NaN's
      // does not matter: their row has no candidates).
      const uint32_t o = nth_largest(ordered(mt), W);
      t = fmaxf(t, unordered(o));
      if (lane == 0 && o > ordered(-FLT_MAX)) atomicMax(shared, o);
    }
    t = fmaxf(t, unordered(*(volatile uint32_t*)shared));
    uint32_t hits = 0;  // of the lane's values, those that reach t
    if (mt >= t) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) hits |= x[i] >= t ? 1u << i : 0u;
    }
    bool full = false;
#pragma unroll 1
    for (;;) {  // one of a lane at a time
      const unsigned mask = __ballot_sync(kAll, hits != 0);
      if (mask != 0 ? n + __popc(mask) > kList : full || last || n >= W + kSlack) {
        n = sort_out(list, room, n, W);
        if (n == W) {
          // An equal value of a later chunk comes too late (of this one it may not: its
          // values come in no order of their indices).
          const uint32_t lowest = (uint32_t)(list[W - 1] >> 32);
          if (mask == 0) t = fmaxf(t, unordered(lowest + 1));
          if (lane == 0) atomicMax(shared, lowest);
        }
        full = true;
      }
      if (mask == 0) break;
      if (hits != 0) {
        const int i = __ffs(hits) - 1;
        list[n + __popc(mask & ((1u << lane) - 1))] =
            key_of(pick(x, i), Raw<T, VEC>::index(base, i));
        hits &= hits - 1;
      }
      n += __popc(mask);
    }
  }
  if (lane >= n && lane < W) list[lane] = 0;
  const float M = unordered(__reduce_max_sync(kAll, ordered(m)));
  return make_float2(M, add_up(l, m, M));
}

// What the merge holds: per row (beam) of the cluster its best keys, maximum and sum.
struct Rows {
  Key* top;   // [W][W]
  float2* ml;  // [W]
};

// log x of a sum, to 2^-25: e log 2 + log f, x = 2^e f with f in [1 / sqrt 2, sqrt 2), so
// that fp32's half steps are those of a number below 0.35.
__device__ __forceinline__ double log_of(float x) {
  int e;
  float f = frexpf(x, &e);
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  return e * 0.69314718055994531 + (double)logf(f);
}

// The best over the beams, one CTA to a request; alive: the beams whose rows were taken.
__device__ __forceinline__ void choose(const BeamSelectArgs& a, int b, uint32_t alive, Rows r,
                                       Key* cand, double* s_lse, float end_x) {
  const int W = a.W, tid = threadIdx.x, lane = tid & 31;
  const float sc = lane < W ? a.scores[b * W + lane] : -INFINITY;
  if (tid < 32) {
    double lse = -INFINITY;
    if (alive >> lane & 1) {
      const float2 ml = r.ml[lane];
      // Nothing allowed (a sum of 0) gives no candidate; NaN or +inf among the logits neither.
      if (isnan(ml.y))
        flag_status(a.status, PA_DEV_BAD_LOGITS);
      else if (ml.y > 0.f)
        lse = (double)ml.x + log_of(ml.y);
    }
    s_lse[lane] = lse;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < W * W; i += kThreads) {
    const int w = i / W;
    const Key k = (alive >> w & 1) ? r.top[i] : 0;
    const double lse = s_lse[w];
    // (0: none; what a finite number is ordered as is not)
    cand[i] = k != 0 && lse > -INFINITY
                  ? ordered((double)a.scores[b * W + w] + ((double)value_of(k) - lse) + 0.0)
                  : 0;
  }
  __syncthreads();
  if (tid >= 32) return;
  // Lane i holds the next candidate of beam i.
  int at = 0;
  Key c = lane < W ? cand[lane * W] : 0;
  Key my_c = 0, my_key = 0, last_c = 0, last_key = 0;  // of place `lane`; of the last place
  int my_beam = lane, last_beam = 0;
#pragma unroll 1
  for (int j = 0; j < W; ++j) {
    const Key best = warp_max(c);
    last_c = best;
    if (best == 0) break;
    last_beam = __ffs(__ballot_sync(kAll, c == best)) - 1;
    const int place = __shfl_sync(kAll, at, last_beam);
    last_key = r.top[last_beam * W + place];
    if (lane == j) {
      my_c = best;
      my_beam = last_beam;
      my_key = last_key;
    }
    if (lane == last_beam) {
      ++at;
      c = at < W ? cand[lane * W + at] : 0;
    }
  }
  if (lane >= W) return;
  const int o = b * W + lane;
  a.tokens[o] = my_key != 0 ? index_of(my_key) : a.pad;
  a.parents[o] = my_beam;
  a.new_scores[o] = my_c != 0 ? (float)unordered(my_c) : -INFINITY;
  // Ends that are better than the last one chosen.
  float ended = -INFINITY;
  const double lse = s_lse[lane];
  if (lse > -INFINITY && a.eos >= 0) {
    const double e = (double)sc + ((double)end_x - lse) + 0.0;
    const Key eo = ordered(e);
    const bool ahead = last_c != 0 && lane == last_beam
                           ? key_of(end_x, a.eos) > last_key
                           : eo > last_c || (eo == last_c && lane < last_beam);
    if (end_x > -INFINITY && ahead) ended = (float)e;
  }
  a.ended[o] = ended;
}

// The beam of the i-th live row.
__device__ __forceinline__ int live_beam(uint32_t alive, int i) {
#pragma unroll 1
  for (; i > 0; --i) alive &= alive - 1;
  return __ffs(alive) - 1;
}

// A cluster to a request.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) beam_select_kernel(const BeamSelectArgs a) {
  extern __shared__ Key s_dyn[];
  __shared__ Key s_list[kWarps][kList];
  __shared__ Key s_room[kWarps][kMaxBeams];
  __shared__ float2 s_ml[kWarps];
  __shared__ uint32_t s_threshold[kMaxBeams];
  __shared__ double s_lse[32];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = a.ranks, b = blockIdx.x / ranks, rank = blockIdx.x - b * ranks, W = a.W;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kMaxBeams) s_threshold[tid] = 0;  // below any value
  pdl_wait();
  pdl_launch_dependents();
  // A beam whose score is not finite is not there.
  const uint32_t alive =
      __ballot_sync(kAll, lane < W && isfinite(a.scores[b * W + (lane < W ? lane : 0)]));
  const int rows = __popc(alive);
  // What the choice needs of the beams, a lane to each.
  float end_x = -INFINITY;
  if (rank == 0 && warp == 0 && (alive >> lane & 1) && a.eos >= 0)
    end_x = to_float<T>(
        static_cast<const T*>(a.logits)[(long long)(b * W + lane) * a.row_stride + a.eos]);
  // Pieces of a row: whole 16-byte pieces each, the last ones may be empty.
  const int pieces = min(kMaxPieces, ranks * kWarps / max(rows, 1));
  const int length = ((a.V + pieces - 1) / pieces + 15) / 16 * 16;
  __syncthreads();
  // A row's pieces go to neighbouring warps, which share a threshold.
  const int per = (rows * pieces + ranks - 1) / ranks, task = rank * per + warp;
  if (warp < per && task < rows * pieces) {
    const int r = task / pieces, w = live_beam(alive, r);
    const int begin = (int)min((long long)(task - r * pieces) * length, (long long)a.V);
    const int end = (int)min((long long)begin + length, (long long)a.V);
    const T* x = static_cast<const T*>(a.logits) + (long long)(b * W + w) * a.row_stride;
    const float2 ml = scan<T, VEC>(x, begin, end, a.eos, W, s_list[warp], s_room[warp],
                                    &s_threshold[w]);
    if (lane == 0) s_ml[warp] = ml;
  }
  if (ranks > 1)
    cluster.sync();
  else
    __syncthreads();
  if (rank == 0) {
    // All lists, [row][piece][W], and their maxima and sums.
    Key* keys = s_dyn;
    const int lists = rows * pieces;
    float2* ml = reinterpret_cast<float2*>(keys + (size_t)ranks * kWarps * W);
    Rows r = {reinterpret_cast<Key*>(ml + ranks * kWarps), nullptr};
    r.ml = reinterpret_cast<float2*>(r.top + W * W);
    Key* cand = reinterpret_cast<Key*>(r.ml + kMaxBeams);
    auto at_rank = [&](auto* p, int r) { return ranks > 1 ? cluster.map_shared_rank(p, r) : p; };
#pragma unroll 1
    for (int i = tid; i < lists * W; i += kThreads) {
      const int q = i / W, from = q / per;
      keys[i] = *at_rank(&s_list[q - from * per][i - q * W], from);
    }
#pragma unroll 1
    for (int q = tid; q < lists; q += kThreads)
      ml[q] = *at_rank(&s_ml[q % per], q / per);
    __syncthreads();
    // A warp to a beam: rounds of the largest head of its lists, two to a lane.
#pragma unroll 1
    for (int i = warp; i < rows; i += kWarps) {
      const int w = live_beam(alive, i);
      const Key* mine = keys + (size_t)i * pieces * W;
      int at[2] = {0, 0};
      Key head[2];
      float m[2], l[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int q = lane + 32 * e;
        const bool has = q < pieces;
        head[e] = has ? mine[(size_t)q * W] : 0;
        const float2 v = has ? ml[i * pieces + q] : make_float2(-INFINITY, 0.f);
        m[e] = v.x;
        l[e] = v.y;
      }
      const float M = unordered(__reduce_max_sync(kAll, max(ordered(m[0]), ordered(m[1]))));
      const float L = add_up(l[0], m[0], M) + add_up(l[1], m[1], M);
      if (lane == 0) r.ml[w] = make_float2(M, L);
#pragma unroll 1
      for (int j = 0; j < W; ++j) {
        const Key k = warp_max(max(head[0], head[1]));
        if (lane == 0) r.top[w * W + j] = k;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (k != 0 && head[e] == k) {
            ++at[e];
            head[e] = at[e] < W ? mine[(size_t)(lane + 32 * e) * W + at[e]] : 0;
          }
      }
    }
    __syncthreads();
    choose(a, b, alive, r, cand, s_lse, end_x);
  }
  if (ranks > 1) cluster.sync();  // nobody leaves while its lists are read
}

int dynamic_bytes(int W, int ranks) {
  return ranks * kWarps * (W + 1) * 8 + (2 * W * W + kMaxBeams) * 8;
}

template <typename T, bool VEC>
cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t stream) {
  constexpr auto kern = beam_select_kernel<T, VEC>;
  const int smem = dynamic_bytes(a.W, a.ranks);
  if (smem > 24 * 1024) {  // (with the lists more than 48 KB)
    const cudaError_t e = ensure_dynamic_smem<kern>(dynamic_bytes(kMaxBeams, kMaxCluster));
    if (e != cudaSuccess) return e;
  }
  if (a.ranks > 8) {
    const cudaError_t e = ensure_large_cluster<kern>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ranks * a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)a.ranks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T>
cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 &&
                   (a.B * a.W == 1 || a.row_stride * (int)sizeof(T) % 16 == 0);
  return vec ? launch_t<T, true>(a, stream) : launch_t<T, false>(a, stream);
}

}  // namespace

// CTAs of a request: as many as the GPU holds at two to an SM, and as there are chunks of
// its rows for their warps.
int beam_select_ranks(int B, int W, int V) {
  const int nsm = sm_count() > 0 ? sm_count() : 152;
  const long long warps = (long long)W * ((V - 1) / kChunk + 1);
  int c = W > kWarps ? 2 : 1;  // (a warp to a row at least)
  while (c < kMaxCluster && 2LL * c * B <= 2 * nsm && c * kWarps < warps) c *= 2;
  return c;
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t stream) {
  return a.dtype == PA_F32    ? launch_t<float>(a, stream)
         : a.dtype == PA_BF16 ? launch_t<__nv_bfloat16>(a, stream)
                              : launch_t<__half>(a, stream);
}

}  // namespace pk
