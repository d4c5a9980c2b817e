// beam_select.cu -- the best continuations of a request's beams over the vocabulary.
//
// With x = logits of beam w and lse_w = log sum_v exp(x[v]), candidate (w, v) has
//     c(w, v) = scores[w] + (x[v] - lse_w);
// the W largest with v != eos are chosen, best first, ties to the lowest (w, v).
//
// Only a row's own W best can be among them, and they are found while the row's sum is:
// one pass over the logits, one launch.  A request is a cluster of CTAs whose warps share
// out its live beams' rows, a piece of a row to each; no warp waits for another until all
// pieces are done.  A warp's piece comes through a ring of its own in shared memory
// (asynchronous copies of 16 bytes a lane), so that its loop takes few registers and
// little code; every lane keeps a running maximum and sum.  The piece's W best are a
// sorted list of (ordered value, ~index) keys over the lanes, into which values that reach
// a threshold are inserted one by one: the W-th of the list, or what the row's other warps
// of the CTA know.  In a chunk where many values reach that (the first one) it is raised to
// the W-th largest of the lanes' maxima first (W rounds), or, for more than 8 beams, these
// are merged into the list as a whole until few lanes are left.  The cluster's first CTA then
// merges the pieces' lists by beam and the beams' lists, in order: by as many rounds of a
// maximum over the lists' heads as there are beams, or, for more than 8, by bitonic merges.
// (The merges against rounds, with the lanes' maxima merged either way: 32 beams of 32,000
// bf16 logits 21.7 -> 16.3 us, 156 requests of 32 x 1,152 fp32 88 -> 50, 2 of 16 x 140,000
// bf16 17.2 -> 16.6; a kernel of its own, since its code costs the small calls 0.2 us.)
//
// Rounding: sums in fp32, candidates in 64 bits (two beams' can be nearer than fp32 tells
// apart), the scores once to fp32.  A sum goes by the values' index, and not by the row's
// alignment or by the cluster that takes it, so equal rows of a request have equal sums.
//
// Bound: HBM, or, for few rows, the trip from the logits to the lists to the merge, on
// which the code itself comes from memory: it is kept short (24 to 31 KB a kernel).  A warp
// takes 0.65 us to a chunk of 512 values, whatever their type, where an SM has 16 warps.
// Measured (GB300, in a replayed graph): one request of 4 beams and 32,000 fp32 logits
// 6.1 us; 64 of 4 and 50,001 bf16 in rows of odd lengths 14.8 us; 32 of 16 and 255,999
// fp32, of which 430 MB are live beams', 80 us, 5.4 TB/s, 0.79 of the copy rate (clusters
// of 4 on 128 SMs, each at the 50 bytes a ns that an SM takes in).  There chunks of 256
// values took 143 us, chunks without a ring 116, two CTAs to an SM with half the ring 84.
#include <cuda_bf16.h>
#include <float.h>
#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "pk_beam.h"
#include "pk_common.cuh"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 16;          // of a CTA
constexpr int kEach = 16;           // values of a lane and chunk
constexpr int kChunk = 32 * kEach;  // values of a warp's chunk
constexpr int kRing = 8320;         // bytes of a warp's ring: four or eight chunks and 16 each
constexpr int kMany = 64;           // values of a chunk that are too many to be inserted
constexpr int kManyLanes = 8;       // lanes whose values are merged rather than inserted
constexpr int kFewBeams = 8;        // most for which W rounds of a maximum are done
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

// The sum over the lanes of l relative to maximum m, relative to M.  (A lane without
// values has m = -inf and l = 0; a NaN among l stays one.)
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

__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
// Waits until at most `left` of the lane's groups are still under way.
template <int left>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
}

// A piece of a row in a warp's ring, chunk by chunk.  The copies are of whole 16 bytes, from
// `lead` bytes before the piece on where rows are not aligned (the 16 bytes that hold the
// first value; a chunk then ends in 16 bytes more).  A lane's values: VEC, every row being
// aligned, 16 bytes each time; otherwise one at a time, neighbours in neighbouring lanes.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = 16 / (int)sizeof(T);  // values of 16 bytes
  static constexpr int kCopies = kEach / N, kBytes = kChunk * (int)sizeof(T);
  static constexpr int kSlot = kBytes + 16, kSlots = kRing / kSlot;
  const T* from;    // the first value's 16 bytes
  int lead, bytes;  // before the first value, in all
  uint8_t* ring;

  static __device__ __forceinline__ int index(int base, int j) {  // of value j of the lane
    const int lane = threadIdx.x & 31;
    return VEC ? base + (j / N * 32 + lane) * N + j % N : base + j * 32 + lane;
  }
  // Requests chunk i, if there is one; a group in any case.
  __device__ __forceinline__ void request(int i) const {
    const int lane = threadIdx.x & 31, at = i * kBytes + lane * 16;
    const uint32_t to = smem_u32(ring) + i % kSlots * kSlot + lane * 16;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(from) + at;
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      if (at + q * 512 < bytes)
        copy_async(to + q * 512, src + q * 512, min(bytes - at - q * 512, 16));
    if (!VEC && lane == 0 && at + kBytes < bytes)
      copy_async(to + kBytes, src + kBytes, min(bytes - at - kBytes, 16));
    copy_commit();
  }
  // Values from index `end` on read as -inf.
  __device__ __forceinline__ void get(int i, int base, int end, float (&x)[kEach]) const {
    const int lane = threadIdx.x & 31;
    const uint8_t* slot = ring + i % kSlots * kSlot;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < kCopies; ++q) {
        T v[N];
        *reinterpret_cast<uint4*>(v) =
            *reinterpret_cast<const uint4*>(slot + q * 512 + lane * 16);
#pragma unroll
        for (int j = 0; j < N; ++j) x[q * N + j] = to_float<T>(v[j]);
      }
    } else {
      const T* v = reinterpret_cast<const T*>(slot + lead) + lane;
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = to_float<T>(v[j * 32]);
    }
    if (base + kChunk > end) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (index(base, j) >= end) x[j] = -INFINITY;
    }
  }
};

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

// The 32 largest of two keys a lane, in order: mine in order, rising the other way round: the
// larger of every two, a bitonic merge.
__device__ __forceinline__ Key merge_sorted(Key mine, Key rising) {
  const int lane = threadIdx.x & 31;
  Key x = mine > rising ? mine : rising;
#pragma unroll 1
  for (int j = 16; j > 0; j >>= 1) {
    const Key y = __shfl_xor_sync(kAll, x, j);
    x = (x > y) == ((lane & j) == 0) ? x : y;
  }
  return x;
}

// The same with the others in any order: a bitonic sort ahead of it.
__device__ __forceinline__ Key merge_lanes(Key mine, Key other) {
  const int lane = threadIdx.x & 31;
  Key x = other;
#pragma unroll 1
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      const Key y = __shfl_xor_sync(kAll, x, j);
      const bool smaller = ((lane & k & 31) == 0) == ((lane & j) == 0);
      x = (x < y) == smaller ? x : y;
    }
  return merge_sorted(mine, x);
}

__device__ __forceinline__ float largest(const float (&x)[kEach]) {
  float m = fmaxf(x[0], x[1]);
#pragma unroll
  for (int j = 2; j < kEach; j += 2) m = max3f(m, x[j], x[j + 1]);
  return m;
}

// What the warps of a CTA on one row know of it, as ordered values by warp; 0: nothing yet.
struct Known {
  uint32_t* wth;  // W of the warp's values reach it
  uint32_t* kth;  // k of them do
  int warps, k;   // warps * k >= W: so W values of the row reach the least of these
};

// A warp's piece [begin, end) of a row: its W best, in order, a lane to each (0: none), and
// its maximum and sum.  me: the warp among those of its row.
template <typename T, bool VEC, bool FEW>
__device__ __forceinline__ Key scan(const T* row, int begin, int end, int eos, int W,
                                    uint8_t* ring, Known known, int me, float2& max_sum) {
  using P = Piece<T, VEC>;
  const int lane = threadIdx.x & 31;
  P p;
  p.ring = ring;
  p.lead = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(row + begin) & 15);
  p.from = row + begin - p.lead / (int)sizeof(T);
  p.bytes = begin < end ? p.lead + (end - begin) * (int)sizeof(T) : 0;
#pragma unroll 1
  for (int i = 0; i < P::kSlots; ++i) p.request(i);
  Key mine = 0;
  float m = -INFINITY, l = 0.f;
  float t = -FLT_MAX;  // values from it on are candidates (-inf and NaN never)
#pragma unroll 1
  for (int i = 0, base = begin; base < end; ++i, base += kChunk) {
    copy_wait<P::kSlots - 1>();
    __syncwarp();
    float x[kEach];
    p.get(i, base, end, x);
    __syncwarp();
    p.request(i + P::kSlots);  // (into the room of this chunk, which all lanes have read)
    float mt = largest(x);
    if (mt > m) {
      l *= ex2_approx((m - mt) * kLog2e);  // (m = -inf: l is 0)
      m = mt;
    }
    // (From the maximum first: a product of its own would round, or overflow, before.)
    const float ref = m == -INFINITY ? 0.f : -m;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < kEach; j += 2) {
      float a, b;
      add_f32x2(a, b, x[j], x[j + 1], ref, ref);
      mul_f32x2(a, b, a, b, kLog2e, kLog2e);
      add_f32x2(s0, s1, s0, s1, ex2_approx(a), ex2_approx(b));
    }
    l += s0 + s1;
    if ((unsigned)(eos - base) < (unsigned)kChunk) {  // the end is no candidate
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (P::index(base, j) == eos) x[j] = -INFINITY;
      mt = largest(x);
    }
    if (!__any_sync(kAll, mt >= t)) continue;
    const bool other = lane < known.warps;
    const uint32_t least =
        __reduce_min_sync(kAll, other ? *(volatile uint32_t*)(known.kth + lane) : ~0u);
    uint32_t reached =
        max(__reduce_max_sync(kAll, other ? *(volatile uint32_t*)(known.wth + lane) : 0u), least);
    uint32_t hits;  // of the lane's values, those that reach t
#pragma unroll 1
    for (;;) {
      t = fmaxf(t, unordered(max(reached, ordered(-FLT_MAX))));
      hits = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) hits |= x[j] >= t ? 1u << j : 0u;
      if (FEW ? __reduce_add_sync(kAll, (unsigned)__popc(hits)) <= kMany
              : __popc(__ballot_sync(kAll, hits != 0)) <= kManyLanes)
        break;
      if constexpr (FEW) {
        // The lanes' maxima, largest first: W values reach the W-th.  (A lane whose values do
        // not reach t, or are all NaN, has none.)
        uint32_t o = mt >= t ? ordered(mt) : 0;
#pragma unroll 1
        for (int j = 0; j < W; ++j) {
          reached = __reduce_max_sync(kAll, o);
          if (lane == __ffs(__ballot_sync(kAll, o == reached)) - 1) o = 0;
        }
        // Equal ones: all of them.  So are those of fewer than W lanes, whose W-th is 0, a NaN.
        // (Every other turn raises t, and to what it finds again: the second is the last.)
        if (!(unordered(reached) > t)) break;
      } else {
        // The lanes' maxima into the list at once.
        int at = 0;
#pragma unroll
        for (int j = kEach - 1; j >= 0; --j) at = x[j] == mt ? j : at;
        const Key key = mt >= t ? key_of(mt, P::index(base, at)) : 0;
        if (!__any_sync(kAll, key > __shfl_sync(kAll, mine, W - 1))) {
          hits = 0;  // (equal ones, behind those that are held)
          break;
        }
        mine = merge_lanes(mine, key);
#pragma unroll
        for (int j = 0; j < kEach; ++j) x[j] = j == at ? -INFINITY : x[j];
        mt = largest(x);
        reached = (uint32_t)(__shfl_sync(kAll, mine, W - 1) >> 32);
      }
    }
#pragma unroll 1
    for (unsigned mask; (mask = __ballot_sync(kAll, hits != 0)) != 0;) {
      const int j = hits != 0 ? __ffs(hits) - 1 : 0;
      const Key key = key_of(pick(x, j), P::index(base, j));
      hits &= hits - 1;
#pragma unroll 1
      for (; mask != 0; mask &= mask - 1) {
        const Key k = __shfl_sync(kAll, key, __ffs(mask) - 1);
        const int above = __popc(__ballot_sync(kAll, mine > k));
        const Key up = __shfl_up_sync(kAll, mine, 1);
        mine = lane < above ? mine : lane == above ? k : up;
      }
    }
    const uint32_t value = (uint32_t)(mine >> 32);
    if (lane == known.k - 1) known.kth[me] = value;
    if (lane == W - 1) known.wth[me] = value;
    // (an equal value of a later chunk comes too late)
    const uint32_t last = __shfl_sync(kAll, value, W - 1);
    if (last != 0) t = fmaxf(t, unordered(last + 1));
  }
  copy_wait<0>();
  const float M = unordered(__reduce_max_sync(kAll, ordered(m)));
  max_sum = make_float2(M, add_up(l, m, M));
  return lane < W ? mine : 0;
}

// log x of a sum, x >= 1, to 2^-25: e log 2 + log f, x = 2^e f with f in [1 / sqrt 2,
// sqrt 2), so that fp32's half steps are those of a number below 0.35.
__device__ __forceinline__ double log_of(float x) {
  const uint32_t u = __float_as_uint(x);
  int e = (int)(u >> 23) - 127;
  float f = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
  if (f >= 1.41421356f) {
    f *= 0.5f;
    ++e;
  }
  return e * 0.69314718055994531 + (double)logf(f);
}

// a / b, rounded down, of small numbers, b > 0 (the quotient's error is far below 0.5 / b).
__device__ __forceinline__ int small_div(int a, int b) {
  return (int)__fdividef((float)a + 0.5f, (float)b);
}

// The 32 best of two lists of candidates, (value, beam and place), over the lanes, the second
// one the other way round: the better of every two, a bitonic merge.
__device__ __forceinline__ void merge_best(Key& c, uint32_t& id, Key other, uint32_t other_id) {
  const int lane = threadIdx.x & 31;
  auto ahead = [](Key a, uint32_t i, Key b, uint32_t j) { return a > b || (a == b && i < j); };
  if (ahead(other, other_id, c, id)) {
    c = other;
    id = other_id;
  }
#pragma unroll 1
  for (int j = 16; j > 0; j >>= 1) {
    const Key y = __shfl_xor_sync(kAll, c, j);
    const uint32_t yi = __shfl_xor_sync(kAll, id, j);
    if (ahead(c, id, y, yi) != ((lane & j) == 0)) {
      c = y;
      id = yi;
    }
  }
}

// What is chosen from the beams' best keys, top [W][W], and the logarithms of their sums; a
// lane of the first warp has its beam's score and the logit of its end.  cand: room for
// kCand keys; all threads of a CTA, a barrier ahead of it.  Few beams' lists by W rounds of a
// maximum over their heads, more of them by merges: a warp's two, then four warps' each, then
// all (32 beams 8,600 cycles in rounds).
constexpr int kCand = kWarps * 32 * 3 / 2;
template <bool FEW>
__device__ __forceinline__ void choose(const BeamSelectArgs& a, int b, uint32_t alive,
                                       const Key* top, Key* cand, const double* s_lse,
                                       const float* s_score, float score, float end_x) {
  const int W = a.W, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool here = alive >> lane & 1;
  // ---- candidates (0: none; what a finite number is ordered as is not)
  auto candidate = [&](int w) -> Key {
    const double lse = s_lse[w];
    const Key k = lane < W && (alive >> w & 1) ? top[w * W + lane] : 0;
    return k != 0 && lse > -INFINITY
               ? ordered((double)s_score[w] + ((double)value_of(k) - lse) + 0.0)
               : 0;
  };
  Key my_c = 0, my_key = 0, last_c = 0, last_key = 0;  // of place `lane`; of the last place
  int my_beam = lane, last_beam = 0;
  if constexpr (FEW) {
    if (warp < W) {
      const Key c = candidate(warp);
      if (lane < W) cand[warp * W + lane] = c;
    }
    __syncthreads();
    if (warp > 0) return;
    // ---- the choice: lane i holds the next candidate of beam i
    int at = lane * W;
    Key c = here ? cand[at] : 0, k = here ? top[at] : 0;
#pragma unroll 1
    for (int j = 0; j < W; ++j) {
      const Key best = warp_max(c);
      last_c = best;
      if (best == 0) break;
      last_beam = __ffs(__ballot_sync(kAll, c == best)) - 1;
      last_key = __shfl_sync(kAll, k, last_beam);
      if (lane == j) {
        my_c = best;
        my_beam = last_beam;
        my_key = last_key;
      }
      if (lane == last_beam) {
        ++at;
        c = at < (lane + 1) * W ? cand[at] : 0;
        k = at < (lane + 1) * W ? top[at] : 0;
      }
    }
  } else {
    uint32_t* ids = reinterpret_cast<uint32_t*>(cand + kWarps * 32);
    const int lists = min(W, kWarps);
    uint32_t id = warp << 5 | lane;
    if (warp < lists) {
      my_c = candidate(warp);
      if (warp + kWarps < W) {
        const Key c = candidate(warp + kWarps);
        merge_best(my_c, id, __shfl_xor_sync(kAll, c, 31), (warp + kWarps) << 5 | (31 - lane));
      }
      cand[warp * 32 + lane] = my_c;
      ids[warp * 32 + lane] = id;
    }
    __syncthreads();
#pragma unroll 1
    for (int step = 1; step < kWarps; step *= 4) {  // lists `step` apart, four to a warp
      const int first = warp * 4 * step;
      if (first < lists) {
        my_c = cand[first * 32 + lane];
        id = ids[first * 32 + lane];
#pragma unroll 1
        for (int i = 1; i < 4 && first + i * step < lists; ++i) {
          const int from = (first + i * step) * 32 + 31 - lane;
          merge_best(my_c, id, cand[from], ids[from]);
        }
        cand[first * 32 + lane] = my_c;
        ids[first * 32 + lane] = id;
      }
      __syncthreads();
    }
    if (warp > 0) return;
    if (my_c != 0) {
      my_beam = (int)(id >> 5);
      my_key = top[my_beam * W + (id & 31)];
    }
    last_c = __shfl_sync(kAll, my_c, W - 1);
    last_key = __shfl_sync(kAll, my_key, W - 1);
    last_beam = __shfl_sync(kAll, my_beam, W - 1);
  }
  if (lane >= W) return;
  const int o = b * W + lane;
  a.tokens[o] = my_key != 0 ? index_of(my_key) : a.pad;
  a.parents[o] = my_beam;
  a.new_scores[o] = my_c != 0 ? (float)unordered(my_c) : -INFINITY;
  // Ends that are better than the last one chosen.
  float ended = -INFINITY;
  const double lse = here ? s_lse[lane] : -INFINITY;
  if (lse > -INFINITY && end_x > -INFINITY) {
    const double e = (double)score + ((double)end_x - lse) + 0.0;
    const Key eo = ordered(e);
    const bool ahead = last_c != 0 && lane == last_beam
                           ? key_of(end_x, a.eos) > last_key
                           : eo > last_c || (eo == last_c && lane < last_beam);
    if (ahead) ended = (float)e;
  }
  a.ended[o] = ended;
}

// A cluster to a request, or to a group of its rows.
template <typename T, bool VEC, bool FEW>
__global__ void __launch_bounds__(32 * kWarps, 1) beam_select_kernel(const BeamSelectArgs a) {
  extern __shared__ __align__(16) uint8_t s_dyn[];  // the warps' rings, then what is merged
  __shared__ uint32_t s_wth[kWarps], s_kth[kWarps];
  __shared__ double s_lse[32];
  __shared__ float s_score[32];
  const int ranks = a.ranks, cluster = blockIdx.x / ranks, rank = blockIdx.x - cluster * ranks;
  const int b = cluster / a.groups, group = cluster - b * a.groups, W = a.W;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (ranks > 1) cluster_arrive();  // (nobody stores to a CTA that has not begun)
  if (lane == 0) s_wth[warp] = s_kth[warp] = 0;
  pdl_wait();
  pdl_launch_dependents();
  // A beam whose score is not finite is not there.
  const float score = lane < W ? a.scores[b * W + lane] : -INFINITY;
  bool here = isfinite(score);
  uint32_t alive = __ballot_sync(kAll, here);
  // Rows of a cluster, at most: the pieces go by these, so that all rows of a request are cut
  // alike and equal ones have equal sums.
  int most = __popc(alive);
  if (a.groups > 1) {  // every groups-th of them
    most = small_div(most + a.groups - 1, a.groups);
    const int nth = __popc(alive & ((1u << lane) - 1));
    here = here && nth % a.groups == group;
    alive = __ballot_sync(kAll, here);
  }
  const int rows = __popc(alive);
  // What the choice needs of the beams, a lane to each.
  float end_x = -INFINITY;
  if (rank == 0 && warp == 0) {
    s_score[lane] = score;
    if (here && a.eos >= 0)
      end_x = to_float<T>(
          static_cast<const T*>(a.logits)[(long long)(b * W + lane) * a.row_stride + a.eos]);
  }
  // The beam of the i-th live row.
  const int nth = __popc(alive & ((1u << lane) - 1));
  auto live_beam = [&](int i) { return __ffs(__ballot_sync(kAll, here && nth == i)) - 1; };
  // Pieces of a row, multiples of 16 values, the last ones may be empty.
  const int pieces = min(kMaxPieces, small_div(ranks * kWarps, max(most, 1)));
  const int length = ((int)(__fdividef((float)a.V, (float)pieces) * 1.000001f) + 16) & ~15;
  // What is merged, in the first CTA: per list, [row][piece], its keys, maximum and sum;
  // per beam its best keys and what they are as candidates.
  Key* keys = reinterpret_cast<Key*>(s_dyn + kWarps * kRing);
  float2* mls = reinterpret_cast<float2*>(keys + ranks * kWarps * W);
  Key* top = reinterpret_cast<Key*>(mls + ranks * kWarps);
  Key* cand = reinterpret_cast<Key*>(s_dyn);  // (over the rings)
  __syncthreads();
  // A row's pieces go to neighbouring warps, which share thresholds.
  const int per = small_div(rows * pieces + ranks - 1, ranks), task = rank * per + warp;
  const bool work = warp < per && task < rows * pieces;
  if (work) {
    const int r = small_div(task, pieces), w = live_beam(r);
    const int begin = (int)min((long long)(task - r * pieces) * length, (long long)a.V);
    const int end = (int)min((long long)begin + length, (long long)a.V);
    const T* x = static_cast<const T*>(a.logits) + (long long)(b * W + w) * a.row_stride;
    // The row's warps of this CTA (its pieces may begin or go on in a neighbour).
    const int first = max(r * pieces - rank * per, 0);
    const int n = min((r + 1) * pieces - rank * per, per) - first;
    const Known known = {&s_wth[first], &s_kth[first], n, small_div(W + n - 1, n)};
    float2 ml;
    const Key mine = scan<T, VEC, FEW>(x, begin, end, a.eos, W, s_dyn + warp * kRing, known,
                                  warp - first, ml);
    if (ranks > 1) cluster_wait();
    if (lane < W) store_cluster(keys + task * W + lane, 0, mine);
    if (lane == 0) store_cluster(mls + task, 0, ml);
  } else if (ranks > 1) {
    cluster_wait();
  }
  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank > 0) return;
  } else {
    __syncthreads();
  }
  // ---- the first CTA: by row a warp for the keys and one for the sum
#pragma unroll 1
  for (int i = warp; i < 2 * rows; i += kWarps) {
    const bool sums = i >= rows;
    const int r = sums ? i - rows : i, w = live_beam(r);
    if (sums) {
      float2 v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v[e] = lane + 32 * e < pieces ? mls[r * pieces + lane + 32 * e]
                                      : make_float2(-INFINITY, 0.f);
      const float M = unordered(__reduce_max_sync(kAll, ordered(fmaxf(v[0].x, v[1].x))));
      float l = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (v[e].y != 0.f) l += v[e].y * ex2_approx((v[e].x - M) * kLog2e);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(kAll, l, d);
      // Nothing allowed (a sum of 0) gives no candidate; NaN or +inf among the logits neither.
      if (isnan(l) && lane == 0) flag_status(a.status, PA_DEV_BAD_LOGITS);
      if (lane == 0) s_lse[w] = l > 0.f ? (double)M + log_of(l) : -INFINITY;
    } else if (const Key* mine = keys + r * pieces * W; !FEW && pieces < W) {
      // One after the other.
      Key kept = lane < W ? mine[lane] : 0;
#pragma unroll 1
      for (int p = 1; p < pieces; ++p)
        kept = merge_sorted(kept, 31 - lane < W ? mine[p * W + 31 - lane] : 0);
      if (lane < W) top[w * W + lane] = kept;
    } else {
      // Rounds of the largest head of the row's lists, two to a lane.
      int at[2] = {lane * W, (lane + 32) * W};
      Key head[2], kept = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) head[e] = lane + 32 * e < pieces ? mine[at[e]] : 0;
#pragma unroll 1
      for (int j = 0; j < W; ++j) {
        const Key k = warp_max(max(head[0], head[1]));
        if (lane == j) kept = k;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (k != 0 && head[e] == k) {
            ++at[e];
            head[e] = at[e] < (lane + 32 * e + 1) * W ? mine[at[e]] : 0;
          }
      }
      if (lane < W) top[w * W + lane] = kept;
    }
  }
  __syncthreads();
  if (a.groups > 1) {  // to be chosen from when all groups are done
#pragma unroll 1
    for (int i = warp; i < rows; i += kWarps) {
      const int w = live_beam(i);
      if (lane < W) a.ws_top[(size_t)(b * W + w) * W + lane] = top[w * W + lane];
      if (lane == 0) a.ws_lse[b * W + w] = s_lse[w];
    }
    return;
  }
  choose<FEW>(a, b, alive, top, cand, s_lse, s_score, score, end_x);
}

// The choice where the rows of a request were shared out among several clusters.
template <typename T, bool FEW>
__global__ void __launch_bounds__(32 * kWarps) beam_choose_kernel(const BeamSelectArgs a) {
  __shared__ Key s_top[kMaxBeams * kMaxBeams], s_cand[kCand];
  __shared__ double s_lse[32];
  __shared__ float s_score[32];
  const int b = blockIdx.x, W = a.W, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const float score = lane < W ? a.scores[b * W + lane] : -INFINITY;
  const bool here = isfinite(score);
  const uint32_t alive = __ballot_sync(kAll, here);
  float end_x = -INFINITY;
  if (warp == 0) {
    s_score[lane] = score;
    s_lse[lane] = here ? a.ws_lse[b * W + lane] : -INFINITY;
    if (here && a.eos >= 0)
      end_x = to_float<T>(
          static_cast<const T*>(a.logits)[(long long)(b * W + lane) * a.row_stride + a.eos]);
  }
#pragma unroll 1
  for (int w = warp; w < W; w += kWarps)
    if (lane < W && (alive >> w & 1))
      s_top[w * W + lane] = a.ws_top[(size_t)(b * W + w) * W + lane];
  __syncthreads();
  choose<FEW>(a, b, alive, s_top, s_cand, s_lse, s_score, score, end_x);
}

int dynamic_bytes(int W, int ranks) {
  return kWarps * kRing + ranks * kWarps * (W + 1) * 8 + W * W * 8;
}

template <typename T, bool VEC, bool FEW>
cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t stream) {
  constexpr auto kern = beam_select_kernel<T, VEC, FEW>;
  const int smem = dynamic_bytes(a.W, a.ranks);
  cudaError_t e = ensure_dynamic_smem<kern>(dynamic_bytes(kMaxBeams, kMaxCluster));
  if (e != cudaSuccess) return e;
  if (a.ranks > 8) {
    e = ensure_large_cluster<kern>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ranks * a.groups * a.B);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)a.ranks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.ranks > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || a.groups == 1) return e;
  cfg.gridDim = dim3(a.B);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_choose_kernel<T, FEW>, a);
}

template <typename T>
cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 &&
                   (a.B * a.W == 1 || a.row_stride * (int)sizeof(T) % 16 == 0);
  if (a.W <= kFewBeams)
    return vec ? launch_t<T, true, true>(a, stream) : launch_t<T, false, true>(a, stream);
  return vec ? launch_t<T, true, false>(a, stream) : launch_t<T, false, false>(a, stream);
}

}  // namespace

int clusters_at_once(int ranks) {
  static std::atomic<int> cached[64][kMaxCluster + 1];
  const int nsm = sm_count() > 0 ? sm_count() : 152;
  int dev = 0, n = 0;
  if (ranks == 1) return nsm;
  const bool slot = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
  if (slot && (n = cached[dev][ranks].load(std::memory_order_relaxed)) > 0) return n - 1;
  constexpr auto kern = beam_select_kernel<float, true, true>;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)ranks, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = dynamic_bytes(kMaxBeams, ranks);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!slot || ensure_dynamic_smem<kern>(dynamic_bytes(kMaxBeams, kMaxCluster)) != cudaSuccess ||
      ensure_large_cluster<kern>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return ranks > 8 ? 0 : nsm / ranks;
  }
  cached[dev][ranks].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Clusters of a request (its rows are shared out among these, and chosen from in a second
// launch, if there are several) and their CTAs: those with the least time.  That is, in units
// of 0.05 us, by what was measured: for every time that the GPU is filled with clusters, the
// chunks of a warp (the more warps an SM has, the longer) and what comes before and after
// them, which grows with the beams; and the second launch.  What it chooses is within 8 % of
// the best of up to 25 others over 40 sizes (one request of one beam and 32,000 logits to 80
// of 16 x 128,000).  Against the largest cluster a request with an SM to each CTA: one
// request of 32 x 260,000 fp32 logits 48 -> 24 us (32 clusters of 4), one of 16 x 256,000
// 28 -> 17.2, 8 of 32 x 260,000 74 -> 56.6, 16 of these 150 (two fills) -> 95; 80 requests
// of 16 x 128,000 bf16, more than half of the SMs, 119 -> 108 (clusters of 3, two fills).
void beam_select_shape(int B, int W, int V, int* groups, int* ranks) {
  const long long chunks = (V - 1) / kChunk + 1;  // of a row
  const int around = 9 * W < 100 + 5 * W / 2 ? 70 + 9 * W : 170 + 5 * W / 2;
  long long least = LLONG_MAX;
  *groups = 1;
  *ranks = W > kWarps ? 2 : 1;
  for (int r = 1; r <= kMaxCluster; r = r == 8 ? kMaxCluster : r + 1) {
    const int fit = clusters_at_once(r);
    if (fit == 0) continue;
    for (int several = 0; several < 2; ++several) {
      int g = several ? fit / B : 1;
      if (several && (g < 2 || W < 2)) break;
      const int rows = (W + g - 1) / g;
      g = (W + rows - 1) / rows;
      if (rows > r * kWarps) continue;  // (a warp to a row)
      int pieces = r * kWarps / rows;
      if (pieces > kMaxPieces) pieces = kMaxPieces;
      const long long fills = ((long long)B * g - 1) / fit + 1;
      const int warps = (rows * pieces - 1) / r + 1;  // of a CTA
      const long long time =
          fills * (around + 5 * rows / 2 + (10 + warps) * ((chunks - 1) / pieces + 1) / 2) +
          (fills - 1) * 60 + (g > 1 ? 40 : 0);
      if (time < least) {
        least = time;
        *groups = g;
        *ranks = r;
      }
    }
  }
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t stream) {
  return a.dtype == PA_F32    ? launch_t<float>(a, stream)
         : a.dtype == PA_BF16 ? launch_t<__nv_bfloat16>(a, stream)
                              : launch_t<__half>(a, stream);
}

}  // namespace pk
