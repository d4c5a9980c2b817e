// grouped_decode.cu -- decode attention with grouped K/V heads over the paged
// cache: one query token per sequence, G = H / Hkv query heads reading the same
// K/V head, fp16 or bf16.
//
//     s_jg = scale * q_g . k_j,  out_g = sum_j 2^(..) v_j / sum_j 2^(..)
//
// Bound: HBM.  A K and a V row of D values serve G heads, so the work per byte
// is G times that of one head per K/V head: 2 G multiply-adds a byte, too much
// for scalar arithmetic at 8 TB/s beyond two or three heads, and far too little
// to fill the tcgen05 tiles of 128 rows.  Warp MMAs (m16n8k16) sit between:
// with the keys as the 16 rows and the heads as the 8 columns,
//     S^T [16 keys x 8 heads] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16] P^T,
// a group of up to 8 heads wastes no rows on padding to 16 (two column tiles
// serve up to 16 heads, more heads take more CTAs), K is the row operand as it
// lies in the cache, V^T comes from transposing ldmatrix loads, and the
// accumulators of S^T become the column operand of the second product by one
// 8 x 8 transposition in registers (movmatrix).
//
// One CTA takes one partition of a sequence's keys for one K/V head; its four
// warps take every fourth stage of 16 keys, each through its own ring of TMA
// boxes (K and V, 8 KB a stage at D = 128), with its own running maximum and
// sums, and merge through shared memory at the end.  Three CTAs share an SM
// (66 KB of shared memory each), 192 KB of loads in flight; neighbouring CTAs
// read the heads of the same tokens, so that 256-byte rows of one head add up to
// whole DRAM pages (one wave of warps with equal, contiguous pieces, which reads
// different tokens for different heads, took 47.5 us for the 38-sequence batch
// where this grid took 36.6).  Partitions of a longer context merge by
// log-sum-exp: as a cluster through each other's shared memory while the whole
// grid fits at once, otherwise through the workspace in a second, dependent
// launch.
//
// Measured (GB300): 4 x 60-131 thousand keys, 64 heads on 8, bf16: 250 us, 6.76
// TB/s of keys and values, 1.01 of the measured copy rate; 38 sequences of
// 128-2,048 keys, 40 on 8, fp16: 33.5 us, 5.2 TB/s (the start, the last CTAs and
// the merge are 8 us of it); one of 1,000 keys, 32 on 8: 5.3 us, of which a launch
// and four trips to memory are all.
//
// Cross attention with few queries (CROSS): the beams of a request are further heads of its
// groups, so its states come from memory once for up to 16 (query, head) pairs, as boxes of
// 16 consecutive rows.  One request of 4 beams on 1,500 states, 16 heads, D = 64, fp16: 6.3
// us; 32 of 4 on 200-1,500: 22.8 us, 4.5 TB/s (start, last CTAs and the merge's launch: 7 us
// around the traffic); 4 of 4 on 30,000-65,536, 32 on 8, D = 128, bf16: 141 us, 6.3 TB/s,
// 0.93 of the copy rate.
//
// Rounding: scores, maxima, sums and outputs in fp32; the weights 2^(s - m) <= 1
// enter the second product as a high and a low half in the cache's type, so that they
// keep 16 bits and more, as pa_decode's do, and the result is rounded once.  (One
// rounded weight would be off by as much as the result's own rounding; the halves cost
// 1 to 3 % in ragged batches, 5 % where 64 sequences of 1,500 keys fill every SM alike,
// and up to 14 % with two column tiles at D = 64.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "pk_common.cuh"
#include "pk_grouped.h"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;   // keys of a stage
constexpr int kRing = 2;    // stages in flight per warp
constexpr int kSpan = kWarps * kKeys;   // keys the CTA takes a round
constexpr int kMaxPart = 32 * kSpan;    // a warp's table entries sit one per lane
constexpr int kMaxCluster = 8;          // partitions that merge in a cluster, at most

// A stage's atoms (8 keys x 64 dims, 1 KB): paged, by key group and then by half, as blocks'
// boxes land; rows of another array (CROSS), by half and then by key group.
template <int D, bool CROSS = false>
struct DCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int GROUP = CROSS ? 1024 : HALVES * 1024;  // to the next 8 keys
  static constexpr int HALF = CROSS ? 2048 : 1024;            // from dims 0-63 to dims 64-127
  static constexpr int TILE = HALVES * 2048;                  // K (or V) of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int RING_BYTES = kWarps * kRing * STAGE;
};

// Shared memory: the rings (reused for the merge of the warps), then per warp
// and head (m, l), then the barriers.
template <int D, int NT>
constexpr int merge_bytes() { return kWarps * NT * 8 * D * 4; }
template <int D, int NT>
constexpr int smem_bytes() {
  const int ring = DCfg<D>::RING_BYTES, mrg = merge_bytes<D, NT>();
  return (ring > mrg ? ring : mrg) + kWarps * NT * 8 * 8 + kWarps * kRing * 8 + 1024;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Two weights 0 <= x, y <= 1, times kRaise, as 16-bit pairs hi + lo: hi cut off and lo
// the rest, rounded, so within 2^-15 (bf16) or 2^-21 (fp16) of the weight.  fp16 is raised
// to where its smallest step, 2^-24, is 2^-39 of the largest weight: in steps of 2^-24 of
// it many small weights beside it would be lost.  lo is above 0 where hi is, so that an
// infinite value times a weight is infinite and not NaN.
template <typename T>
constexpr float kRaise = std::is_same<T, __half>::value ? 32768.f : 1.f;
template <typename T>
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (std::is_same<T, __half>::value) {
    x *= kRaise<T>;
    y *= kRaise<T>;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack<T>(fmaxf(x - h.x, h.x > 0.f ? 0x1p-24f : 0.f),
                 fmaxf(y - h.y, h.y > 0.f ? 0x1p-24f : 0.f));
  } else {
    const uint32_t hx = __float_as_uint(x) & 0xffff0000u, hy = __float_as_uint(y) & 0xffff0000u;
    hi = __byte_perm(hx, hy, 0x7632);
    lo = pack<T>(fmaxf(x - __uint_as_float(hx), x * 0x1p-24f),
                 fmaxf(y - __uint_as_float(hy), y * 0x1p-24f));
  }
}

template <typename T>
__device__ __forceinline__ T round_to(float x) {
  if constexpr (std::is_same<T, __half>::value)
    return __float2half_rn(x);
  else
    return __float2bfloat16_rn(x);
}

// NT column tiles of 8 heads; grid (Hkv * head chunks, B, partitions).  CL: the
// partitions of a sequence are one cluster and merge through each other's shared
// memory; otherwise through the workspace.  CROSS: the columns are a request's
// (query, head) pairs, ql * G of them, and its keys are consecutive rows.
template <typename T, int D, int NT, bool CL, bool CROSS>
__global__ void __launch_bounds__(kThreads)
    grouped_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const GroupedDecodeArgs a) {
  using C = DCfg<D, CROSS>;
  constexpr int HEADS = NT * 8;
  constexpr int KS = D / 16;  // 16-dim steps of either product
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t raw = smem_u32(smem_dyn);
  uint8_t* smem = smem_dyn + (((raw + 1023u) & ~1023u) - raw);
  constexpr int kRoom =
      C::RING_BYTES > merge_bytes<D, NT>() ? C::RING_BYTES : merge_bytes<D, NT>();
  float* s_o = reinterpret_cast<float*>(smem);                  // [warp][head][D], after the rings
  float2* s_ml = reinterpret_cast<float2*>(smem + kRoom);       // [warp][head]
  // A cluster's partition result, behind the warps' (CL): [head][D], then [head]
  float* s_part = s_o + kWarps * HEADS * D;
  float2* s_pml = reinterpret_cast<float2*>(s_part + HEADS * D);
  static_assert(!CL || merge_bytes<D, NT>() + HEADS * (D * 4 + 8) <= kRoom, "cluster merge room");
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRoom + kWarps * HEADS * 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = ((CROSS ? a.max_q : 1) * a.G + HEADS - 1) / HEADS;
  const int hkv = blockIdx.x / chunks, g0 = (blockIdx.x % chunks) * HEADS;
  const int b = blockIdx.y, part = blockIdx.z;
  int heads = min(HEADS, a.G - g0);  // live columns
  int q0 = b;                        // first query of the sequence
  // The row of column g of this CTA among all (query, head) pairs.
  auto row_at = [&](int g) {
    if (!CROSS) return (size_t)b * a.H + hkv * a.G + g0 + g;
    const int tok = (g0 + g) / a.G;
    return (size_t)(q0 + tok) * a.H + hkv * a.G + (g0 + g - tok * a.G);
  };
  uint64_t* bar = bars + warp * kRing;

  if (lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    for (int s = 0; s < kRing; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  // The table entries of this warp's stages, one stage to a lane, are fetched
  // with the length and not behind it: the row is there whatever the length, and
  // a CTA's start is two trips to memory instead of three.
  const int bs = a.block_size, k0 = part * a.part_tokens;
  const int my_key = k0 + (warp + kWarps * lane) * kKeys;
  const int32_t* row_of = CROSS ? nullptr : a.block_tables + (size_t)b * a.max_blocks;
  int ent_lo = 0, ent_hi = 0;
  if (!CROSS && (warp + kWarps * lane) * kKeys < a.part_tokens) {
    const int blk = my_key / bs;
    if (blk < a.max_blocks) ent_lo = row_of[blk];
    if (bs < kKeys && blk + 1 < a.max_blocks) ent_hi = row_of[blk + 1];
  }
  int n = a.context_lens[b], kv0 = 0;
  bool bad = n < 0 || n > a.max_context;
  if constexpr (CROSS) {
    q0 = a.q_offsets[b];
    kv0 = a.kv_starts[b];
    const int end = a.q_offsets[b + 1];
    const bool lost = q0 < 0 || end < q0 || end > a.T;  // its rows do not exist
    const int ql = lost ? 0 : end - q0;
    bad = ql > a.max_q || ((bad || kv0 < 0 || (long long)kv0 + n > a.Tk) && ql > 0);
    if ((bad || lost) && threadIdx.x == 0 && part == 0)
      flag_status(a.status, PA_DEV_BAD_CONTEXT);
    if (bad) n = 0;
    if ((long long)ql * a.G <= g0) return;
    // (columns past the last chunk's: of a bad request, whose rows are zeros)
    heads = bad && g0 / HEADS == chunks - 1 ? ql * a.G - g0 : min(HEADS, ql * a.G - g0);
  } else if (bad) {
    if (threadIdx.x == 0 && part == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
    n = n < 0 ? 0 : a.max_context;
  }
  if (k0 >= n) {
    if (part == 0)  // an empty context: zero rows
      for (long long i = threadIdx.x; i < (long long)heads * D; i += kThreads)
        static_cast<T*>(a.out)[row_at((int)(i / D)) * D + i % D] = round_to<T>(0.f);
    return;
  }
  const int k1 = min(n, k0 + a.part_tokens);
  const bool alone = n <= a.part_tokens;  // the only partition of its sequence
  // This warp's stages: keys k0 + (warp + 4 i) * 16 ...
  const int n_st = (k1 - k0 + kKeys - 1) / kKeys;
  const int mine = n_st > warp ? (n_st - warp + kWarps - 1) / kWarps : 0;

  // Lane i holds the pool row of the first slot of the warp's i-th stage, and
  // for 8-token blocks that of its second half.
  int row_lo = 0, row_hi = 0;
  if (!CROSS && lane < mine) {
    auto pool_row = [&](int key, int phys) {
      if (key >= n) return a.num_blocks * bs * a.Hkv;  // past the sequence: outside the map
      if (phys < 0 || phys >= a.num_blocks) {
        flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
        phys = a.num_blocks;
      }
      return phys * bs * a.Hkv;
    };
    row_lo = pool_row(my_key, ent_lo);
    if (bs < kKeys) row_hi = pool_row(my_key + 8, ent_hi);
  }
  __syncwarp();

  uint8_t* ring = smem + warp * kRing * C::STAGE;
  auto request = [&](int i) {
    if constexpr (CROSS) {  // 16 rows of one head; rows past the array read as zeros
      if (elect_one()) {
        uint8_t* st = ring + (i % kRing) * C::STAGE;
        uint64_t* full = &bar[i % kRing];
        const int row = kv0 + k0 + (warp + kWarps * i) * kKeys;
        mbar_arrive_expect_tx(full, C::STAGE);
        tma_load_4d(st, &kmap, 0, row, 0, hkv, full);
        tma_load_4d(st + C::TILE, &vmap, 0, row, 0, hkv, full);
      }
      return;
    }
    const int lo = __shfl_sync(kAll, row_lo, i), hi = __shfl_sync(kAll, row_hi, i);
    if (elect_one()) {
      uint8_t* st = ring + (i % kRing) * C::STAGE;
      uint64_t* full = &bar[i % kRing];
      mbar_arrive_expect_tx(full, C::STAGE);
      if (bs >= kKeys) {  // a box of two key groups, from the stage's place in the block
        const int grp = ((k0 + (warp + kWarps * i) * kKeys) % bs) / 8;
        tma_load_5d(st, &kmap, 0, 0, 0, grp, lo + hkv, full);
        tma_load_5d(st + C::TILE, &vmap, 0, 0, 0, grp, lo + hkv, full);
      } else {  // two blocks of one key group
        tma_load_5d(st, &kmap, 0, 0, 0, 0, lo + hkv, full);
        tma_load_5d(st + C::GROUP, &kmap, 0, 0, 0, 0, hi + hkv, full);
        tma_load_5d(st + C::TILE, &vmap, 0, 0, 0, 0, lo + hkv, full);
        tma_load_5d(st + C::TILE + C::GROUP, &vmap, 0, 0, 0, 0, hi + hkv, full);
      }
    }
  };
  for (int i = 0; i < kRing && i < mine; ++i) request(i);

  // Q^T as the column operand: lane holds head lane / 4, dims 2 (lane % 4) + {0, 1}
  // and those + 8 of each 16-dim step.
  const int col = lane >> 2, two = 2 * (lane & 3);
  uint32_t qf[NT][KS][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int g = t * 8 + col;
    const T* qr = static_cast<const T*>(a.q) + two;
    if (CROSS) {
      const int tok = (g0 + g) / a.G;
      if (g < heads)
        qr += (size_t)(q0 + tok) * a.q_stride + (size_t)(hkv * a.G + g0 + g - tok * a.G) * D;
    } else {
      qr += row_at(g) * D;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[t][ks][e] =
            g < heads ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8 * e) : 0u;
  }

  float o[NT][KS][4];  // O^T: dims lane / 4 (+ 8), heads two, two + 1
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) o[t][ks][0] = o[t][ks][1] = o[t][ks][2] = o[t][ks][3] = 0.f;
  float m[NT][2], l[NT][2];  // heads two, two + 1; l: this lane's keys only
#pragma unroll
  for (int t = 0; t < NT; ++t) m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
  const float sl2 = a.scale_log2;
  const int mi = lane >> 3, rr = lane & 7;  // ldmatrix: matrix and row of this lane
  bool ok = true;
  int done = 0;
  for (; done < mine; ++done) {
    if (!__all_sync(kAll, mbar_wait(&bar[done % kRing], (done / kRing) & 1))) {
      ok = false;
      break;
    }
    uint8_t* st = ring + (done % kRing) * C::STAGE;
    const uint32_t kb = smem_u32(st), vb = kb + C::TILE;
    const int key0 = k0 + (warp + kWarps * done) * kKeys;
    const int live = k1 - key0;  // keys of this stage, if below 16
    if (live < kKeys) {
      // V rows past the keys hold anything, and 0 * NaN is NaN: zero them.
      for (int i = lane; i < (kKeys - live) * (D / 8); i += 32) {
        const int r = live + i / (D / 8), c = i % (D / 8);
        *reinterpret_cast<uint4*>(st + C::TILE + (r >> 3) * C::GROUP + (c >> 3) * C::HALF +
                                  (r & 7) * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    // 16-byte chunk c of key r: chunk c ^ (r & 7) of the row in its swizzled atom
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int c = 2 * ks + (mi >> 1);
      uint32_t kf[4];  // keys 0-7 / 8-15 (mi & 1), dims 0-7 / 8-15 (mi >> 1)
      ldsm4(kb + (mi & 1) * C::GROUP + (c >> 3) * C::HALF + rr * 128 + (((c & 7) ^ rr) << 4), kf);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma<T>(s[t], kf, qf[t][ks][0], qf[t][ks][1]);
    }
    uint32_t pf[NT][2][2];  // high, low halves
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // scaled before they are masked: any finite scale, 0 and below included
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] *= sl2;
      if (live < kKeys) {
        if (col >= live) s[t][0] = s[t][1] = -INFINITY;
        if (col + 8 >= live) s[t][2] = s[t][3] = -INFINITY;
      }
      float p[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[t][e], s[t][2 + e]);
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
        const float m_new = fmaxf(m[t][e], mx);
        // Scores of -inf alone so far (infinite keys): -inf + inf is NaN, so their
        // weights, all zero, are taken with maximum 0.
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(m[t][e] - ref);
        m[t][e] = m_new;
        p[e] = ex2_approx(s[t][e] - ref);
        p[2 + e] = ex2_approx(s[t][2 + e] - ref);
        l[t][e] = l[t][e] * alpha + (p[e] + p[2 + e]);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          o[t][ks][e] *= alpha;
          o[t][ks][2 + e] *= alpha;
        }
      }
      split<T>(p[0], p[1], pf[t][0][0], pf[t][1][0]);
      split<T>(p[2], p[3], pf[t][0][1], pf[t][1][1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // two heads of key lane / 4 (+ 8): now two keys of a head
        pf[t][0][e] = transpose8(pf[t][0][e]);
        pf[t][1][e] = transpose8(pf[t][1][e]);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int c = 2 * ks + (mi & 1);
      uint32_t vf[4];  // dims 0-7 / 8-15 (mi & 1), keys 0-7 / 8-15 (mi >> 1), transposed
      ldsm4_t(vb + (mi >> 1) * C::GROUP + (c >> 3) * C::HALF + rr * 128 + (((c & 7) ^ rr) << 4), vf);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma<T>(o[t][ks], vf, pf[t][0][0], pf[t][0][1]);
        mma<T>(o[t][ks], vf, pf[t][1][0], pf[t][1][1]);
      }
    }
    __syncwarp();
    if (done + kRing < mine) {
      if (elect_one()) fence_proxy_async_smem();  // this stage's reads before its refill
      request(done + kRing);
    }
  }
  if (!ok) {
    if (lane == 0) flag_status(a.status, PA_DEV_TIMEOUT);
    for (int i = done; i < mine && i < done + kRing; ++i)
      mbar_wait(&bar[i % kRing], (i / kRing) & 1);
  }
  // Sums over the lanes that share a head.
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[t][e];
      x += __shfl_xor_sync(kAll, x, 4);
      x += __shfl_xor_sync(kAll, x, 8);
      x += __shfl_xor_sync(kAll, x, 16);
      l[t][e] = x;
    }
  __syncthreads();  // every warp's stages are read: their room takes the outputs
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g = t * 8 + two + e;
      float* dst = s_o + ((size_t)warp * HEADS + g) * D + col;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        dst[ks * 16] = o[t][ks][e] * (1.f / kRaise<T>);
        dst[ks * 16 + 8] = o[t][ks][2 + e] * (1.f / kRaise<T>);
      }
      if (col == 0) s_ml[warp * HEADS + g] = make_float2(m[t][e], l[t][e]);
    }
  }
  __syncthreads();
  // Thread: one dim pair of every (kThreads / (D / 2))-th head.
  constexpr int kPairs = D / 2, kStep = kThreads / kPairs;
  const int d = 2 * (threadIdx.x % kPairs);
  for (int g = threadIdx.x / kPairs; g < heads; g += kStep) {
    float2 ml[kWarps];
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = s_ml[w * HEADS + g];
      if (ml[w].y != 0.f) M = fmaxf(M, ml[w].x);
    }
    float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (ml[w].y == 0.f) continue;  // a warp without stages
      const float wgt = ex2_approx(ml[w].x - M);
      const float2 v = *reinterpret_cast<const float2*>(s_o + ((size_t)w * HEADS + g) * D + d);
      L += wgt * ml[w].y;
      x += wgt * v.x;
      y += wgt * v.y;
    }
    const size_t row = row_at(g);
    if (alone) {
      const float inv = L != 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D + d) =
          pack<T>(x * inv, y * inv);
    } else if constexpr (CL) {
      *reinterpret_cast<float2*>(s_part + g * D + d) = make_float2(x, y);
      if (d == 0) s_pml[g] = make_float2(M, L);
    } else {
      const size_t pr = row * a.num_parts + part;
      *reinterpret_cast<float2*>(a.ws_o + pr * D + d) = make_float2(x, y);
      if (d == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * pr) = make_float2(M, L);
    }
  }
  if constexpr (CL) {
    if (alone) return;
    // The CTAs with keys (the others of the cluster have left, which its barrier
    // allows for) share out the (head, dim pair)s and merge them by log-sum-exp.
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int live = (n + a.part_tokens - 1) / a.part_tokens;
    cluster.sync();
    for (int i = part * kThreads + threadIdx.x; i < heads * kPairs; i += live * kThreads) {
      const int g = i / kPairs, dd = 2 * (i % kPairs);
      float2 ml[kMaxCluster], v[kMaxCluster];
      float M = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p) {
        ml[p] = make_float2(-INFINITY, 0.f);
        if (p < live) {
          ml[p] = *cluster.map_shared_rank(s_pml + g, p);
          v[p] = *cluster.map_shared_rank(reinterpret_cast<float2*>(s_part + g * D + dd), p);
        }
        if (ml[p].y != 0.f) M = fmaxf(M, ml[p].x);
      }
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p) {
        if (ml[p].y == 0.f) continue;
        const float wgt = ex2_approx(ml[p].x - M);
        L += wgt * ml[p].y;
        x += wgt * v[p].x;
        y += wgt * v[p].y;
      }
      const float inv = L != 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row_at(g) * D + dd) =
          pack<T>(x * inv, y * inv);
    }
    cluster.sync();  // nobody leaves while another reads its shared memory
  }
}

// Merges the partitions of a (sequence, head), CROSS of a (query, head) whose request is
// blockIdx.y: W warps take every W-th one.
template <typename T, int D, int W, bool CROSS>
__global__ void __launch_bounds__(32 * W) grouped_decode_merge(const GroupedDecodeArgs a) {
  constexpr int EPL = D / 32;
  __shared__ float s_o[W][D];
  __shared__ float2 s_ml[W];
  size_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The lengths come from before the first kernel, which let this one start only when
  // all its blocks had waited for them: they are read while it still runs.
  int n = a.context_lens[CROSS ? blockIdx.y : row / a.H];
  if constexpr (CROSS) {
    const int q0 = a.q_offsets[blockIdx.y], end = a.q_offsets[blockIdx.y + 1];
    const int kv0 = a.kv_starts[blockIdx.y], tok = blockIdx.x / a.H;
    if (q0 < 0 || end < q0 || end > a.T || end - q0 > a.max_q || tok >= end - q0 ||
        n > a.max_context || kv0 < 0 || (long long)kv0 + n > a.Tk)
      n = 0;
    row += (size_t)q0 * a.H;
  } else {
    n = min(max(n, 0), a.max_context);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (n <= a.part_tokens) return;  // written by its only partition (or empty)
  const int parts = (n + a.part_tokens - 1) / a.part_tokens;
  float M = -INFINITY, L = 0.f, o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
  constexpr int kAhead = 4;  // partitions whose loads are in flight together
  for (int p0 = warp; p0 < parts; p0 += kAhead * W) {
    float2 ml[kAhead];
    float v[kAhead][EPL];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + k * W;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (p < parts) {
        const size_t pr = row * a.num_parts + p;
        ml[k] = *reinterpret_cast<const float2*>(a.ws_ml + 2 * pr);
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
          const float2 f = *reinterpret_cast<const float2*>(a.ws_o + pr * D + lane * EPL + e);
          v[k][e] = f.x, v[k][e + 1] = f.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (ml[k].y == 0.f) continue;
      const float m_new = fmaxf(M, ml[k].x);
      const float keep = ex2_approx(M - m_new), take = ex2_approx(ml[k].x - m_new);
      M = m_new;
      L = L * keep + ml[k].y * take;
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = o[e] * keep + v[k][e] * take;
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) s_o[warp][lane * EPL + e] = o[e];
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp > 0) return;
    float mx = M;
#pragma unroll
    for (int w = 1; w < W; ++w)
      if (s_ml[w].y != 0.f) mx = fmaxf(mx, s_ml[w].x);
    float keep = L != 0.f ? ex2_approx(M - mx) : 0.f;
    L *= keep;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= keep;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      if (s_ml[w].y == 0.f) continue;
      const float take = ex2_approx(s_ml[w].x - mx);
      L += s_ml[w].y * take;
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] += s_o[w][lane * EPL + e] * take;
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  T* dst = static_cast<T*>(a.out) + row * D + lane * EPL;
#pragma unroll
  for (int e = 0; e < EPL; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack<T>(o[e] * inv, o[e + 1] * inv);
}

template <typename T, int D, int NT, bool CROSS>
cudaError_t launch_t(const GroupedDecodeArgs& a, const void* k_cache, const void* v_cache,
                     cudaStream_t stream) {
  using C = DCfg<D, CROSS>;
  using u64 = unsigned long long;
  CUtensorMap kmap, vmap;
  cudaError_t e = cudaSuccess;
  if constexpr (CROSS) {
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
      const u64 dims[4] = {64, (u64)(a.Tk > 0 ? a.Tk : 1), (u64)C::HALVES, (u64)a.Hkv};
      const u64 st[3] = {(u64)(i ? a.v_stride : a.k_stride) * 2, 128, (u64)D * 2};
      const unsigned box[4] = {64, kKeys, (unsigned)C::HALVES, 1};
      e = make_map_4d(i ? &vmap : &kmap, i ? v_cache : k_cache, dims, st, box, true);
    }
  } else {
    // Rows (slot, head) of D values; inside a block (64 dims, 8 keys, halves, key
    // groups), at its first slot's row.
    const u64 rowb = (u64)D * 2, tok = rowb * a.Hkv;
    const u64 dims[5] = {64, 8, (u64)C::HALVES, (u64)a.block_size / 8,
                         (u64)a.num_blocks * a.block_size * a.Hkv};
    const u64 st[4] = {tok, 128, 8 * tok, rowb};
    const unsigned box[5] = {64, 8, (unsigned)C::HALVES, a.block_size >= kKeys ? 2u : 1u, 1};
    e = make_map_5d(&kmap, k_cache, dims, st, box, true);
    if (e == cudaSuccess) e = make_map_5d(&vmap, v_cache, dims, st, box, true);
  }
  if (e != cudaSuccess) return e;
  constexpr int smem = smem_bytes<D, NT>();
  cudaLaunchConfig_t cfg = {};
  const int cols = (CROSS ? a.max_q : 1) * a.G;  // of a sequence and a K/V head
  cfg.gridDim = dim3(a.Hkv * ((cols + 8 * NT - 1) / (8 * NT)), a.B, a.num_parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.num_parts > 1 && grouped_decode_in_cluster(a.B, cols * a.Hkv, a.Hkv, a.num_parts)) {
    constexpr auto kern = grouped_decode_kernel<T, D, NT, true, CROSS>;
    e = ensure_dynamic_smem<kern>(smem);
    if (e != cudaSuccess) return e;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {1, 1, (unsigned)a.num_parts};
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, a);
  }
  constexpr auto kern = grouped_decode_kernel<T, D, NT, false, CROSS>;
  e = ensure_dynamic_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kern, kmap, vmap, a);
  if (e != cudaSuccess || a.num_parts == 1) return e;
  cfg.gridDim = CROSS ? dim3(a.max_q * a.H, a.B) : dim3(a.B * a.H);
  cfg.dynamicSmemBytes = 0;
  if (a.num_parts <= 16) {
    cfg.blockDim = dim3(32);
    return cudaLaunchKernelEx(&cfg, grouped_decode_merge<T, D, 1, CROSS>, a);
  }
  cfg.blockDim = dim3(32 * 8);
  return cudaLaunchKernelEx(&cfg, grouped_decode_merge<T, D, 8, CROSS>, a);
}

}  // namespace

// Partition length where the caller leaves it open, 64 to 2,048 keys: the one of
// least cost, the cost in microseconds over the traffic itself being that of the
// last CTAs (0.0045 a key, 0.0052 with two column tiles, 0.0073 at D = 64, whose keys
// take the same round trips for half the bytes) and that of starting, ending and
// merging the grid's CTAs (4.5 for each round of them, three to an SM).  Fitted over
// sweeps of 81 batches, 4 % above the least on average, with weights of one rounding;
// now 38 ragged sequences of up to 2,048 tokens 33.4 us of 32.5 (40 heads on 2: 22.5 of
// 19.1), four of 60-131 thousand 244.6 of 244.4; furthest off where all sequences are
// alike and fill a round and a bit (64 x 1,500 with 64 heads on 4: 51.7 of 39.1), which
// for ragged ones is right (27.6 of 26.5).
// A single sequence is as long as it may be and seldom fills the GPU: its keys count
// more, its CTAs only past a quarter of those that run at once, and the merge with
// them (2,000 keys 6.5 -> 6.1 us, with 64 heads on 4 7.6 -> 6.4, at D = 64 5.9 -> 4.6
// with weights of one rounding; now 6.6, 6.8 and 4.9, the least 5.9, 6.8 and 4.9).
int grouped_decode_partition(int B, int H, int Hkv, int D, int max_context) {
  const int G = H / Hkv;
  const double pairs = (double)B * Hkv * (G <= 8 ? 1 : (G + 15) / 16);
  const int nsm = sm_count() > 0 ? sm_count() : 152;
  const double per_key = D == 64 ? 0.0073 : G > 8 ? 0.0052 : 0.0045, per_cta = 4.5 / (3.0 * nsm);
  // CTAs at once, as fitted (by shared memory; with two column tiles at D = 64 the
  // registers of the kernel without clusters leave room for four)
  const double slots = (D == 128 ? 3.0 : 6.0) * nsm;
  int best = kSpan;
  double least = 0.0;
  for (int p = kSpan; p <= kMaxPart; p += kSpan) {
    const int parts = (max_context + p - 1) / p;
    const double ctas = pairs * parts;
    double cost = per_key * p + per_cta * ctas;
    if (B == 1) {
      cost = 0.0075 * p * (ctas > slots ? 0.7 : 1.0) + ceil(ctas / slots);
      if (ctas > 0.25 * slots) cost += 6.0 * (ctas / slots - 0.25);
      if (parts > 1) cost += grouped_decode_in_cluster(B, H, Hkv, parts) ? 0.8 : 2.0;
    }
    if (p == kSpan || cost < least) {
      best = p;
      least = cost;
    }
    if (p >= max_context) break;
  }
  return best;
}

// Partitions that merge through shared memory need no second launch and no
// workspace, but a cluster starts only where all its CTAs fit at once, and holds
// them until the last is done: worth it while the whole grid does, with room to
// place the clusters (at most 2.6 CTAs an SM of the 3 it holds).  One sequence of
// 1,000 tokens 5.7 -> 5.0 us, eight of 2,000-4,000 in 384 CTAs 23.6 -> 22.2; past
// that 38 ragged sequences in 608 CTAs 33.1 -> 38.1 (weights of one rounding).
bool grouped_decode_in_cluster(int B, int H, int Hkv, long long parts) {
  const int G = H / Hkv, nsm = sm_count() > 0 ? sm_count() : 152;
  const double ctas = (double)B * Hkv * (G <= 8 ? 1 : (G + 15) / 16) * parts;
  return parts <= 1 || (parts <= kMaxCluster && ctas <= 2.6 * nsm);
}

cudaError_t launch_grouped_decode(const GroupedDecodeArgs& a, const void* k_cache,
                                  const void* v_cache, cudaStream_t stream) {
  const int cols = (a.kv_starts != nullptr ? a.max_q : 1) * a.G;
#define PK_GD(TT, DD)                                                               \
  (a.kv_starts != nullptr                                                           \
       ? (cols <= 8 ? launch_t<TT, DD, 1, true>(a, k_cache, v_cache, stream)        \
                    : launch_t<TT, DD, 2, true>(a, k_cache, v_cache, stream))       \
   : cols <= 8 ? launch_t<TT, DD, 1, false>(a, k_cache, v_cache, stream)            \
               : launch_t<TT, DD, 2, false>(a, k_cache, v_cache, stream))
  if (a.bf16) return a.D == 128 ? PK_GD(__nv_bfloat16, 128) : PK_GD(__nv_bfloat16, 64);
  return a.D == 128 ? PK_GD(__half, 128) : PK_GD(__half, 64);
#undef PK_GD
}

}  // namespace pk
