// rope_write.cu -- rotary positions with up to four axes, fused with the write
// of the rotated keys and of the values into the paged cache.
//
// Pair i of a head's first R dims turns by angle = position[axis(i)][t] *
// inv_freq(i):  (x, y) -> (x cos - y sin, y cos + x sin); the pair is
// (x_i, x_{i + R/2}) in the split layout, (x_2i, x_{2i+1}) in the interleaved
// one; dims R .. D-1 pass unchanged.  Queries go to q_out, keys to k_out and to
// the cache slot of their token, values to the slot.
//
// The angle: a table entry holds F = inv_freq / 2 pi as a 64-bit binary
// fraction of a turn, and position * F modulo 2^64 (one integer product, which
// drops whole turns exactly, for negative positions too) is the fraction of a
// turn that remains.  Its top 32 bits go to fp32: at most 2^-26 of a turn off,
// at any 32-bit position, where position * inv_freq in fp32 is off by
// position * 2^-25 radians.  F itself is off by 2^-62 at most (its two low bits
// carry the axis), 2^-31 of a turn at position 2^31.  Sines and products are
// fp32; one rounding at the end.
//
// Bound: HBM for long prompts ((2H + 4 Hkv [+ Hkv if k_out]) * D * 2 bytes a
// token, each read or written once), launch latency for single tokens.  The sines
// of a CTA's tokens are computed once, by all its threads, into shared memory and
// serve all H + Hkv heads; each thread's first rows are loaded before the barrier,
// so that loads and sines overlap.  Measured: 16,001 tokens, 32 heads on 8, three
// axes, bf16: 68.2 us, 6.25 TB/s, 0.93 of the measured copy rate (one token to a
// CTA: 92 us, half of the time at the barrier behind too few sines); 38 tokens, 40
// heads on 8: 2.3 us.
#include <cuda_bf16.h>

#include "pk_common.cuh"
#include "pk_grouped.h"

namespace pk {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kItems = 2;  // items a thread has in flight

__device__ __forceinline__ float2 to_f2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
__device__ __forceinline__ float2 to_f2(uint32_t w, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t from_f2(float x, float y, __half) {
  __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t from_f2(float x, float y, __nv_bfloat16) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Eight pairs in the split layout: their x in lo, their y in hi.
template <typename T>
__device__ __forceinline__ void turn_split(uint4& lo, uint4& hi, const float2* cs) {
  uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = to_f2(l[i], T()), y = to_f2(h[i], T());
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    l[i] = from_f2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y, T());
    h[i] = from_f2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y, T());
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
}

// Four interleaved pairs.
template <typename T>
__device__ __forceinline__ void turn_pairs(uint4& v, const float2* cs) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = to_f2(w[i], T()), c = cs[i];
    w[i] = from_f2(p.x * c.x - p.y * c.y, p.y * c.x + p.x * c.y, T());
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

// TOK tokens to a CTA: their TOK * R / 2 sines are computed by all threads at once,
// behind the first loads; then each thread keeps its 16-dim column of a head and
// walks the TOK * rows head rows of the tokens (queries, keys, values).
template <typename T, int D, bool IL, int TOK>
__global__ void __launch_bounds__(kRopeThreads, TOK == 1 ? 1 : 5)
    rope_write_kernel(const RopeArgs a) {
  constexpr int IPH = D / 16;                      // items of a head row
  constexpr int STEP = kRopeThreads / IPH;         // head rows of a pass
  __shared__ float2 cs[TOK][D / 2];
  __shared__ long long s_slot[TOK];
  const int tid = threadIdx.x, c = tid % IPH;
  const int half = a.R / 2;
  // The item's two chunks of a row, 8 c and D / 2 + 8 c: neighbouring threads take
  // neighbouring chunks, so a load or store is whole lines.  In the split layout
  // they are the two halves of eight pairs if R is D; with a smaller R the columns
  // below R / 16 take 8 c and R / 2 + 8 c, the others 16 of the dims past R.
  const bool turned = c < a.R / 16;
  const int e0 = IL || a.R == D ? 8 * c : turned ? 8 * c : 16 * c;
  const int e1 = IL || a.R == D ? D / 2 + 8 * c : turned ? a.R / 2 + 8 * c : 16 * c + 8;
  const int rows = a.H + a.Hkv + (a.k_cache != nullptr ? a.Hkv : 0);
  const int t0 = blockIdx.x * TOK, toks = min(TOK, a.T - t0);
  const int n_rows = toks * rows, step = STEP * gridDim.y;
  pdl_wait();
  pdl_launch_dependents();

  // Where this thread stands: token tk, head row hr (it advances by step).
  int tk = 0, hr = blockIdx.y * STEP + tid / IPH, at = hr;
  auto settle = [&]() {
    while (hr >= rows && tk < TOK) {
      hr -= rows;
      ++tk;
    }
  };
  settle();
  uint4 lo[kItems], hi[kItems];
  auto load = [&]() {  // the next kItems items, from a copy of the place
    int ltk = tk, lhr = hr, lat = at;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (lat < n_rows) {
        const int t = t0 + ltk;
        const T* src;
        if (lhr < a.H) {
          src = static_cast<const T*>(a.q) + t * a.q_stride + lhr * D;
        } else if (lhr < a.H + a.Hkv) {
          src = static_cast<const T*>(a.k) + t * a.k_stride + (lhr - a.H) * D;
        } else {
          src = static_cast<const T*>(a.v) + t * a.v_stride + (lhr - a.H - a.Hkv) * D;
        }
        lo[j] = load_stream(src + e0);
        hi[j] = load_stream(src + e1);
      }
      lat += step;
      lhr += step;
      while (lhr >= rows && ltk < TOK) {
        lhr -= rows;
        ++ltk;
      }
    }
  };
  load();
  if (tid < toks) {
    long long slot = a.k_cache != nullptr ? a.slots[t0 + tid] : -1;
    if (slot >= a.n_slots) {
      if (blockIdx.y == 0) flag_status(a.status, PA_DEV_BAD_SLOT);
      slot = -1;
    }
    s_slot[tid] = slot;
  }
  for (int i = tid; i < toks * half; i += kRopeThreads) {
    const int k = i / half, p = i - k * half;
    const unsigned long long f = a.table[p];
    const int axis = min((int)(f & 3), a.n_axes - 1);
    const long long pos = a.positions[(size_t)axis * a.T + t0 + k];
    const unsigned long long turn = (unsigned long long)pos * (f & ~3ull);
    // signed fraction of a turn in halves of a turn: the sine's argument is pi times it
    const float x = (float)(int)(turn >> 32) * 0x1p-31f;
    float s, co;
    sincospif(x, &s, &co);
    cs[k][p] = make_float2(co, s);
  }
  __syncthreads();
  while (at < n_rows) {
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (at < n_rows) {
        const int t = t0 + tk;
        const long long slot = s_slot[tk];
        const bool is_q = hr < a.H, is_v = hr >= a.H + a.Hkv;
        if (!is_v) {
          if constexpr (IL) {
            if (e0 < a.R) turn_pairs<T>(lo[j], cs[tk] + e0 / 2);
            if (e1 < a.R) turn_pairs<T>(hi[j], cs[tk] + e1 / 2);
          } else if (turned) {
            turn_split<T>(lo[j], hi[j], cs[tk] + 8 * c);
          }
        }
        T* dst = is_q ? static_cast<T*>(a.q_out) + t * a.q_out_stride + hr * D
                 : !is_v && a.k_out != nullptr
                     ? static_cast<T*>(a.k_out) + t * a.k_out_stride + (hr - a.H) * D
                     : nullptr;
        if (dst != nullptr) {
          *reinterpret_cast<uint4*>(dst + e0) = lo[j];
          *reinterpret_cast<uint4*>(dst + e1) = hi[j];
        }
        if (!is_q && slot >= 0) {
          const int h = is_v ? hr - a.H - a.Hkv : hr - a.H;
          T* row = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + ((size_t)slot * a.Hkv + h) * D;
          *reinterpret_cast<uint4*>(row + e0) = lo[j];
          *reinterpret_cast<uint4*>(row + e1) = hi[j];
        }
      }
      at += step;
      hr += step;
      settle();
    }
    if (at < n_rows) load();
  }
}

template <typename T, int D, int TOK>
cudaError_t launch_tok(const RopeArgs& a, int gy, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + TOK - 1) / TOK, gy);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.interleaved ? cudaLaunchKernelEx(&cfg, rope_write_kernel<T, D, true, TOK>, a)
                       : cudaLaunchKernelEx(&cfg, rope_write_kernel<T, D, false, TOK>, a);
}

template <typename T, int D>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t stream) {
  // Few tokens: one to a CTA, or spread over as many as give each thread one item.
  const int rows = a.H + a.Hkv + (a.k_cache != nullptr ? a.Hkv : 0);
  constexpr int kPass = kRopeThreads / (D / 16);
  if (a.T <= 2 * sm_count()) return launch_tok<T, D, 1>(a, (rows + kPass - 1) / kPass, stream);
  // Two tokens to a CTA at D = 128, four at 64 (40 head rows: 2,000 tokens 12.8 us
  // with two, 14.0 with one, 12.9 with four; at 64 7.3 us with one, 4.1 with four).
  return launch_tok<T, D, 256 / D>(a, 1, stream);
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, cudaStream_t stream) {
  if (a.bf16)
    return a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, stream)
                      : launch_t<__nv_bfloat16, 64>(a, stream);
  return a.D == 128 ? launch_t<__half, 128>(a, stream) : launch_t<__half, 64>(a, stream);
}

}  // namespace pk
