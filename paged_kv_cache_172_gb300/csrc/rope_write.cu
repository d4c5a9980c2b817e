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
// token, each read or written once), launch latency for single tokens.  One
// CTA takes one token: its R/2 sines and cosines are computed once into shared
// memory and serve all H + Hkv heads, and a work item is two 16-byte chunks (the
// two halves of eight pairs).  Each thread's first items are loaded before the
// barrier, so that loads and sines overlap.
#include <cuda_bf16.h>

#include "pk_common.cuh"
#include "pk_internal.h"

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

// Eight pairs: the split layout has their x in lo and their y in hi; the
// interleaved one has pairs 0-3 in lo and 4-7 in hi.
template <typename T, bool IL>
__device__ __forceinline__ void turn8(uint4& lo, uint4& hi, const float2* cs) {
  uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (IL) {
      const float2 a = to_f2(l[i], T()), b = to_f2(h[i], T());
      const float2 ca = cs[i], cb = cs[4 + i];
      l[i] = from_f2(a.x * ca.x - a.y * ca.y, a.y * ca.x + a.x * ca.y, T());
      h[i] = from_f2(b.x * cb.x - b.y * cb.y, b.y * cb.x + b.x * cb.y, T());
    } else {
      const float2 x = to_f2(l[i], T()), y = to_f2(h[i], T());
      const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
      l[i] = from_f2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y, T());
      h[i] = from_f2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y, T());
    }
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
}

template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs a) {
  constexpr int IPH = D / 16;  // items of a head
  __shared__ float2 cs[D / 2];
  const int tid = threadIdx.x;
  const int half = a.R / 2, turned = a.R / 16;
  const int n_items = (a.H + a.Hkv + (a.k_cache != nullptr ? a.Hkv : 0)) * IPH;
  const int first = blockIdx.y * kRopeThreads + tid, step = gridDim.y * kRopeThreads;
  pdl_wait();
  pdl_launch_dependents();

  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    // Item -> its source row, dims of its two chunks, head and kind (0 q, 1 k, 2 v).
    auto place = [&](int item, const T*& src, int& d0, int& d1, int& head, int& kind) {
      int r = item / IPH;
      const int c = item % IPH;
      kind = r < a.H ? 0 : r < a.H + a.Hkv ? 1 : 2;
      head = kind == 0 ? r : kind == 1 ? r - a.H : r - a.H - a.Hkv;
      const T* base = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
      const long long stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
      src = base + t * stride + head * D;
      if (!IL && kind < 2 && c < turned) {
        d0 = 8 * c;
        d1 = half + 8 * c;
      } else {  // interleaved pairs, dims past R, values: 16 dims in a row
        d0 = 16 * c;
        d1 = d0 + 8;
      }
    };
    const T* src[kItems];
    int d0[kItems], d1[kItems], head[kItems], kind[kItems];
    uint4 lo[kItems], hi[kItems];
    auto load = [&](int base) {
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int item = base + j * step;
        if (item < n_items) {
          place(item, src[j], d0[j], d1[j], head[j], kind[j]);
          lo[j] = load_stream(src[j] + d0[j]);
          hi[j] = load_stream(src[j] + d1[j]);
        }
      }
    };
    load(first);
    long long slot = a.k_cache != nullptr ? a.slots[t] : -1;
    if (slot >= a.n_slots) {
      if (tid == 0 && blockIdx.y == 0) flag_status(a.status, PA_DEV_BAD_SLOT);
      slot = -1;
    }
    for (int i = tid; i < half; i += kRopeThreads) {
      const unsigned long long f = a.table[i];
      const int axis = min((int)(f & 3), a.n_axes - 1);
      const long long pos = a.positions[(size_t)axis * a.T + t];
      const unsigned long long turn = (unsigned long long)pos * (f & ~3ull);
      // signed fraction of a turn in halves of a turn: the sine's argument is pi times it
      const float x = (float)(int)(turn >> 32) * 0x1p-31f;
      float s, c;
      sincospif(x, &s, &c);
      cs[i] = make_float2(c, s);
    }
    __syncthreads();
    for (int base = first; base < n_items; base += kItems * step) {
      if (base != first) load(base);
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int item = base + j * step;
        if (item >= n_items) continue;
        const int c = item % IPH;
        if (kind[j] < 2 && c < turned) turn8<T, IL>(lo[j], hi[j], cs + 8 * c);
        if (kind[j] == 0 || (kind[j] == 1 && a.k_out != nullptr)) {
          T* dst = kind[j] == 0 ? static_cast<T*>(a.q_out) + t * a.q_out_stride
                                : static_cast<T*>(a.k_out) + t * a.k_out_stride;
          dst += head[j] * D;
          *reinterpret_cast<uint4*>(dst + d0[j]) = lo[j];
          *reinterpret_cast<uint4*>(dst + d1[j]) = hi[j];
        }
        if (kind[j] > 0 && slot >= 0) {
          T* dst = static_cast<T*>(kind[j] == 1 ? a.k_cache : a.v_cache) +
                   ((size_t)slot * a.Hkv + head[j]) * D;
          *reinterpret_cast<uint4*>(dst + d0[j]) = lo[j];
          *reinterpret_cast<uint4*>(dst + d1[j]) = hi[j];
        }
      }
    }
    __syncthreads();  // the sines are free for the next token
  }
}

template <typename T, int D>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t stream) {
  const int n_items = (a.H + a.Hkv + (a.k_cache != nullptr ? a.Hkv : 0)) * (D / 16);
  cudaLaunchConfig_t cfg = {};
  // Few tokens: spread a token's items over as many CTAs as give each thread one.
  const int rounds = (n_items + kRopeThreads - 1) / kRopeThreads;
  const int gy = a.T <= 2 * sm_count() ? rounds : 1;
  cfg.gridDim = dim3(a.T, gy);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.interleaved ? cudaLaunchKernelEx(&cfg, rope_write_kernel<T, D, true>, a)
                       : cudaLaunchKernelEx(&cfg, rope_write_kernel<T, D, false>, a);
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, cudaStream_t stream) {
  if (a.bf16)
    return a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, stream)
                      : launch_t<__nv_bfloat16, 64>(a, stream);
  return a.D == 128 ? launch_t<__half, 128>(a, stream) : launch_t<__half, 64>(a, stream);
}

}  // namespace pk
