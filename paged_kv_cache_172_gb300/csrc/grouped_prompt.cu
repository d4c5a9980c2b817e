// grouped_prompt.cu -- causal attention of packed new tokens with grouped K/V
// heads on the sm_103a tensor cores (tcgen05, accumulators in tensor memory):
// whole prompts over their own K/V (contiguous rows) and chunks over a paged
// cache.  Without the mask, cross attention: queries over rows of another array.
//
// Query i of a sequence with ql new tokens and n keys sits at position
// n - ql + i and sees keys 0 .. n - ql + i (a prompt has n = ql):
//     out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * q_i . k_j - max).
//
// Tiles.  The G = H / Hkv query heads that share a K/V head go into one tile:
// its 128 rows are floor(128 / G) consecutive tokens x G heads, row r = token
// r / G, head r mod G (the order in which one TMA box of a packed [T, H, D]
// array lands).  A key tile then serves all heads of the group, and a chunk of
// a few tokens still fills rows instead of leaving a tile of 128 tokens to
// each head.  A CTA takes two such tiles A and B, one after the other in the
// sequence, of one K/V head, and walks the visible keys in tiles of 128:
//   warps 0-3, 4-7  softmax of tile A, B: one row per thread (TMEM lane = row);
//   warp 8          requests K_0, K_1, V_0, K_2, V_1, ... into a ring;
//   warp 9          issues S = Q K^T (one thread), owns the tensor memory;
//   warp 10         issues O += P V (one thread);
//   warp 11         schedules, and requests Q.
// Tensor memory: S [0, 128) shared by both tiles, P_A [128, 192), P_B
// [192, 256) as 16-bit pairs, O_A, O_B from column 256 (D columns each); cross attention
// at D = 64 has room for an S of each tile, [0, 256), and the others 128 further on.  Q
// stays in shared memory (A operand of the S products) and P in tensor memory
// (A operand of the P V products): the placement that asks least of the shared
// memory's bandwidth, as in the fp16 chunk kernel of this library.
//
// Scheduling.  One persistent CTA for each SM.  Lengths live on the device, so
// the host knows only a bound on the units of two tiles (T / tokens of a unit + B
// for each K/V head); warp 11 ranks them by the number of key tiles they read,
// longest first, deals them to the CTAs in rounds and posts each CTA's next two in
// shared memory.  The rank needs no sort: how many units of a sequence read at
// least t key tiles has a closed form, and a binary search over t with sums over
// the sequences finds the unit.  K/V loads run on into the next item, Q is
// requested tile by tile as the S products of the item before let go of it, and
// the output leaves through a slot of the K/V ring.  Few units with many keys:
// each is cut into up to `split` key ranges whose (o, m, l) rows go to the
// workspace and are merged by log-sum-exp.
//
// Cross attention.  All tiles of a request read all its keys, so that its units are alike;
// the keys' first row stands in for the position.  At D = 64, where two S and two O leave
// room, every tile's next S is computed while its softmax still works on the last one, and
// the softmax bounds the steady state: 2,000 cycles a pair of tiles, where its exponentials,
// sums and conversions are 1,196 of a scheduler's, the rest loads, stores and waits, and the
// four products 1,080 of the tensor core's.  8 encoder sequences of 500-4,096, 16 heads:
// 169 us, 1,060 TFLOP/s, 0.55 of the burst rate (one S region 180 us, P told in halves 178;
// the same at D = 128 takes 225).  Two threads to a row, 16 softmax warps, took 204 us, the
// next S loaded while P is stored 185: loads then wait for the products.  16 requests of
// 1-400 queries on 0-4,096 keys, 40 on 8, D = 128: 145 us, 1,160 TFLOP/s (0.60): S chain,
// start (10,000 cycles), three to four units a CTA of unequal length.
//
// Rounding: scores, maxima, sums and O are fp32; P is rounded to the 16-bit
// type of the inputs (the tensor core's operand; its values are at most 2^8
// before scaling, since O is rescaled only when the maximum grew by more than
// that; in fp16 times 2^6, so that many small weights are not lost below its
// smallest step), the result once more at the end.
//
// Bound: the tensor pipe by intensity; in the steady state the chain from one S
// product to the next through the one S region (2 x 1,320 cycles per pair of
// tiles, where four products take 2,048), and over long prompts the power cap.
// Besides that a unit costs about 4,000 cycles around its end (last P V product,
// output, next Q).  Measured (GB300, 32 heads on 8, D = 128, bf16), by call among
// many and so under the power cap: one prompt of 16,001 tokens 1,315 us, 1,595
// TFLOP/s, 0.82 of the measured burst rate and 0.91 of the sustained one; eight of
// 500-4,096 384 us, 1,312 TFLOP/s (0.68; 350 in a short run, at a clock that is
// higher by as much); chunks of 512 on 3,584 (40 on 8, fp16) 277 us, 1,163 TFLOP/s
// (0.60, 262 in a short run: 704 units on 152 SMs are five rounds where 4.6 would
// do, 125 rows of 128 are used, and with all keys in L2 they are 1.5 % quicker); 16
// chunks of 1-48 on up to 8,192 keys 70 us, 4.3 TB/s (bound by the chain above over
// 32 key tiles, not by HBM).  A
// launch reaches its first S product after 8,000 to 13,000 cycles: the search for
// the first unit and the code of every role run from a cold instruction cache.  A
// search looks at all sequences, past the first 32 in memory: 256 prompts of 1-60
// tokens 73 us, 1,000 416, 4,000 5,819.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "pk_common.cuh"
#include "pk_grouped.h"

namespace pk {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTile = 128;               // query rows of a tile, keys of a key tile
constexpr int kSlab = 128 * 128;         // 128 rows x 64 dims (128 bytes)
constexpr int kQRoom = 2 * kSlab;        // a Q tile's room, up to 128 dims
constexpr int kThreadsG = 384;           // 8 softmax warps, K/V loads, 2 MMA issuers, scheduler
constexpr int kWarpLoad = 8, kWarpS = 9, kWarpPv = 10, kWarpSched = 11;
constexpr int kItems = 3;                // items posted ahead
constexpr int kCols = 512;               // tensor memory columns
constexpr int kWindow = 256;             // block-table entries staged at a time
constexpr int kMaxRing = 8;
constexpr int kBars = 4 * kMaxRing + 14 + 2 * kItems + 1;
constexpr float kLazy = 8.0f;            // log2 of the growth that forces a rescale
// log2 of what weights are multiplied by (which the quotient drops): fp16 holds them in
// steps of 2^-24 at least, and 2^6 makes that 2^-30 of the largest.  (The largest is then
// 2^14, far enough below 2^16 for an exponent that rounding raises.)
template <typename T>
constexpr float kRaiseLog2 = std::is_same<T, __half>::value ? 6.0f : 0.0f;

// Where the keys are and who sees them: a prompt's own rows up to itself, the paged
// cache up to itself, or rows of another array, all of them.
enum Form { kPrompt, kChunk, kCross };

// Tensor memory: whether each tile has an S region of its own (where O leaves room), then
// the columns of S, P and O.
template <int D, Form F>
constexpr bool kOwnS = F == kCross && D == 64;
template <int D, Form F>
struct Col {
  static constexpr uint32_t S = 0, P = kOwnS<D, F> ? 256 : 128, O = P + kTile;
  static constexpr uint32_t nextS = kOwnS<D, F> ? kTile : 0;  // from tile A's S to tile B's
  static_assert(O + 2 * D <= kCols, "tensor memory");
};

// Layout of a K or V tile in shared memory.  Paged: key groups of 8 keys x D
// dims, each the 1 KB atoms of dims 0-63 and 64-127 (the order in which a
// block's box lands).  Contiguous rows: two slabs of 128 keys x 64 dims.
template <int D, bool PAGED>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int RING = D == 128 ? 5 : 8;
  static_assert(RING <= kMaxRing, "barriers");
  static constexpr int GROUP = PAGED ? 8 * D * 2 : 1024;  // 8 keys
  static constexpr int HALF = PAGED ? 1024 : kSlab;       // from dims 0-63 to dims 64-127
  static constexpr int OFF_KV = 2 * kQRoom;
  static constexpr int OFF_BAR = OFF_KV + RING * TILE_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + kBars * 8;  // TMEM address, stage counters, items
  static constexpr int OFF_TBL = (OFF_MISC + 16 + kMaxRing * 4 + kItems * 64 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_TBL + (PAGED ? kWindow * 4 : 0) + 1024;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Instruction descriptors: idesc_f16_f32 with the operand type (1: bf16).
template <typename T>
__host__ __device__ constexpr uint32_t operand_type() {
  return std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
}

// A sequence of the packed step, as every CTA sees it.
struct Seq {
  int start, ql, n;  // first packed row, new tokens, keys
  int kv;            // kCross: first row of its keys
  int nu;            // units
  bool bad;          // its rows are zeros
  bool lost;         // its rows do not exist: nothing to write
};

__device__ __forceinline__ int divide(int x, DivBy d) {
  return (int)(((unsigned long long)(unsigned)x * d.m) >> (31 + d.s));
}

template <Form F>
__device__ __forceinline__ Seq sequence(const GroupedArgs& a, int b) {
  Seq s;
  s.kv = 0;
  s.start = a.q_offsets[b];
  const int end = a.q_offsets[b + 1];
  s.ql = end - s.start;
  s.lost = s.start < 0 || end < s.start || end > a.T;
  if (s.lost) s.ql = 0;
  s.n = s.ql;
  s.bad = s.lost;
  if (F == kCross && s.ql > 0) {
    const int n = a.context_lens[b], kv = a.kv_starts[b];
    s.n = 0;
    if (s.ql > a.max_q || n < 0 || n > a.max_context || kv < 0 || (long long)kv + n > a.Tk) {
      s.bad = true;
    } else {
      s.n = n;
      s.kv = kv;
    }
  }
  if (F == kChunk && s.ql > 0) {
    const int n = a.context_lens[b];
    if (n < s.ql || n > a.max_context)
      s.bad = true;
    else
      s.n = n;
  }
  s.nu = divide(s.ql + a.span - 1, a.by_span);
  return s;
}

// Key tiles that unit i (tokens i * span .. ) of a sequence reads (at least one, so that
// a unit without keys is found too and its rows are written).
template <Form F>
__device__ __forceinline__ int unit_tiles(const Seq& s, int span, int i) {
  if (F == kCross) return max(1, (int)((unsigned)(s.n + kTile - 1) / kTile));
  return (int)((unsigned)(s.n - s.ql + min((i + 1) * span, s.ql) + kTile - 1) / kTile);
}

// Units of a sequence that read at least t (>= 1) key tiles: the last ones.
template <Form F>
__device__ __forceinline__ int units_from(const GroupedArgs& a, const Seq& s, int t) {
  if (F == kCross) return t <= unit_tiles<F>(s, 0, 0) ? s.nu : 0;
  const int k = (t - 1) * kTile + 1;  // keys such a unit needs at least
  if (s.n < k) return 0;  // (an empty sequence too)
  const int over = k - (s.n - s.ql);  // its tokens needed at least
  const int first = over <= 0 ? 0 : divide(over - 1, a.by_span);
  return s.nu - min(first, s.nu - 1);
}

// Key ranges a unit of that many key tiles is cut into.
__device__ __forceinline__ int unit_parts(int tiles, int split) {
  return max(1, min(split, (int)((unsigned)tiles / kGroupedMinPartTiles)));
}

// Walks the units by key tiles, longest first (one warp, all lanes alike).
template <Form F>
struct Units {
  const GroupedArgs& a;
  Seq mine;          // the lane's among the first 32 sequences, read once
  int bound, above;  // no unit asked for later reads `bound` key tiles or more; how many do
  int tiles, base0, before;  // where the last scan ended: sequences from base0, units before

  __device__ Units(const GroupedArgs& args)
      : a(args), bound(args.max_tiles + 1), above(0), tiles(0), base0(0), before(0) {
    const int lane = threadIdx.x & 31;
    mine = lane < a.B ? sequence<F>(a, lane) : Seq{0, 0, 0, 0, 0, true, true};
  }

  // Sequence b, the same for all lanes.
  __device__ Seq get(int b) const {
    if (b >= 32) return sequence<F>(a, b);
    Seq s;
    s.start = __shfl_sync(kAll, mine.start, b);
    s.ql = __shfl_sync(kAll, mine.ql, b);
    s.n = __shfl_sync(kAll, mine.n, b);
    s.kv = F == kCross ? __shfl_sync(kAll, mine.kv, b) : 0;
    s.nu = 0;  // (not asked for)
    s.bad = __shfl_sync(kAll, (int)mine.bad, b);
    s.lost = false;  // (a lost one has no units)
    return s;
  }

  // The unit of a rank: (b, i), or false behind the last unit.  Ranks rise from
  // call to call.
  __device__ bool find(int rank, int& b_out, int& i_out) {
    const int lane = threadIdx.x & 31;
    // units with >= lo tiles: more than rank (lo = 0: taken as such); >= hi: at most rank
    int lo = 0, hi = bound, over = above;
    // (A short loop: the first search of a launch runs from a cold instruction
    // cache, where a longer body cost more than the passes it saved.)
#pragma unroll 1
    while (hi - lo > 1) {
      const int t = (lo + hi) >> 1;
      int c = 0;
#pragma unroll 1
      for (int b = lane; b < a.B; b += 32) {
        Seq s = mine;
        if (b >= 32) s = sequence<F>(a, b);
        c += units_from<F>(a, s, t);
      }
      c = __reduce_add_sync(kAll, c);
      if (c > rank) {
        lo = t;
      } else {
        hi = t;
        over = c;
      }
    }
    bound = hi;
    above = over;
    if (lo == 0) return false;
    // The units that read exactly lo tiles, sequences in order: the (rank - over)-th.
    if (lo != tiles) {
      tiles = lo;
      base0 = before = 0;
    }
    int left = rank - over - before;
#pragma unroll 1
    for (int base = base0; base < a.B; base += 32) {
      const int b = base + lane;
      int c = 0, upper = 0, nu = 0;
      if (b < a.B) {
        Seq s = mine;
        if (b >= 32) s = sequence<F>(a, b);
        upper = units_from<F>(a, s, lo + 1);
        c = units_from<F>(a, s, lo) - upper;
        nu = s.nu;
      }
      int x = c;  // inclusive scan
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kAll, x, d);
        if (lane >= d) x += y;
      }
      const unsigned hit = __ballot_sync(kAll, x > left);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        base0 = base;
        before = rank - over - left;
        b_out = base + src;
        i_out = __shfl_sync(kAll, nu - 1 - upper - (left - (x - c)), src);
        return true;
      }
      left -= __shfl_sync(kAll, x, 31);
    }
    return false;
  }
};

// The registers of a thread: the softmax warps hold a row of S, the others next
// to nothing (128 * (2 * 200 + 104) = 384 * 168, what the block is launched with).
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
}
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
}

// A wait that is not on the chain of products: polled rarely.
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    __nanosleep(200);
    if (clock64() - t0 > kWaitLimitCycles) return false;
  }
  return true;
}

// Ring index of K_t and V_t among n_kv key tiles (K_0, then K_{t+1}, V_t).
__device__ __forceinline__ int ring_k(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int ring_v(int t, int n_kv) {
  return t + 1 < n_kv ? 2 * t + 2 : 2 * t + 1;
}

// Parts in the workspace.  Row r of a K/V head's packed rows (token r / G, head r
// mod G; a tile's rows are consecutive) has its D outputs as D / 4 groups of four,
// group c of all rows together: [part][Hkv][D / 4][T * G] float4, so that a warp's
// 32 rows store and load whole lines.  Behind them (max, normaliser) as
// [part][Hkv][T * G] float2.
__device__ __forceinline__ float2* part_ml(const GroupedArgs& a, int D, int part, int hkv) {
  const size_t plane = (size_t)a.T * a.G;
  return reinterpret_cast<float2*>(a.ws + (size_t)a.split * a.Hkv * plane * D) +
         (size_t)(part * a.Hkv + hkv) * plane;
}

// What the scheduler posts of a work item: a unit, or one of its key ranges.
static_assert(kThreadsG == 384, "register split");
struct Item {
  int valid;             // 0: no more items
  int row0, hkv;         // packed row of tile A's first token; K/V head
  int toks_a, toks_b;    // tokens of the tiles in this sequence
  int pos_a;             // position of tile A's first token; kCross: first row of the keys
  int kt0, n_kv;         // first key tile, key tiles
  int ntile_a, ntile_b;  // of those, the ones each tile reads
  int parts, part;
  int b, n;              // sequence and its keys
};

template <typename T, int D, Form F>
__global__ void __launch_bounds__(kThreadsG, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const GroupedArgs a) {
  constexpr bool PAGED = F == kChunk;
  using C = Cfg<D, PAGED>;
  constexpr int kRing = C::RING;
  constexpr uint32_t kColS = Col<D, F>::S, kColP = Col<D, F>::P, kColO = Col<D, F>::O;
  constexpr uint32_t kNextS = Col<D, F>::nextS;
  // P is handed over in halves for contiguous rows, so that its product with V starts
  // 64 keys early (one prompt of 8,192 353 -> 343 us); with the paged loader's code
  // beside it the longer loops cost more than that (16 x 2,048 keys 457 -> 470 us).
  constexpr int kHalves = PAGED ? 1 : 2;
  // With an S region to each tile the softmax is the longest chain, which the second
  // handing over lengthens: P is stored in halves there, but waited for and told once
  // (8 encoder sequences of 500-4,096, 16 heads, 177.3 -> 166.9 us; stored at once 169.2).
  constexpr bool kTold = kHalves > 1 && !kOwnS<D, F>;  // in halves
  constexpr float kRaise = kRaiseLog2<T>;
  constexpr uint32_t kIdS = tc::idesc_f16_f32(kTile, kTile, false, false) | operand_type<T>();
  constexpr uint32_t kIdO = tc::idesc_f16_f32(kTile, D, false, true) | operand_type<T>();
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t raw = smem_u32(smem_dyn);
  uint8_t* smem = smem_dyn + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  // The slots of the ring are given out in one order (K_0, K_1, V_0, ..., an item's
  // stage) and let go one by one, but what lands in them is told by kind, the i-th K,
  // V or stage at [i % ring]: whoever waits there takes every one of its kind in turn,
  // so a wait can never see the phase of two rounds before (of a slot that another
  // role has yet to wait for) and pass too early.
  uint64_t* k_full = bars;
  uint64_t* v_full = k_full + kRing;
  uint64_t* st_full = v_full + kRing;
  uint64_t* kv_empty = st_full + kRing;
  uint64_t* q_full = kv_empty + kRing;  // [2] per tile: Q of the item landed
  uint64_t* q_free = q_full + 2;        // [2]: the item's S products are done with it
  uint64_t* s_full = q_free + 2;        // [2]: an S product computed
  uint64_t* s_free = s_full + 2;        // [2]: its softmax holds S in registers
  uint64_t* p_half = s_free + 2;        // [2]: P of the first 64 keys stored
  uint64_t* p_full = p_half + 2;        // [2]: all of P stored
  uint64_t* pv_done = p_full + 2;       // [2]: O += P V completed
  uint64_t* it_full = pv_done + 2;      // [kItems]: an item is posted
  uint64_t* it_empty = it_full + kItems;  // [kItems]: every role has copied it
  uint64_t* drain = it_empty + kItems;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* stage_left = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);  // [ring] see the epilogue
  Item* items = reinterpret_cast<Item*>(smem + C::OFF_MISC + 16 + kMaxRing * 4);
  int32_t* tbl = reinterpret_cast<int32_t*>(smem + C::OFF_TBL);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = a.span / 2;  // tokens of a tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&st_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);  // one arrival per softmax warp
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int s = 0; s < kRing; ++s) stage_left[s] = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], kWarpSched);  // every other warp
    }
    mbar_init(drain, 2);
    fence_mbar_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == kWarpS) {
    tc::tmem_alloc(tmem_at, kCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  bool ok = true;
  int issued = 0, issued_v = 0;  // K tiles, or Q loads, requested; V tiles

  // The k-th item of this CTA, copied; the scheduler may then reuse its room.
  auto take = [&](int k, Item& it) {
    if (!(ok = __all_sync(kAll, mbar_wait(&it_full[k % kItems], (k / kItems) & 1)))) return false;
    it = items[k % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_empty[k % kItems]);
    return it.valid != 0;
  };

  if (warp < kWarpLoad) {
    // ------------------------------------------------------------ softmax
    reg_inc();
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int my_tok = (row * a.g_magic) >> 16;  // row / G
    const uint32_t t_lane = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + t_lane + kColS + x * kNextS, t_o = tmem + t_lane + kColO + x * D;
    const float sl2 = a.scale_log2;
    int done = 0;    // key tiles of the items before and of this one
    int u0 = 0;      // ring slots of the items before
    int stages = 0;  // of those, stages
    Item it;
    for (int k = 0; take(k, it); ++k) {
      const int pos0 = F == kCross ? it.n - 1 : it.pos_a + (x ? tpt : 0);
      const int ntile = x ? it.ntile_b : it.ntile_a;
      const bool live = my_tok < (x ? it.toks_b : it.toks_a);  // a row of this sequence
      const int pos = F == kCross ? pos0 : pos0 + my_tok;  // last key that the row sees
      float m = -INFINITY, l = 0.f;
      // (Where there are registers for it, summed up behind the last tile: 166.9 -> 164.7.)
      float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < ntile; ++j, ++done) {
        if (!(ok = __all_sync(kAll, mbar_wait(&s_full[x], done & 1)))) break;
        tc::fence_after_sync();
        const int kbase = (it.kt0 + j) * kTile;
        uint32_t r[4][32];
        float cm[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld_32x32_max(t_s + c * 32, r[c], cm[c]);
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[x]);
        float mt = max3f(cm[0], cm[1], fmaxf(cm[2], cm[3]));
        if (kbase + kTile - 1 > pos0) {  // keys past some row's position
          // (By chunks, with a warp's fully seen and fully hidden ones told apart
          // by branches, this took fewer instructions and spilled: 30 % slower.)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int seen = pos - (kbase + c * 32);  // last key of these 32 it sees
            const uint32_t hide = seen < 0 ? ~0u : seen >= 31 ? 0u : ~0u << (seen + 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((hide >> i) & 1) r[c][i] = __float_as_uint(-INFINITY);
          }
          float mx[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx[(i >> 1) & 7] = max3f(mx[(i >> 1) & 7], __uint_as_float(r[c][i]),
                                       __uint_as_float(r[c][i + 1]));
          mt = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]),
                     fmaxf(mx[6], mx[7]));
        }
        mt *= sl2;
        const float m_new = fmaxf(m, mt);
        const bool resc = live && m_new > m + kLazy;
        float alpha = 1.f;
        if (resc) {
          alpha = ex2_approx(m - m_new);
          m = m_new;
          l *= alpha;
          if constexpr (kOwnS<D, F>) {
#pragma unroll
            for (int i = 0; i < 8; ++i) rs[i] *= alpha;
          }
        }
        // A row that has seen masked keys alone (a part whose range starts past
        // its position) has m = -inf, and -inf + inf is NaN: taken with maximum 0
        // its weights are all zero and its partial row is empty.
        const float neg_m = m == -INFINITY ? 0.f : kRaise - m;
        if constexpr (!kOwnS<D, F>) {
#pragma unroll
          for (int i = 0; i < 8; ++i) rs[i] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          constexpr int kC = 4 / kHalves;
#pragma unroll
          for (int c = kC * h; c < kC * h + kC; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float y0, y1;
              fma_f32x2(y0, y1, __uint_as_float(r[c][2 * e]), __uint_as_float(r[c][2 * e + 1]),
                        sl2, sl2, neg_m, neg_m);
              const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
              const int q = 2 * (e & 3);
              add_f32x2(rs[q], rs[q + 1], rs[q], rs[q + 1], p0, p1);
              r[c][e] = pack2<T>(p0, p1);
            }
          if (h == 0 && j > 0) {  // P V of the tile before done: P is free, O stands still
            if (!(ok = __all_sync(kAll, mbar_wait(&pv_done[x], (done - 1) & 1)))) break;
            tc::fence_after_sync();
            if (__any_sync(kAll, resc)) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc::ld_32x32(t_o + c * 32, o);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tc::st_32x32(t_o + c * 32, o);
              }
              tc::wait_st();
            }
          }
#pragma unroll
          for (int c = kC * h; c < kC * h + kC; ++c)  // the packed pairs, as in the registers
            tc::st_32x16(tmem + t_lane + kColP + x * (kTile / 2) + c * 16, r[c]);
          if (!kTold && h + 1 < kHalves) continue;
          tc::wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(h + 1 == kHalves ? &p_full[x] : &p_half[x]);
        }
        if (!ok) break;
        if constexpr (!kOwnS<D, F>)
          l += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
      }
      if (!ok) break;
      if constexpr (kOwnS<D, F>)
        l = ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
      if (ntile > 0) {  // the last P V
        if (!(ok = __all_sync(kAll, mbar_wait(&pv_done[x], (done - 1) & 1)))) break;
        tc::fence_after_sync();
      }
      // The output, half the columns at a time.  Of a whole unit: each warp turns
      // its 32 rows around in its share of the ring slot granted to the item, so
      // that the stores to global memory are whole row halves and not 16 bytes of
      // 32 rows (which took 3,000 cycles a tile); rows that are not the sequence's
      // are left out, the next packed rows being another one's.  Of a part: the
      // unnormalised row.
      const bool whole = it.parts == 1;
      const int stage_u = u0 + 2 * it.n_kv;
      const int stage_i = stages;
      u0 = stage_u + whole;
      stages += whole;
      const int toks = x ? it.toks_b : it.toks_a, first = it.row0 + (x ? tpt : 0);
      if (toks == 0) continue;  // (tile B of a unit that ends in tile A)
      if (whole &&
          !(ok = __all_sync(kAll, mbar_wait(&st_full[stage_i % kRing], (stage_i / kRing) & 1))))
        break;
      constexpr int kHalf = D / 2, kChunks = kHalf / 8;  // columns; 16-byte chunks of them
      const float inv = l != 0.f ? 1.f / l : 0.f;
      uint8_t* stage = sKV + (stage_u % kRing) * C::TILE_BYTES + warp * (32 * D);
      auto at = [&](int r, int c) {  // chunk c of row r, conflict-free both ways
        return stage + r * D + ((c ^ (kChunks == 8 ? r & 7 : (r >> 1) & 3)) * 16);
      };
      T* out0 = static_cast<T*>(a.out) + ((size_t)first * a.H + it.hkv * a.G) * D;
      const size_t prow = (size_t)first * a.G + row, plane = (size_t)a.T * a.G;  // see part_ml
      float4* part_o =
          reinterpret_cast<float4*>(a.ws) + (size_t)(it.part * a.Hkv + it.hkv) * (D / 4) * plane;
      // (Rolled: the code of the hot loop above and of the other roles has to
      // stay in the instruction cache.)
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[kHalf / 32][32];
        if (ntile > 0) {
#pragma unroll
          for (int c = 0; c < kHalf / 32; ++c) tc::ld_32x32(t_o + hf * kHalf + c * 32, o[c]);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) o[i >> 5][i & 31] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int q = 0; q < kChunks; ++q) {
            uint32_t hv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              hv[i] = pack2<T>(__uint_as_float(o[q >> 2][8 * (q & 3) + 2 * i]) * inv,
                               __uint_as_float(o[q >> 2][8 * (q & 3) + 2 * i + 1]) * inv);
            *reinterpret_cast<uint4*>(at(lane, q)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
          }
          __syncwarp();
          const int c = lane % kChunks;
#pragma unroll 4
          for (int i = 0; i < kChunks; ++i) {
            const int r = i * (32 / kChunks) + lane / kChunks, rt = quarter * 32 + r;
            const int tok = (rt * a.g_magic) >> 16;  // rt / G
            if (tok < toks)
              *reinterpret_cast<uint4*>(out0 + ((size_t)tok * a.H + rt - tok * a.G) * D +
                                        hf * kHalf + c * 8) =
                  *reinterpret_cast<const uint4*>(at(r, c));
          }
          __syncwarp();
        } else if (live) {
          float4* dst = part_o + hf * (kHalf / 4) * plane + prow;
#pragma unroll
          for (int i = 0; i < kHalf / 4; ++i, dst += plane)
            *dst = make_float4(__uint_as_float(o[i >> 3][4 * (i & 7)]),
                               __uint_as_float(o[i >> 3][4 * (i & 7) + 1]),
                               __uint_as_float(o[i >> 3][4 * (i & 7) + 2]),
                               __uint_as_float(o[i >> 3][4 * (i & 7) + 3]));
        }
      }
      tc::fence_before_sync();  // O is read before the next item's P V overwrites it
      if (whole) {
        // The last of the four or eight warps that use the stage lets the slot go
        // (to TMA, the async proxy, which these accesses come before).  A count
        // and not a barrier: a tile may be several items ahead of the other.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          if (atomicAdd(&stage_left[stage_u % kRing], 1) == (it.toks_b > 0 ? 7 : 3)) {
            __threadfence_block();
            stage_left[stage_u % kRing] = 0;
            mbar_arrive(&kv_empty[stage_u % kRing]);
          }
        }
      } else if (live) {
        part_ml(a, D, it.part, it.hkv)[prow] = make_float2(m, l);
      }
    }
  } else if (warp == kWarpSched) {
    // ------------------------------------------------------------ scheduler, Q loads
    reg_dec();
    Units<F> units(a);
    const unsigned n_items = (unsigned)a.max_units * a.Hkv * a.split;  // below 2^31
    unsigned round = 0;
    int last_rank = -1, b = 0, unit = 0;
    bool more = true;
    // Items are dealt in rounds, every other one backwards, so that no CTA
    // gets the longest of every round.
    auto next = [&](Item& it) {
      it.valid = 0;
      while (more) {
        const unsigned at = (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        const unsigned idx = round * gridDim.x + at;
        ++round;
        if (!(more = idx < n_items)) break;
        const unsigned unit_head = divide((int)idx, a.by_split);
        const int rank = divide((int)unit_head, a.by_hkv);
        it.part = (int)(idx - unit_head * a.split);
        it.hkv = (int)(unit_head - rank * a.Hkv);
        if (rank != last_rank && !(more = units.find(rank, b, unit))) break;
        last_rank = rank;
        const Seq s = units.get(b);
        const int tok0 = unit * a.span;
        const int all = unit_tiles<F>(s, a.span, unit);
        it.parts = unit_parts(all, a.split);
        if (it.part >= it.parts) continue;
        it.valid = 1;
        it.b = b;
        it.n = s.n;
        it.row0 = s.start + tok0;
        it.toks_a = min(tpt, s.ql - tok0);
        it.toks_b = max(0, min(tpt, s.ql - tok0 - tpt));
        it.pos_a = F == kCross ? s.kv : s.n - s.ql + tok0;
        it.kt0 = 0;
        it.n_kv = all;
        if (it.parts > 1) {  // (at most 32 parts of 2^24 tiles)
          const unsigned at = (unsigned)it.part * all, parts = it.parts;
          it.kt0 = (int)(at / parts);
          it.n_kv = (int)((at + all) / parts) - it.kt0;
        }
        auto reads = [&](int pos, int toks) {
          if (F == kCross) return toks > 0 ? it.n_kv : 0;
          const int t = toks > 0 ? (int)((unsigned)(pos + toks - 1) / kTile) + 1 : 0;
          return min(max(t - it.kt0, 0), it.n_kv);
        };
        it.ntile_a = reads(it.pos_a, it.toks_a);
        it.ntile_b = reads(it.pos_a + tpt, it.toks_b);
        if (s.bad || (F == kCross && s.n == 0)) {  // no keys: zero rows, by the first part
          if (s.bad && lane == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
          if (it.part > 0) {
            it.valid = 0;
            continue;
          }
          it.parts = 1;
          it.kt0 = it.n_kv = it.ntile_a = it.ntile_b = 0;
        }
        break;
      }
    };
    auto post = [&](int k, const Item& it) {
      if (!(ok = __all_sync(kAll, wait_slow(&it_empty[k % kItems], ((k / kItems) & 1) ^ 1))))
        return;
      if (lane == 0) {
        items[k % kItems] = it;
        mbar_arrive(&it_full[k % kItems]);  // (release: the stores above are seen)
      }
      __syncwarp();
    };
    // Item k is posted ahead of the Q loads of item k - 1; the first item's Q goes with
    // it (behind the second one, the first products waited 3,000 cycles for it).
    Item cur;
    int q_row = 0, q_hkv = 0;
    bool q_due = false;
    for (int k = 0; ok; ++k) {
      next(cur);
      post(k, cur);
      if (k != 1) {
        const int j = k == 0 ? 0 : k - 1;  // the item whose Q is due
        if (k == 0) {
          q_due = cur.valid;
          q_row = cur.row0;
          q_hkv = cur.hkv;
        }
        // Tile by tile as the products of the item before that let go of it: boxes of
        // tpt tokens x G heads x 64 dims; rows past the array read as zeros.
        if (ok && lane == 0 && q_due)
          for (int x = 0; x < 2 && ok; ++x) {
            if (!(ok = mbar_wait(&q_free[x], (j & 1) ^ 1))) break;
            mbar_arrive_expect_tx(&q_full[x], C::HALVES * tpt * a.G * 128);
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_3d(sQ + x * kQRoom + hf * kSlab, &qmap, 64 * hf, q_hkv * a.G,
                          q_row + x * tpt, &q_full[x]);
            ++issued;
          }
      }
      ok = __shfl_sync(kAll, ok, 0);
      if (!cur.valid) break;
      q_due = k > 0;
      q_row = cur.row0;
      q_hkv = cur.hkv;
    }
    if (blockIdx.x == 0)
      for (int i = lane; i < a.B; i += 32)
        if (sequence<F>(a, i).lost) flag_status(a.status, PA_DEV_BAD_CONTEXT);
  } else if (warp == kWarpLoad) {
    // ------------------------------------------------------------ K and V
    reg_dec();
    const int bpt = PAGED ? kTile / a.block_size : 1;  // blocks of a key tile
    const int bbytes = C::TILE_BYTES / bpt;
    int u = 0, stages = 0;  // ring slots and stages, over all items
    Item it;
    for (int k = 0; take(k, it); ++k) {
      const int nblk = PAGED ? (it.n + a.block_size - 1) / a.block_size : 0;
      // first row of the sequence's keys
      const int row = PAGED ? 0 : F == kCross ? it.pos_a : it.row0 - it.pos_a;
      int win = -kWindow;
      auto load_tile = [&](int t, bool v) {
        const int lb0 = (it.kt0 + t) * bpt;
        if (PAGED && (lb0 < win || lb0 + bpt > win + kWindow)) {
          // K_t is requested before V_{t-1}: the window starts one tile early.
          win = (!v && t > 0) ? lb0 - bpt : lb0;
          __syncwarp();
          int ent[kWindow / 32];
#pragma unroll
          for (int e = 0; e < kWindow / 32; ++e) {
            const int lb = win + lane + 32 * e;
            ent[e] = lb < nblk ? a.block_tables[(size_t)it.b * a.max_blocks + lb]
                               : a.num_blocks;  // past the sequence: zeros
          }
#pragma unroll
          for (int e = 0; e < kWindow / 32; ++e) {
            int phys = ent[e];
            if (phys < 0 || phys > a.num_blocks ||
                (phys == a.num_blocks && win + lane + 32 * e < nblk)) {
              flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
              phys = a.num_blocks;
            }
            tbl[lane + 32 * e] = phys * a.block_size * a.Hkv + it.hkv;  // the box's row
          }
          __syncwarp();
        }
        const int st = u % kRing;
        uint64_t* full = v ? &v_full[issued_v % kRing] : &k_full[issued % kRing];
        if (elect_one()) {
          ok = mbar_wait(&kv_empty[st], ((u / kRing) & 1) ^ 1);
          if (ok) mbar_arrive_expect_tx(full, C::TILE_BYTES);
        }
        ok = __all_sync(kAll, ok);
        if (!ok) return;
        uint8_t* dst = sKV + st * C::TILE_BYTES;
        if constexpr (PAGED) {
          // One box per block: (64 dims, 8 keys, halves, key groups) at row
          // (block * block_size * Hkv + head) of the pool.
          if (elect_one()) {
            const CUtensorMap* map = v ? &vmap : &kmap;
            // (Four at a time: 8 x 512 tokens on 3,584 in 8-token blocks 246 us, 264 from
            // lane to lane and 286 one by one; in larger blocks alike.)
#pragma unroll 1
            for (int j = 0; j < bpt; j += 4, dst += 4 * bbytes) {
              const int4 r = *reinterpret_cast<const int4*>(tbl + lb0 - win + j);
              tma_load_5d(dst, map, 0, 0, 0, 0, r.x, full);
              tma_load_5d(dst + bbytes, map, 0, 0, 0, 0, r.y, full);
              tma_load_5d(dst + 2 * bbytes, map, 0, 0, 0, 0, r.z, full);
              tma_load_5d(dst + 3 * bbytes, map, 0, 0, 0, 0, r.w, full);
            }
          }
        } else if (elect_one()) {
          // 128 tokens of one head, both halves; rows past the array read as zeros.
          tma_load_4d(dst, v ? &vmap : &kmap, 0, row + (it.kt0 + t) * kTile, 0, it.hkv,
                      full);
        }
        ++u;
        ++(v ? issued_v : issued);
      };
      // K_0, then K_{t+1} and V_t in turn (see ring_k).
      if constexpr (PAGED) {
        // One copy of the code: three took half of the warp's time in missed
        // instructions, and of the softmax's with it (16 x 2,048 keys 517 -> 474 us).
#pragma unroll 1
        for (int i = 0; i < 2 * it.n_kv && ok; ++i) {
          const int half = (i + 1) >> 1;
          const bool v = i > 0 && (!(i & 1) || half == it.n_kv);
          load_tile(v ? half - 1 : half, v);
        }
      } else {
        if (it.n_kv > 0) load_tile(0, false);
        for (int j = 0; j < it.n_kv && ok; ++j) {
          if (j + 1 < it.n_kv) load_tile(j + 1, false);
          if (ok) load_tile(j, true);
        }
      }
      // One slot of the ring is the item's output stage.
      if (ok && it.parts == 1) {
        const int st = u % kRing;
        if (lane == 0) {
          ok = mbar_wait(&kv_empty[st], ((u / kRing) & 1) ^ 1);
          if (ok) mbar_arrive(&st_full[stages % kRing]);
        }
        ok = __shfl_sync(kAll, ok, 0);
        ++u;
        ++stages;
      }
      if (!ok) break;
    }
  } else if (warp == kWarpS) {
    // ------------------------------------------------------------ S = Q K^T
    reg_dec();
    const uint64_t dk = tc::smem_desc(smem_u32(sKV), 16, C::GROUP, tc::kSwizzle128B);
    const uint64_t dq = tc::smem_desc(smem_u32(sQ), 16, 1024, tc::kSwizzle128B);
    // (The loops over the two tiles are unrolled: an array indexed at run time
    // would sit in local memory, on the chain from one S product to the next.)
    int u0 = 0, k0 = 0, done[2] = {0, 0};  // ring slots, K tiles and products before
    uint64_t* last_free = nullptr;  // s_free of the product issued last, its phase
    int last_phase = 0;
    Item it;
    for (int k = 0; take(k, it); ++k) {
      const int nt[2] = {it.ntile_a, it.ntile_b};
      if (elect_one()) {
        bool q_there[2] = {false, false};
        for (int t = 0; t < it.n_kv && ok; ++t) {
          // Paged keys are awaited ahead of S, so that nothing but the product stands
          // behind that wait, which is on the chain from one product to the next (8 x
          // 512 on 3,584 248 -> 244 us); rows behind it (8 of 500-4,096 353 -> 348).
          const int st = (u0 + ring_k(t)) % kRing, ki = k0 + t;
          const uint64_t db = dk + st * (C::TILE_BYTES >> 4);
          if (PAGED && !(ok = mbar_wait(&k_full[ki % kRing], (ki / kRing) & 1))) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (t >= nt[x] || !ok) continue;
            if (!q_there[x] && !(ok = q_there[x] = mbar_wait(&q_full[x], k & 1))) continue;
            const uint64_t da = dq + x * (kQRoom >> 4);
            // S is free once the softmax of the product before has loaded it (of the
            // tile's own product where it has a region of its own).
            if (kOwnS<D, F> ? done[x] > 0 && !(ok = mbar_wait(&s_free[x], (done[x] - 1) & 1))
                            : last_free != nullptr && !(ok = mbar_wait(last_free, last_phase)))
              continue;
            if (!PAGED && !(ok = mbar_wait(&k_full[ki % kRing], (ki / kRing) & 1))) continue;
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_f16(tmem + kColS + x * kNextS,
                          da + (((kk >> 2) * kSlab + (kk & 3) * 32) >> 4),
                          db + (((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4), kIdS, kk > 0);
            tc::commit(&s_full[x]);
            if (t + 1 == nt[x]) tc::commit(&q_free[x]);
            last_free = &s_free[x];
            last_phase = done[x] & 1;
            ++done[x];
          }
          if (ok) tc::commit(&kv_empty[st]);
        }
        // A tile that read nothing lets its Q go, once it has landed.
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (ok && nt[x] == 0 && (ok = mbar_wait(&q_full[x], k & 1))) mbar_arrive(&q_free[x]);
        u0 += 2 * it.n_kv + (it.parts == 1);
        k0 += it.n_kv;
      }
      if (!(ok = __all_sync(kAll, ok))) break;
    }
  } else {  // kWarpPv
    // ------------------------------------------------------------ O += P V
    reg_dec();
    const uint64_t dv = tc::smem_desc(smem_u32(sKV), C::HALF, C::GROUP, tc::kSwizzle128B);
    int u0 = 0, v0 = 0, done[2] = {0, 0};  // ring slots, V tiles and products before
    Item it;
    for (int k = 0; take(k, it); ++k) {
      const int nt[2] = {it.ntile_a, it.ntile_b};
      // Rows of the last key tile past the sequence's keys hold whatever the
      // block's tail, or the next sequence's rows, hold: 0 * NaN is NaN, so the
      // warp zeroes them once V has landed.
      // (Two rounds through one copy of the code: the tiles up to it, by one lane
      // without meeting the others, and it alone.)
      const int live = it.n - (it.kt0 + it.n_kv - 1) * kTile;
      const int whole = it.n_kv - (it.n_kv > 0 && live < kTile ? 1 : 0);
      for (int t0 = 0, t1 = whole; t0 < it.n_kv; t0 = t1, t1 = it.n_kv) {
        if (t0 == whole) {
          const int st = (u0 + ring_v(t0, it.n_kv)) % kRing, vi = v0 + t0;
          if (lane == 0) ok = mbar_wait(&v_full[vi % kRing], (vi / kRing) & 1);
          if (!(ok = __shfl_sync(kAll, ok, 0))) break;
          uint8_t* vt = sKV + st * C::TILE_BYTES;
          constexpr int kChunks = D / 8;
          for (int i = lane; i < (kTile - live) * kChunks; i += 32) {
            const int r = live + i / kChunks, c = i % kChunks;
            *reinterpret_cast<uint4*>(vt + (r >> 3) * C::GROUP + (c >> 3) * C::HALF +
                                      (r & 7) * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (elect_one())
          for (int t = t0; t < t1 && ok; ++t) {
            const int st = (u0 + ring_v(t, it.n_kv)) % kRing, vi = v0 + t;
            const uint64_t db = dv + st * (C::TILE_BYTES >> 4);
            if (!(ok = mbar_wait(&v_full[vi % kRing], (vi / kRing) & 1))) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (t >= nt[x] || !ok) continue;
              const uint32_t ta = tmem + kColP + x * (kTile / 2);
              // (P of an item's first tile is stored behind the item before's last
              // read of O by the same warps: O may then be overwritten.)
              if (!(ok = mbar_wait(kTold ? &p_half[x] : &p_full[x], done[x] & 1))) continue;
              tc::fence_after_sync();
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk) {
                if (kTold && kk == kTile / 32) {
                  if (!(ok = mbar_wait(&p_full[x], done[x] & 1))) break;
                  tc::fence_after_sync();
                }
                tc::mma_f16_ts(tmem + kColO + x * D, ta + kk * 8,
                               db + ((kk * 2 * C::GROUP) >> 4), kIdO, t > 0 || kk > 0);
              }
              if (!ok) continue;
              tc::commit(&pv_done[x]);
              ++done[x];
            }
            if (ok) tc::commit(&kv_empty[st]);
          }
        if (!(ok = __all_sync(kAll, ok))) break;
      }
      if (!ok) break;
      u0 += 2 * it.n_kv + (it.parts == 1);
      v0 += it.n_kv;
    }
  }

  // All roles meet.  After a wait that gave up, the loaders let their copies
  // land and the issuers their MMAs end (all bounded) before the CTA leaves.
  tc::fence_before_sync();
  if (__syncthreads_or(!ok)) {
    if (threadIdx.x == 0) flag_status(a.status, PA_DEV_TIMEOUT);
    if (warp == kWarpSched && lane == 0)
      for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait(&q_full[i & 1], (i >> 1) & 1);
    if (warp == kWarpLoad && lane == 0) {
      for (int i = max(0, issued - kRing); i < issued; ++i)
        mbar_wait(&k_full[i % kRing], (i / kRing) & 1);
      for (int i = max(0, issued_v - kRing); i < issued_v; ++i)
        mbar_wait(&v_full[i % kRing], (i / kRing) & 1);
    }
    if ((warp == kWarpS || warp == kWarpPv) && elect_one()) {  // (who issued them)
      tc::commit(drain);
      mbar_wait(drain, 0);
    }
    __syncthreads();
  }
  if (warp == kWarpS) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
  }
}

// Merges the parts of split units by log-sum-exp (m, l in the log2 domain).  A
// block takes 32 consecutive rows of a K/V head, a lane each; its warps first
// take the parts' (m, l) in turn and leave every part's weight in shared memory,
// then D / 8 columns each, four parts' loads in flight.  (One thread to a row
// with all its parts one after the other: 64 us for 32 parts, all latency.)
constexpr int kMergeWarps = 8;
template <typename T, int D, Form F>
__global__ void __launch_bounds__(32 * kMergeWarps) grouped_merge_kernel(const GroupedArgs a) {
  constexpr int kC = D / 4 / kMergeWarps;  // groups of four columns of a warp
  __shared__ float s_w[kGroupedMaxSplit][32];     // m, then the weight of a part
  __shared__ float s_m[kMergeWarps][32], s_l[kMergeWarps][32];
  __shared__ uint2 s_out[32][D / 4 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hkv = blockIdx.y;
  const size_t plane = (size_t)a.T * a.G, row0 = (size_t)blockIdx.x * 32, r = row0 + lane;
  // The lengths come from before the attention kernel, which let this one start only
  // when all its blocks had waited for them: they are read while it still runs.
  int parts = 0;  // of this lane's row; 0: nothing to merge
  const int t = r < plane ? (int)(r / a.G) : -1;
  Seq s = {0, 0, 0, 0, true, true};  // the sequence that holds row t
  auto holds = [&]() { return !s.lost && t >= s.start && t < s.start + s.ql; };
  if (t >= 0) {  // by halving, as offsets rise
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.q_offsets[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    s = sequence<F>(a, lo);
  }
  // A row of no sequence, or one beside offsets that fall: the sequences that these
  // belong to are not computed, but the others are, and looking at all finds theirs.
  if (__any_sync(kAll, t >= 0 && !holds())) {
    int falls = 0;
    for (int b = lane; b < a.B; b += 32) falls |= a.q_offsets[b] > a.q_offsets[b + 1];
    if (__any_sync(kAll, falls) && t >= 0)
      for (int b = 0; b < a.B && !holds(); ++b) s = sequence<F>(a, b);
  }
  if (t >= 0 && !s.bad && holds())
    parts = unit_parts(unit_tiles<F>(s, a.span, divide(t - s.start, a.by_span)), a.split);
  if (parts == 1) parts = 0;  // (written by its only part)
  pdl_wait();
  pdl_launch_dependents();
  const int most = __reduce_max_sync(kAll, parts);
  if (most == 0) return;  // (alike in all warps)
  float M = -INFINITY;
  float m[kGroupedMaxSplit / kMergeWarps], l[kGroupedMaxSplit / kMergeWarps];
#pragma unroll
  for (int i = 0; i < kGroupedMaxSplit / kMergeWarps; ++i) {
    const int p = warp + i * kMergeWarps;
    m[i] = -INFINITY;
    l[i] = 0.f;
    if (p < parts) {
      const float2 ml = part_ml(a, D, p, hkv)[r];
      m[i] = ml.x;
      l[i] = ml.y;
    }
  }
#pragma unroll
  for (int i = 0; i < kGroupedMaxSplit / kMergeWarps; ++i)
    if (l[i] != 0.f) M = fmaxf(M, m[i]);
  s_m[warp][lane] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, s_m[w][lane]);
  float L = 0.f;
#pragma unroll
  for (int i = 0; i < kGroupedMaxSplit / kMergeWarps; ++i) {
    // an empty part's row is no number: weight 0 stands for leaving it out
    const float w = l[i] != 0.f ? ex2_approx(m[i] - M) : 0.f;
    s_w[warp + i * kMergeWarps][lane] = w;
    if (l[i] != 0.f) L += w * l[i];
  }
  s_l[warp][lane] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) L += s_l[w][lane];
  const float inv = L != 0.f ? 1.f / L : 0.f;
  float4 acc[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src =
      reinterpret_cast<const float4*>(a.ws) + ((size_t)hkv * (D / 4) + warp * kC) * plane + r;
  const size_t step = (size_t)a.Hkv * (D / 4) * plane;  // to the next part
#pragma unroll 4
  for (int p = 0; p < most; ++p) {
    const float w = s_w[p][lane];
    if (p < parts && w != 0.f) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const float4 v = src[p * step + c * plane];
        acc[c].x += w * v.x;
        acc[c].y += w * v.y;
        acc[c].z += w * v.z;
        acc[c].w += w * v.w;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kC; ++c)
    s_out[lane][warp * kC + c] = make_uint2(pack2<T>(acc[c].x * inv, acc[c].y * inv),
                                            pack2<T>(acc[c].z * inv, acc[c].w * inv));
  __syncthreads();
  // Whole rows, a warp one at a time (lane q's count says whether row q is merged).
  for (int q = warp; q < 32; q += kMergeWarps) {
    if (__shfl_sync(kAll, parts, q) == 0) continue;
    const size_t rr = row0 + q, t = rr / a.G;
    T* dst = static_cast<T*>(a.out) + (t * a.H + hkv * a.G + (rr - t * a.G)) * D;
    for (int c = lane; c < D / 4; c += 32) reinterpret_cast<uint2*>(dst)[c] = s_out[q][c];
  }
}

template <typename T, int D, Form F>
cudaError_t launch_t(const GroupedArgs& a, const void* q, const void* k, const void* v,
                     long long q_stride, long long k_stride, long long v_stride,
                     cudaStream_t stream) {
  constexpr bool PAGED = F == kChunk;
  using C = Cfg<D, PAGED>;
  using u64 = unsigned long long;
  CUtensorMap qmap, kmap, vmap;
  {
    const u64 dims[3] = {(u64)D, (u64)a.H, (u64)a.T};
    const u64 st[2] = {(u64)D * 2, (u64)q_stride * 2};
    const unsigned box[3] = {64, (unsigned)a.G, (unsigned)(a.span / 2)};
    const cudaError_t e = make_map_3d(&qmap, q, dims, st, box, true);
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; i < 2; ++i) {
    CUtensorMap* map = i ? &vmap : &kmap;
    cudaError_t e;
    if constexpr (PAGED) {
      // Rows (slot, head) of D values; inside a block (64 dims, 8 keys, halves,
      // key groups), at its first slot's row.
      const u64 rowb = (u64)D * 2, tok = rowb * a.Hkv;
      const u64 dims[5] = {64, 8, (u64)C::HALVES, (u64)a.block_size / 8,
                           (u64)a.num_blocks * a.block_size * a.Hkv};
      const u64 st[4] = {tok, 128, 8 * tok, rowb};
      const unsigned box[5] = {64, 8, (unsigned)C::HALVES, (unsigned)a.block_size / 8, 1};
      e = make_map_5d(map, i ? v : k, dims, st, box, true);
    } else {
      const int rows = F != kCross ? a.T : a.Tk > 0 ? a.Tk : 1;
      const u64 dims[4] = {64, (u64)rows, (u64)C::HALVES, (u64)a.Hkv};
      const u64 st[3] = {(u64)(i ? v_stride : k_stride) * 2, 128, (u64)D * 2};
      const unsigned box[4] = {64, kTile, (unsigned)C::HALVES, 1};
      e = make_map_4d(map, i ? v : k, dims, st, box, true);
    }
    if (e != cudaSuccess) return e;
  }
  constexpr auto kern = grouped_kernel<T, D, F>;
  cudaError_t e = ensure_dynamic_smem<kern>(C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // One CTA for each SM, or for each item where there are fewer.
  const long long items = (long long)a.max_units * a.Hkv * a.split;
  const int nsm = sm_count() > 0 ? sm_count() : 1;
  cfg.gridDim = dim3((unsigned)(items < nsm ? items : nsm));
  cfg.blockDim = dim3(kThreadsG);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, a);
  if constexpr (F != kPrompt) {
    if (e != cudaSuccess || a.split == 1) return e;
    cudaLaunchConfig_t cm = cfg;
    cm.gridDim = dim3((unsigned)(((long long)a.T * a.G + 31) / 32), a.Hkv);
    cm.blockDim = dim3(32 * kMergeWarps);
    cm.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cm, grouped_merge_kernel<T, D, F>, a);
  }
  return e;
}

}  // namespace

int grouped_span(int G) { return G <= kTile ? 2 * (kTile / G) : 0; }

int grouped_split(int B, int T, int H, int Hkv, int max_context) {
  const int span = grouped_span(H / Hkv);
  const int nsm = sm_count();
  if (span == 0 || nsm <= 0) return 1;
  // Lengths are on the device, so the cost of s parts to a unit is a weighted sum of
  // two guesses, in key tiles, a part costing kPartCost tiles besides its own.  All
  // sequences alike: whole rounds of equal parts over the SMs.  Ragged ones, where
  // there are several (half a unit lost at each one's end, contexts of 0.7 of the
  // longest on average): the longest part, or all of them spread over the SMs.
  // Fitted to sweeps of s on twenty batches: 4 x 64 tokens on 16,384 keys 67 us (99
  // with the spread alone), 2 x 128 on 8,192 41 (55), 16 on 65,536 66 (85, the least
  // 61); furthest from its least is 16 x 16 on 4,096 with 60 of 50, taken for ragged.
  constexpr double kMean = 0.7, kPartCost = 3.0, kRagged = 2.5;
  const double alike = (double)B * ((((long long)T + B - 1) / B + span - 1) / span) * Hkv;
  double units = (double)T / span + 0.5 * B;
  if (units < B) units = B;
  units *= Hkv;
  const double tiles = ((double)max_context + kTile - 1) / kTile;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= kGroupedMaxSplit && (s == 1 || s * kGroupedMinPartTiles <= tiles); ++s) {
    const double cost = s > 1 ? kPartCost : 0.0;
    const double longest = tiles / s + cost;
    double t = ceil(alike * s / nsm) * longest;
    if (B > 1) {
      const double spread = units * s * (kMean * tiles / s + cost) / nsm;
      t += kRagged * (longest > spread ? longest : spread);
    }
    if (s == 1 || t < least) {
      best = s;
      least = t;
    }
  }
  return best;
}

size_t grouped_workspace_bytes(int B, int T, int H, int Hkv, int D, int max_context) {
  const int s = grouped_split(B, T, H, Hkv, max_context);
  return s <= 1 ? 0 : (size_t)s * T * H * (D + 2) * sizeof(float);
}

cudaError_t launch_grouped(const GroupedArgs& a, const void* q, const void* k, const void* v,
                           long long q_stride, long long k_stride, long long v_stride,
                           cudaStream_t stream) {
#define PK_GROUPED(TT, DD)                                                                     \
  (a.kv_starts != nullptr                                                                      \
       ? launch_t<TT, DD, kCross>(a, q, k, v, q_stride, k_stride, v_stride, stream)            \
   : a.block_tables != nullptr                                                                 \
       ? launch_t<TT, DD, kChunk>(a, q, k, v, q_stride, k_stride, v_stride, stream)            \
       : launch_t<TT, DD, kPrompt>(a, q, k, v, q_stride, k_stride, v_stride, stream))
  if (a.bf16) return a.D == 128 ? PK_GROUPED(__nv_bfloat16, 128) : PK_GROUPED(__nv_bfloat16, 64);
  return a.D == 128 ? PK_GROUPED(__half, 128) : PK_GROUPED(__half, 64);
#undef PK_GROUPED
}

}  // namespace pk
