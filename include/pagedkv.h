/*
 * pagedkv.h -- C ABI of libpagedkv: attention over a paged KV cache on one
 * NVIDIA GB300 (sm_103a), plus the two cache-maintenance copies.
 *
 * The problem statement these calls implement comes from three pages:
 *  - blog "PagedAttention origin and evolution" (PagedAttention的起源与演进),
 *    sec. 3.2.1 (K and V pools of shape [num_blocks, block_size, num_heads,
 *    head_dim], fp16) and sec. 3.2.2 (forward pass: per request, gather K/V
 *    through block_tables[batch, max_num_blocks], cut to context_lens,
 *    Q K^T / sqrt(head_dim), softmax, weighted sum of V);
 *  - tutorial chapter "4. PagedAttention机制：vLLM的核心创新", sections
 *    "PagedAttention的核心思想" (fixed-size blocks of 16 or 32 tokens, not
 *    contiguous, mapped by a Block Table), "Block管理策略" (blocks taken and
 *    returned through a free list as the cache grows) and
 *    "PagedAttention的注意力计算" (per logical block: physical =
 *    block_table[logical], score every token, softmax, weighted V);
 *  - study notes "DataWhale组队学习笔记--llm-algo-leetcode(五)", sections
 *    "3. PagedAttention 的工作机制" (the lookup is transparent to the model)
 *    and "4. PagedAttention 带来的核心红利" (sequences sharing a prompt point
 *    at the same physical blocks; a block is copied when one of them writes).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - fp16 data (pa_half) is IEEE binary16, passed as raw 16-bit patterns.
 *  - Every pointer argument except the host-side scalars is a DEVICE pointer
 *    of the current CUDA device, row-major and contiguous.  Where a call says
 *    so, an argument may instead be the device address of mapped page-locked
 *    host memory (pa_host_device_pointer): the kernel then reads or writes
 *    it across the host link itself.  The caller owns all memory; the
 *    library allocates nothing and never synchronises.
 *  - Every call is asynchronous on `stream` (0 = the legacy default stream).
 *  - Argument errors are reported synchronously, before anything is
 *    launched: PA_ERR_INVALID for a bad pointer, size or alignment,
 *    PA_ERR_UNSUPPORTED for a head_dim / block_size pair with no kernel,
 *    PA_ERR_WORKSPACE for a workspace that is too small, PA_ERR_CUDA when a
 *    launch fails (pa_last_cuda_error() then holds the cudaError_t value).
 *  - Errors in device-resident data (a block id outside [0, num_blocks), a
 *    context length out of range, a slot outside the pool, a copy pair out
 *    of range) are detected by the kernels: the affected work is skipped or
 *    clamped, never read or written out of bounds, and the PA_DEV_* bit is
 *    OR-ed into `*status` when `status` (a device int32) is not NULL.  The
 *    caller zeroes *status before the call and reads it afterwards.
 *  - Buffers that a call reads must not be written by the same call
 *    (no aliasing between inputs and outputs).
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t pa_half;               /* IEEE binary16 bit pattern */
typedef struct CUstream_st *pa_stream_t; /* same type as cudaStream_t */

typedef enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID = 1,
    PA_ERR_UNSUPPORTED = 2,
    PA_ERR_WORKSPACE = 3,
    PA_ERR_CUDA = 4
} pa_status;

/* Bits OR-ed into the device status word. */
#define PA_DEV_BAD_BLOCK_ID 0x1   /* a needed block-table entry is outside [0, num_blocks) */
#define PA_DEV_BAD_CONTEXT 0x2    /* context length < 0, > max_context_len or > table capacity */
#define PA_DEV_BAD_SLOT 0x4       /* a slot >= num_blocks * block_size */
#define PA_DEV_BAD_PAIR 0x8       /* a copy pair outside [0, num_blocks) */
#define PA_DEV_TIMEOUT 0x10       /* a bounded wait inside a kernel gave up */
#define PA_DEV_NO_BLOCKS 0x20     /* the free ring holds fewer blocks than a step needs */
#define PA_DEV_BAD_BEAM 0x40      /* a parent or beam outside [0, W), a length past the steps */
#define PA_DEV_BAD_LOGITS 0x80    /* NaN or +inf among a live beam's logits */

/* Element type of the calls that take one: 2 bytes each, and 4 of logits. */
typedef enum pa_dtype {
    PA_F16 = 0,  /* IEEE binary16 */
    PA_BF16 = 1, /* bfloat16 */
    PA_F32 = 2   /* IEEE binary32, pa_beam_select's logits only */
} pa_dtype;

/* Human-readable name of a status code (static storage). */
const char *pa_status_string(pa_status s);

/* cudaError_t value behind the last PA_ERR_CUDA returned on this thread. */
int pa_last_cuda_error(void);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int pa_version(void);

/* Device address of page-locked host memory: memory from cudaHostAlloc /
 * cudaMallocHost, or registered with cudaHostRegister, that is mapped into
 * the current device's address space (always so with unified addressing).
 * The device address lets a kernel load and store that memory directly,
 * with no staging copy.  host_ptr may point anywhere inside the
 * allocation.  Returns PA_ERR_INVALID, with *device_ptr set to NULL, when
 * host_ptr is NULL or is not mapped page-locked memory; device_ptr must not
 * be NULL.  Synchronous, launches nothing. */
pa_status pa_host_device_pointer(const void *host_ptr, void **device_ptr);

/* ---------------------------------------------------------------------------
 * Decode attention (one query token per sequence).
 *
 * Definition (blog sec. 3.2.2, tutorial "PagedAttention的注意力计算"): for each
 * sequence b and head h, with n = context_lens[b] and key j stored in
 * physical block block_tables[b][j / block_size], token slot j % block_size,
 *     s_j   = scale * sum_d q[b,h,d] * k_cache[blk(j), j % bs, h, d]
 *     p_j   = exp(s_j - max_k s_k) / sum_k exp(s_k - max_k s_k)
 *     out[b,h,:] = sum_j p_j * v_cache[blk(j), j % bs, h, :]
 * for j in [0, n).  n == 0 gives a zero row.  Only the first
 * ceil(n / block_size) entries of a table row are read; later entries may
 * hold anything (conventionally -1).  Pool slots past a sequence's length
 * (the tail of its last block, unreferenced blocks) may hold anything, NaN
 * included, without changing the result.
 *
 * q            [B, H, D] fp16
 * k_cache      [num_blocks, block_size, H, D] fp16 (v_cache alike)
 * block_tables [B, max_blocks_per_seq] int32
 * context_lens [B] int32, each in [0, min(max_context_len,
 *              max_blocks_per_seq * block_size)]
 * out          [B, H, D] fp16, written with round-to-nearest-even from an
 *              fp32 accumulation
 * D in {64, 128}; block_size in {4, 8, 16, 32}; q, k_cache, v_cache and out
 * 16-byte aligned.  q, out, block_tables and context_lens may be mapped
 * page-locked host memory (pa_host_device_pointer); the caches and the
 * workspace are device memory.
 *
 * Long contexts are split into partitions of `partition_tokens` keys (a
 * multiple of block_size, at most 32 blocks; 0 picks one from B, H and
 * max_context_len); each partition's running max, normaliser and
 * unnormalised output go to `workspace` and a second kernel merges them by
 * log-sum-exp.  max_context_len is a host-side bound on every
 * context_lens[b] so the split plan never reads device memory.
 * workspace: device memory of at least
 * pa_decode_workspace_size(B, H, D, block_size, max_context_len,
 * partition_tokens) bytes, 16-byte aligned, owned by the caller, contents
 * need not be initialised; may be NULL when that size is 0.
 * ------------------------------------------------------------------------- */
int pa_decode_partition_tokens(int B, int H, int block_size, int max_context_len);

size_t pa_decode_workspace_size(int B, int H, int D, int block_size,
                                int max_context_len, int partition_tokens);

pa_status pa_decode(const pa_half *q, const pa_half *k_cache,
                    const pa_half *v_cache, const int32_t *block_tables,
                    const int32_t *context_lens, int B, int H, int D,
                    int block_size, int num_blocks, int max_blocks_per_seq,
                    int max_context_len, int partition_tokens, float scale,
                    pa_half *out, void *workspace, size_t workspace_bytes,
                    int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Decode for groups of sequences that share a prefix of physical blocks.
 *
 * Sequences forked from one prompt point at the same physical blocks until
 * they diverge (study notes "4. PagedAttention 带来的核心红利": shared blocks,
 * copy-on-write).  Same result as pa_decode (same arguments, workspace and
 * errors), but every partition of partition_tokens keys that lies entirely
 * inside a group's shared prefix is read from HBM once for the whole group
 * and attended by all its members' queries together; the remaining
 * partitions run per sequence, and all are merged by log-sum-exp.
 *
 * Groups (CSR): members of group g are group_seqs[group_offsets[g] ..
 * group_offsets[g+1]) (sequence indices, at most max_group_size <= 16 per
 * group); group_prefix_len[g] is the number of leading tokens whose blocks
 * all its members share; seq_group[b] is the group of sequence b or -1.  The
 * caller guarantees that members' block tables agree on the shared blocks
 * (the first member's table is read for them) and that every member's
 * context holds the prefix.  max_prefix_len bounds group_prefix_len on the
 * host.  Only whole partitions are shared: choose partition_tokens dividing
 * the shared prefix for the full benefit; partitions are shared only when
 * partition_tokens is a multiple of 16 (with other sizes every member reads
 * its own, same result).  D in {64, 128}, block_size in {4, 8, 16, 32}
 * (4-token blocks are copied by the lanes, the slower path).
 * ------------------------------------------------------------------------- */
pa_status pa_decode_shared_prefix(const pa_half *q, const pa_half *k_cache,
                                  const pa_half *v_cache,
                                  const int32_t *block_tables,
                                  const int32_t *context_lens,
                                  const int32_t *seq_group,
                                  const int32_t *group_offsets,
                                  const int32_t *group_seqs,
                                  const int32_t *group_prefix_len,
                                  int num_groups, int max_group_size,
                                  int max_prefix_len, int B, int H, int D,
                                  int block_size, int num_blocks,
                                  int max_blocks_per_seq, int max_context_len,
                                  int partition_tokens, float scale,
                                  pa_half *out, void *workspace,
                                  size_t workspace_bytes, int32_t *status,
                                  pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Groups for pa_decode_shared_prefix, derived from the block tables (host).
 *
 * Sequences share logical block i when their tables hold the same physical
 * id at position i and at every earlier position (study notes "4.
 * PagedAttention 带来的核心红利": forked sequences map their common prompt
 * to the same blocks).  A prefix tree over each sequence's full blocks
 * (floor(min(context_lens[b], max_blocks_per_seq*block_size) / block_size)
 * leading entries, stopping at the first negative id) groups the sequences:
 * where the sequences below a node part ways, at depth d blocks, they form
 * one group sharing d*block_size tokens; a node holding more than
 * max_group_size sequences first groups those of its children that hold two
 * or more (they share more) and cuts the rest into groups of at most
 * max_group_size at depth d.  No group shares fewer than min_shared_tokens
 * (pass partition_tokens: shorter prefixes hold no whole shared partition).
 * Each group has >= 2 members in increasing index order, groups in increasing
 * order of their first member; the shared prefix is the exact longest common
 * prefix of the members' full blocks.
 *
 * All pointers are HOST memory, row-major [B, max_blocks_per_seq] tables.
 * Outputs, caller-allocated: seq_group[B] (group of b or -1),
 * group_offsets[B/2 + 1], group_seqs[B], group_prefix_len[B/2] (tokens), and
 * *num_groups.  Pass them straight to pa_decode_shared_prefix after copying
 * to the device.  Errors: PA_ERR_INVALID for a null pointer, B < 0,
 * max_blocks_per_seq or block_size <= 0, min_shared_tokens < 0 or
 * max_group_size < 2 (outputs untouched except *num_groups = 0).  Host code
 * only: no CUDA call, thread-safe, O(total full blocks * log) time.
 * ------------------------------------------------------------------------- */
pa_status pa_shared_prefix_groups(const int32_t *block_tables,
                                  const int32_t *context_lens, int B,
                                  int max_blocks_per_seq, int block_size,
                                  int min_shared_tokens, int max_group_size,
                                  int32_t *seq_group, int32_t *group_offsets,
                                  int32_t *group_seqs,
                                  int32_t *group_prefix_len, int *num_groups);

/* ---------------------------------------------------------------------------
 * Decode with append: cache write of the new token fused into decode.
 *
 * Each decode step appends one token per sequence (tutorial "Block管理策略": the
 * cache grows into the sequence's mapped blocks) and attends with it.  For
 * every sequence b with n = context_lens[b] >= 1, the new token sits at
 * position n-1: its K/V rows k_new[b], v_new[b] ([B, H, D] fp16) are stored
 * to slot block_tables[b][(n-1)/bs] * bs + (n-1) % bs of k_cache/v_cache
 * (bit-exact, as pa_kv_cache_write would), and the query attends to keys
 * 0..n-1 exactly as pa_decode, the new key included.  One launch replaces
 * pa_kv_cache_write + pa_decode.  Every other argument, the workspace and
 * the errors are as for pa_decode; a block id outside [0, num_blocks) for
 * the new token's block skips its store and sets PA_DEV_BAD_BLOCK_ID.
 * k_new and v_new must not alias the caches; like q, out, block_tables
 * and context_lens they may be mapped page-locked host memory (16-byte
 * aligned).
 * ------------------------------------------------------------------------- */
pa_status pa_decode_append(const pa_half *q, const pa_half *k_new,
                           const pa_half *v_new, pa_half *k_cache,
                           pa_half *v_cache, const int32_t *block_tables,
                           const int32_t *context_lens, int B, int H, int D,
                           int block_size, int num_blocks,
                           int max_blocks_per_seq, int max_context_len,
                           int partition_tokens, float scale, pa_half *out,
                           void *workspace, size_t workspace_bytes,
                           int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * FP8 (e4m3) KV storage: quantizing cache write and decode over it.
 *
 * The blog's sec. 2.3 lists mixed-precision KV storage; this is its reading
 * here.  Each (token, head) row of K and of V is stored as D e4m3 codes
 * (1 sign, 4 exponent bits with bias 7, 3 fraction bits, largest finite
 * value 448) plus one fp32 scale: value = code * scale, with
 * scale = max|row| / 448 (1 for an all-zero row) and code = e4m3(x / scale)
 * rounded to nearest even (both divisions correctly rounded fp32).  A row is
 * D + 4 bytes instead of 2D, so decode reads about half the bytes.
 *
 * k_cache8, v_cache8  [num_blocks, block_size, H, D] uint8 (e4m3 codes)
 * k_scale, v_scale    [num_blocks, H, block_size] float32
 * pa_kv_cache_write_fp8 takes the same tokens and slots as
 * pa_kv_cache_write (fp16 k, v [T, H, D]) and writes codes and scales;
 * H at most 65535 (as for decode), else PA_ERR_INVALID.
 * pa_decode_fp8 computes pa_decode's result on the dequantized cache
 * (fp32 accumulation, fp16 output), same arguments, workspace and errors.
 * ------------------------------------------------------------------------- */
pa_status pa_kv_cache_write_fp8(const pa_half *k, const pa_half *v,
                                const int64_t *slot_mapping, int T, int H,
                                int D, int block_size, int num_blocks,
                                uint8_t *k_cache8, uint8_t *v_cache8,
                                float *k_scale, float *v_scale,
                                int32_t *status, pa_stream_t stream);

pa_status pa_decode_fp8(const pa_half *q, const uint8_t *k_cache8,
                        const uint8_t *v_cache8, const float *k_scale,
                        const float *v_scale, const int32_t *block_tables,
                        const int32_t *context_lens, int B, int H, int D,
                        int block_size, int num_blocks, int max_blocks_per_seq,
                        int max_context_len, int partition_tokens, float scale,
                        pa_half *out, void *workspace, size_t workspace_bytes,
                        int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Decode attention with no workspace and no allocation.
 *
 * This entry point has no counterpart on the pages; it exists for callers
 * that cannot allocate device memory for a call -- a host runtime that has
 * handed the whole device heap to its own pool, a plugin inside another
 * engine that forbids allocations outside that engine's allocator, or a
 * latency-critical loop that cannot pay for cudaMalloc's implicit device
 * synchronisation.  It computes exactly what pa_decode computes, with the
 * same arguments minus the workspace: the split-KV partition scratch lives
 * in a fixed device array inside the library (PA_DECODE_STATIC_SCRATCH_BYTES,
 * held on every GPU that loads the library until the process exits).
 *  - It calls no cudaMalloc, cudaFree or other allocating routine.
 *  - Arguments are checked as pa_decode checks them, with the same codes;
 *    then a plan needing more scratch than the array holds, i.e.
 *    pa_decode_workspace_size(...) > PA_DECODE_STATIC_SCRATCH_BYTES, is
 *    refused with PA_ERR_WORKSPACE before anything is launched; a smaller
 *    partition count (larger partition_tokens) or batch fits.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current) and caches it; make
 *    that first call before any stream capture.  A failed look-up returns
 *    PA_ERR_CUDA.  The cached address belongs to the device's current
 *    context: after cudaDeviceReset on a device, do not call this entry
 *    point on that device again in the same process.
 *  - All calls share the one array and it keeps the last call's contents;
 *    nothing in it needs to start at zero.  Calls whose kernels overlap on
 *    the GPU (different streams without ordering) race on it: serialise them.
 * ------------------------------------------------------------------------- */
#define PA_DECODE_STATIC_SCRATCH_BYTES (8u << 20)

pa_status pa_decode_static(const pa_half *q, const pa_half *k_cache,
                           const pa_half *v_cache, const int32_t *block_tables,
                           const int32_t *context_lens, int B, int H, int D,
                           int block_size, int num_blocks,
                           int max_blocks_per_seq, int max_context_len,
                           int partition_tokens, float scale, pa_half *out,
                           int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Chunked prefill attention (Lq new query tokens per sequence).
 *
 * The Lq queries of sequence b are its last Lq positions: query i sits at
 * position n - Lq + i, n = context_lens[b] (which counts the chunk, whose
 * K/V must already be in the cache), and attends to keys
 * 0 .. n - Lq + i (causal mask aligned to the end of the context; with
 * Lq == n this is the lower-triangular mask of the blog's sec. 3.2.2, with
 * Lq == 1 it is decode).  Same per-row arithmetic as pa_decode; pool slots
 * past a sequence's length may hold anything, NaN included.
 *
 * q   [B, H, Lq, D] fp16 (the blog's [batch, heads, seq_len, head_dim])
 * out [B, H, Lq, D] fp16
 * context_lens[b] in [Lq, max_blocks_per_seq * block_size]; scale > 0.
 * D in {64, 128} and block_size in {4, 8, 16, 32}, all on the tcgen05
 * tensor-core kernel (blocks of 8 or more tokens arrive by TMA; 4-token
 * blocks are gathered with 16-byte copies, the slower path); any other
 * (D, block_size) returns PA_ERR_UNSUPPORTED.  The pool must hold fewer
 * than 2^31 (slot, head) rows (num_blocks * block_size * H; under 512 GiB
 * per pool at D = 128), else PA_ERR_INVALID.
 *
 * workspace (device, 16-byte aligned, caller-owned, may be NULL): with at
 * least pa_prefill_workspace_size(B, H, Lq, D) bytes, the work units of the
 * grid's last, partial round (one CTA per SM) are each split into key ranges
 * whose partial results are merged by log-sum-exp, so that round fills the
 * GPU; with NULL every unit runs whole (same result up to rounding).  A
 * non-NULL workspace smaller than that returns PA_ERR_WORKSPACE.  The size
 * depends on the SM count of the current device.
 * ------------------------------------------------------------------------- */
size_t pa_prefill_workspace_size(int B, int H, int Lq, int D);

pa_status pa_prefill_chunk(const pa_half *q, const pa_half *k_cache,
                           const pa_half *v_cache, const int32_t *block_tables,
                           const int32_t *context_lens, int B, int H, int Lq,
                           int D, int block_size, int num_blocks,
                           int max_blocks_per_seq, float scale, pa_half *out,
                           void *workspace, size_t workspace_bytes,
                           int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Chunked prefill with a chunk length per sequence.
 *
 * The same computation as pa_prefill_chunk for sequence b's q_lens[b] new
 * queries, which sit in rows 0 .. q_lens[b]-1 of its [H, Lq_max, D] slice
 * of q: query i is at position n - q_lens[b] + i (n = context_lens[b]) and
 * attends to keys 0 .. n - q_lens[b] + i (the blog's sec. 3.2.2 forward pass
 * takes each request's queries on their own).  Rows q_lens[b] .. Lq_max-1
 * of out are written as zeros.  q_lens is [B] int32 on the device (or in
 * mapped page-locked host memory), each in [0, Lq_max] and at most
 * context_lens[b]; a sequence breaking that is flagged PA_DEV_BAD_CONTEXT in
 * *status and its rows are zeros.  q_lens NULL (with B, Lq_max > 0) returns
 * PA_ERR_INVALID.  Every other argument, the workspace rule (with
 * pa_prefill_workspace_size(B, H, Lq_max, D)) and the error behaviour are
 * those of pa_prefill_chunk with Lq = Lq_max.
 * ------------------------------------------------------------------------- */
pa_status pa_prefill_chunk_varlen(const pa_half *q, const pa_half *k_cache,
                                  const pa_half *v_cache, const int32_t *block_tables,
                                  const int32_t *context_lens, const int32_t *q_lens,
                                  int B, int H, int Lq_max, int D, int block_size,
                                  int num_blocks, int max_blocks_per_seq, float scale,
                                  pa_half *out, void *workspace, size_t workspace_bytes,
                                  int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Cache write (scatter new tokens' K/V into their slots).
 *
 * With the caches viewed as [num_blocks * block_size, H, D], for each token
 * t with slot_mapping[t] >= 0:  k_cache[slot] = k[t], v_cache[slot] = v[t]
 * (bit-exact copies).  slot = physical_block * block_size + offset, the
 * address a sequence's block table gives its position (tutorial, "Block管理
 * 策略": the cache grows into newly mapped blocks).  Negative slots are
 * padding and are skipped.  Two tokens with the same slot: undefined which
 * one lands.
 *
 * k, v          [T, H, D] fp16
 * slot_mapping  [T] int64
 * k_cache, v_cache as for pa_decode, written in place.
 * ------------------------------------------------------------------------- */
pa_status pa_kv_cache_write(const pa_half *k, const pa_half *v,
                            const int64_t *slot_mapping, int T, int H, int D,
                            int block_size, int num_blocks, pa_half *k_cache,
                            pa_half *v_cache, int32_t *status,
                            pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Block copy (copy-on-write of shared blocks; study notes sec. 4).
 *
 * For each pair i: physical block pairs[i][1] of k_cache and of v_cache
 * becomes a bit-exact copy of block pairs[i][0] (all block_size * H * D
 * values).  Destinations must be distinct and no destination may be the
 * source of another pair in the same call (otherwise the result is
 * undefined); src == dst is a no-op.  The values are copied as 16 bits each, so the
 * bf16 pools of the calls with grouped heads (H: their K/V heads) are copied as well.
 *
 * pairs [N, 2] int64 (src, dst).
 * ------------------------------------------------------------------------- */
pa_status pa_block_copy(pa_half *k_cache, pa_half *v_cache,
                        const int64_t *pairs, int N, int H, int D,
                        int block_size, int num_blocks, int32_t *status,
                        pa_stream_t stream);

/* ===========================================================================
 * One serving step with grouped K/V heads.
 *
 * The calls below serve models whose H query heads share Hkv <= H key/value
 * heads (query head h reads K/V head h / (H / Hkv); H a multiple of Hkv), in
 * fp16 or bf16 (pa_dtype), with the step's new tokens packed: sequence b's
 * tokens are rows q_offsets[b] .. q_offsets[b+1]-1 of [T, heads, D] arrays,
 * no padding between sequences.  They are, in the order a step uses them:
 * the plan (blocks, slots and positions from the lengths), the rotation of
 * queries and keys with the cache write, and attention of new prompts, of
 * chunks over the cache, and of single tokens.  The cache is the pool of the
 * calls above with Hkv heads: [num_blocks, block_size, Hkv, D].
 *
 * Packed q, k, v may be views of one projection's output: a token's heads
 * are contiguous and 16-byte aligned, *_stride is the distance between
 * tokens in elements, a multiple of 8 and at least heads * D.  Outputs of
 * attention are contiguous.  None of these calls keeps anything between
 * calls, so they may run on several streams and be captured; a workspace
 * belongs to one call at a time.  T is below 2^31 - 32768.  The attention of prompts
 * and chunks is made for some hundreds of sequences a call: past that its time grows
 * with their square (1,000 short prompts 0.4 ms, 4,000 5.8 ms).
 * ========================================================================= */

/* ---------------------------------------------------------------------------
 * Step plan: block tables, slots and positions from the sequences' lengths.
 *
 * Sequence b has cached_lens[b] tokens in the cache and new_lens[b] more in
 * this step (0: it does not run).  With have = ceil(cached / block_size) and
 * want = ceil((cached + new) / block_size), entries have .. want-1 of its
 * table row are filled with blocks from the free list, first in, first out,
 * sequences in order (tutorial, "Block管理策略": Block Table, Free List, growth
 * into new blocks); the others are left as they were.  Written besides:
 *   context_lens [B]    int32  cached + new
 *   q_offsets    [B+1]  int32  first packed row of each sequence, then the total
 *   slot_mapping [T_max] int64 slot of each packed token (as pa_kv_cache_write
 *                              takes it), -1 in the rows behind the last one
 *   positions    [T_max] int32 its position, 0 behind the last one
 *
 * The free list is a ring: free_blocks [num_blocks] int32, free_state [2]
 * int64 = blocks taken and blocks put so far, so it holds free_state[1] -
 * free_state[0] blocks, the next one at index free_state[0] mod num_blocks.
 * context_lens may be cached_lens itself.  free_state_out [2] receives the
 * state after the step and may be free_state itself; a caller returns a block
 * by writing its id at free_state[1] mod num_blocks and adding one to
 * free_state[1].
 *
 * All or nothing: when the blocks needed exceed those held
 * (PA_DEV_NO_BLOCKS) or the new tokens exceed T_max (PA_DEV_BAD_CONTEXT), no
 * block is taken and the step is empty: context_lens = cached, offsets 0,
 * slots -1.  A sequence with a negative length, or that outgrows its table
 * row, is flagged PA_DEV_BAD_CONTEXT, adds nothing and gets context 0; where
 * context_lens is cached_lens its length stays as it was, so that it is flagged
 * again in the next step and its blocks are not taken for a new sequence's (with
 * lengths in two buffers that is the caller's to see to).  An id
 * outside [0, num_blocks), in the ring or in the block that new tokens
 * continue, is flagged PA_DEV_BAD_BLOCK_ID: its tokens get slot -1 (and a
 * fresh entry -1).
 *
 * block_size in {4, 8, 16, 32}; B at most 16384 (else PA_ERR_UNSUPPORTED);
 * max_blocks_per_seq * block_size below 2^31 - 64, T_max below 2^31 - 32768.
 * ------------------------------------------------------------------------- */
pa_status pa_step_plan(const int32_t *cached_lens, const int32_t *new_lens, int B,
                       int block_size, int num_blocks, int max_blocks_per_seq, int T_max,
                       const int32_t *free_blocks, const int64_t *free_state,
                       int32_t *block_tables, int32_t *context_lens, int32_t *q_offsets,
                       int64_t *slot_mapping, int32_t *positions, int64_t *free_state_out,
                       int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Rotary positions with several axes, with the cache write.
 *
 * Pair i (of rotary_dim / 2) of every query and key head turns by
 * angle = positions[axis(i)][t] * inv_freq(i):
 *     x' = x cos(angle) - y sin(angle),  y' = y cos(angle) + x sin(angle)
 * where (x, y) = (dims i, i + rotary_dim / 2), or (2i, 2i + 1) with
 * interleaved != 0; dims from rotary_dim on pass unchanged.  One axis is the
 * usual position of text, three are time, height and width of image and
 * video tokens.  Sines and products are fp32 and exact to fp32 at every int32
 * position (negative ones too); results are rounded once, to nearest even.
 *
 * Rotated q goes to q_out, rotated k to k_out unless that is NULL, and to
 * k_cache at slot_mapping[t]; v is copied to v_cache there.  Negative slots
 * skip the cache write (q_out and k_out are still written); a slot past the
 * pool is flagged PA_DEV_BAD_SLOT and skipped; what a slot
 * that two tokens share receives is undefined.  k_cache, v_cache, v and
 * slot_mapping may all be NULL: rotation only, k_out is then required.  q_out may be q and k_out may
 * be k (the same pointer and stride), no other overlap is allowed.
 *
 * q [T, H, D], k and v [T, Hkv, D] with their strides; q_out, k_out likewise
 * positions [n_axes, T] int32, n_axes 1..4
 * table [rotary_dim / 2] from pa_rope_table, on the device, its axes below
 *       n_axes (a larger one reads the last axis)
 * D in {64, 128}, block_size in {4, 8, 16, 32}; rotary_dim a multiple of 16,
 * 16 .. D.
 *
 * pa_rope_table (host): table[i] = inv_freq[i] / 2 pi as a 64-bit fraction of
 * a turn, axes[i] (0..3; NULL: all 0) in its two low bits.  inv_freq in radians
 * a position, finite and below 2^50 in magnitude; PA_ERR_INVALID otherwise.
 * ------------------------------------------------------------------------- */
pa_status pa_rope_table(const double *inv_freq, const int32_t *axes, int n, uint64_t *table);

pa_status pa_rope_cache_write(const void *q, const void *k, const void *v,
                              const int32_t *positions, const uint64_t *table,
                              const int64_t *slot_mapping, int T, int H, int Hkv, int D,
                              int rotary_dim, int n_axes, int interleaved, pa_dtype dtype,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              int block_size, int num_blocks, void *q_out,
                              int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                              void *k_cache, void *v_cache, int32_t *status,
                              pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention over whole prompts (packed, causal, grouped heads).
 *
 * Token i of sequence b attends to tokens 0 .. i of its own sequence, K and V
 * being packed rows like q (no cache is read):
 *     s_j = scale * q[t,h,:] . k[j,h/G,:],  out[t,h,:] = softmax(s) v[.,h/G,:]
 * with G = H / Hkv, scores and sums in fp32; the softmax weights are rounded to
 * the 16-bit type for their product with v, the result once more, to nearest
 * even.  Rows before q_offsets[0] and behind q_offsets[B] are left as they
 * were.  Other sequences' rows, NaN included, never reach a result, nor does a
 * later token's k; a later token's v must be finite (its weight is an exact zero,
 * and a zero times an infinity or NaN in the same 128 keys is NaN).
 *
 * q [T, H, D], k and v [T, Hkv, D] with their strides; out [T, H, D]
 * q_offsets [B+1] int32, rising, within [0, T]: a sequence breaking that is
 *           flagged PA_DEV_BAD_CONTEXT and not computed.  (Offsets that fall and
 *           so make sequences overlap leave all rows undefined: the work of a
 *           call is bounded by that of T rows, the longest units first.)
 * D in {64, 128}; H / Hkv at most 128 (else PA_ERR_UNSUPPORTED); scale > 0.
 * ------------------------------------------------------------------------- */
pa_status pa_prompt_attention(const void *q, const void *k, const void *v,
                              const int32_t *q_offsets, int B, int T, int H, int Hkv, int D,
                              pa_dtype dtype, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, float scale, void *out, int32_t *status,
                              pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of packed chunks over the paged cache (grouped heads).
 *
 * Sequence b's q_len = q_offsets[b+1] - q_offsets[b] queries are its last
 * positions: query i is at n - q_len + i, n = context_lens[b], and attends to
 * keys 0 .. n - q_len + i of the cache (which holds the chunk's own K/V
 * already).  Otherwise as pa_prompt_attention; the cache as in pa_decode with
 * Hkv heads.  Slots past a sequence's length may hold anything.  A context
 * outside [q_len, max_context_len] is flagged PA_DEV_BAD_CONTEXT and its rows
 * are zeros; a bad block id reads as zeros, flagged PA_DEV_BAD_BLOCK_ID.
 *
 * D in {64, 128}; block_size in {8, 16, 32}; max_context_len at most
 * max_blocks_per_seq * block_size and below 2^31 - 32768; (num_blocks + 1) *
 * block_size * Hkv below 2^31.  workspace (16-byte aligned, may be NULL): with at least
 * pa_chunk_attention_workspace_size(...) bytes, few and long chunks are cut
 * into key ranges merged by log-sum-exp, which fills the GPU; without it every
 * unit runs whole (same result up to rounding).  Smaller and not NULL:
 * PA_ERR_WORKSPACE.
 * ------------------------------------------------------------------------- */
size_t pa_chunk_attention_workspace_size(int B, int T, int H, int Hkv, int D,
                                         int max_context_len);

pa_status pa_chunk_attention(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, const int32_t *context_lens,
                             const int32_t *q_offsets, int B, int T, int H, int Hkv, int D,
                             pa_dtype dtype, int64_t q_stride, int block_size, int num_blocks,
                             int max_blocks_per_seq, int max_context_len, float scale,
                             void *out, void *workspace, size_t workspace_bytes,
                             int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Cross attention: packed queries over other rows, with no causal mask.
 *
 * Request b's queries are the packed rows q_offsets[b] .. q_offsets[b+1]-1; its
 * keys and values are rows kv_starts[b] .. kv_starts[b] + kv_lens[b] - 1 of k and
 * v, an encoder's states of another length, and every query sees all of them:
 *     out[t,h,:] = softmax_j(scale * q[t,h,:] . k[j,h/G,:]) v[j,h/G,:]
 * otherwise as pa_prompt_attention.  The rows of the requests may be packed,
 * padded to one length or slots of a pool, in any order and shared between requests.
 * The beams of a request are queries of it, so its states are read once for all of
 * them.  With k, v and offsets of the queries' own rows it is the attention of an
 * encoder.  A request with no keys gets zero rows.  Rows outside the requests are left
 * as they were.  What other rows of k and v hold, NaN included, never reaches a result.
 *
 * q [T, H, D], k and v [Tk, Hkv, D] with their strides; out [T, H, D]
 * q_offsets [B+1] int32 as for pa_prompt_attention; kv_starts, kv_lens [B] int32
 * max_q_len, max_kv_len  host-side bounds on the requests' lengths: a request past one
 *           of them, or whose keys leave [0, Tk), is flagged PA_DEV_BAD_CONTEXT and its
 *           rows are zeros (max_q_len above T counts as T, 0 as 1)
 * D in {64, 128}; scale > 0.  With max_q_len * H / Hkv at most 16 (up to 48 where B is 1
 * or 2 and all its CTAs run at once; B at most 65535) the kernel of pa_decode_grouped
 * serves the call, to its precision; otherwise that of pa_prompt_attention, to its, and
 * H / Hkv is at most 128 (else PA_ERR_UNSUPPORTED).  So a request's last bits go by the
 * call that it is in.
 *
 * workspace (16-byte aligned, may be NULL): with at least
 * pa_cross_attention_workspace_size(...) bytes few queries over many keys are cut into
 * key ranges merged by log-sum-exp; without it they run whole (same result up to
 * rounding).  Smaller and not NULL: PA_ERR_WORKSPACE.  The size depends on the SM count
 * of the current device and may be 0.
 * ------------------------------------------------------------------------- */
size_t pa_cross_attention_workspace_size(int B, int T, int H, int Hkv, int D, int max_q_len,
                                         int max_kv_len);

pa_status pa_cross_attention(const void *q, const void *k, const void *v,
                             const int32_t *q_offsets, const int32_t *kv_starts,
                             const int32_t *kv_lens, int B, int T, int Tk, int H, int Hkv,
                             int D, pa_dtype dtype, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, int max_q_len, int max_kv_len, float scale,
                             void *out, void *workspace, size_t workspace_bytes,
                             int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Decode with grouped heads: one query token per sequence.
 *
 * pa_decode's result (the softmax weights enter their product with v to 2^-15 in
 * bf16 and 2^-21 in fp16, the result is rounded once) where G = H / Hkv query heads
 * read each K/V head, which comes from memory once for all of them (up to 16; more
 * take it once for every 16).  Arguments, errors and the workspace rule as for pa_decode, with
 * q and out [B, H, D] and the cache [num_blocks, block_size, Hkv, D] in dtype;
 * a context past max_context_len is flagged PA_DEV_BAD_CONTEXT and cut to it, a
 * negative one gives zeros.  partition_tokens: a multiple of 64 up to 2048, or
 * 0 to choose.  The workspace size depends on the SM count of the current device;
 * it is 0 where one partition holds the longest context or all partitions fit
 * the GPU at once (they then merge inside the launch).  D in {64, 128};
 * block_size in {8, 16, 32}; B at most 65535;
 * any finite scale; (num_blocks + 1) * block_size * Hkv below 2^31.
 * ------------------------------------------------------------------------- */
size_t pa_decode_grouped_workspace_size(int B, int H, int Hkv, int D, int block_size,
                                        int max_context_len, int partition_tokens);

pa_status pa_decode_grouped(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, const int32_t *context_lens, int B,
                            int H, int Hkv, int D, pa_dtype dtype, int block_size,
                            int num_blocks, int max_blocks_per_seq, int max_context_len,
                            int partition_tokens, float scale, void *out, void *workspace,
                            size_t workspace_bytes, int32_t *status, pa_stream_t stream);

/* ===========================================================================
 * Beam search over the paged cache.
 *
 * A request has W beams (1 .. 32): sequences b * W .. b * W + W-1 of the calls
 * above, which share blocks until they part (study notes "4. PagedAttention
 * 带来的核心红利": a block is copied when one of them writes).  A step of a decoder:
 * pa_step_plan, pa_rope_cache_write, pa_decode_grouped over all B * W sequences
 * (and pa_cross_attention, the beams being queries of their request), then
 * pa_beam_select on the logits, pa_beam_reorder of the tables, and pa_block_copy
 * with its pairs in every layer's cache.  The steps' tokens and parents are kept,
 * [S, B, W] each (an output of pa_beam_select may be a slice of them), and
 * pa_beam_backtrack gathers sequences from them.  B * W is at most 2^20.  None of
 * these calls keeps anything between calls; a workspace belongs to one call at a
 * time.
 * ========================================================================= */

/* ---------------------------------------------------------------------------
 * Beam selection: the best continuations over beams and vocabulary.
 *
 * With x_w the logits of beam w of a request, candidate (w, v) has the score
 *     c(w, v) = scores[w] + x_w[v] - log sum_u exp(x_w[u])
 * (log-probabilities in place of logits give the same).  The W best candidates
 * with v != eos_token are the next beams, best first; of equal ones the lowest
 * (w, v) comes first.  Two candidates of one beam are compared by their logits, two
 * of different beams by their c in 64 bits, of which the sum under the logarithm is
 * taken in fp32: equal rows of a request have equal sums, but different beams'
 * candidates nearer than its error (at most 1.3e-5 + V * 2^-33 for logits in no
 * particular order) can change places, and its last bits go by B, W, V, the beams that
 * are there and the alignment of logits and row_stride.  Written [B, W]:
 *   tokens, parents  v and w of each
 *   new_scores       c, rounded once; may be scores itself
 *   ended_scores     by beam w: c(w, eos_token) if it is better than the last of
 *                    the W chosen (the hypothesis of beam w ends here), else -inf
 * eos_token -1: no candidate ends.  A score of -inf (any that is not finite) is a
 * beam that is not there: the first step has one of 0 and W - 1 of -inf, a request that
 * is done W of them; its logits are not read.  A logit of -inf is never chosen.  A
 * place that no candidate fills gets pad_token, its own index as parent and -inf.  A
 * beam with NaN or +inf among its logits gives no candidate, flagged PA_DEV_BAD_LOGITS.
 *
 * logits [B * W] rows of V in dtype (PA_F32 too), row_stride >= V elements apart
 * scores [B, W] float32; V at most 2^28; eos_token below V
 * workspace: at least pa_beam_select_workspace_size(B, W, V) bytes, 16-byte aligned, else
 * PA_ERR_WORKSPACE; the size is 0 but for small batches with several beams and a large
 * vocabulary, and depends on the current device.
 * W above 32 returns PA_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */
size_t pa_beam_select_workspace_size(int B, int W, int V);

pa_status pa_beam_select(const void *logits, pa_dtype dtype, int64_t row_stride,
                         const float *scores, int B, int W, int V, int eos_token,
                         int pad_token, int32_t *tokens, int32_t *parents,
                         float *new_scores, float *ended_scores, void *workspace,
                         size_t workspace_bytes, int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Beam reorder: block tables that follow the chosen beams.
 *
 * Beam w of request b goes on from its beam p = parents[b][w]: row b * W + w of
 * tables_out gets the ceil(n / block_size) first entries of row b * W + p, n =
 * context_lens[b * W + p], and -1 in all others; context_lens_out gets n.  p = -1
 * ends the beam: an empty row, length 0.
 *
 * Copy-on-write: when n is no multiple of block_size, the beam's next token goes into
 * the row's last block.  The first beam of the request with that block keeps it; every
 * further one gets a block from the free list (the ring of pa_step_plan, first in, first
 * out, beams in order) in its place, and copy_pairs[b * W + w] = (old, new) for
 * pa_block_copy; of all other beams the pair is (0, 0), which copies nothing.  When n is
 * a multiple, pa_step_plan gives each beam its next block.  This is for beams that are
 * of one length, as a search's are: only last blocks are looked at, so that a half-full
 * last block which a longer beam of the request holds as a full one is not copied for
 * it, and the shorter beam's next token would be written among the longer one's.
 *
 * Back to the list: a block that rows of the request held at a column, and that none of
 * them holds there any more, is written to the ring behind the last one, requests in
 * order, then columns, then beams (so equal inputs give equal rings); columns below
 * shared_lens[b] / block_size are left out (NULL: none).  No counts of holders are
 * needed while a request's beams have grown from one sequence: blocks that requests
 * share are then of a prefix which all beams hold, so that they come back only when all
 * beams of a request end; such a request names its shared tokens in shared_lens.
 *
 * free_state_out: blocks taken and put after the call.  All or nothing: when the blocks
 * needed exceed those held before the call, or free_state is none that a ring of
 * num_blocks can have, PA_DEV_NO_BLOCKS is flagged and everything stays as it was
 * (copied, where outputs are other arrays; no pairs).  A request with a parent outside
 * [-1, W) (PA_DEV_BAD_BEAM), a length that its rows cannot hold or a negative shared
 * length (PA_DEV_BAD_CONTEXT) stays as it was, too.  An id outside [0, num_blocks) in a
 * last block, in the ring (the entry is then -1) or among those that would come back is
 * flagged PA_DEV_BAD_BLOCK_ID and neither copied nor put; others are moved unseen.
 *
 * parents [B, W], block_tables and tables_out [B * W, max_blocks_per_seq], context_lens
 * and context_lens_out [B * W], shared_lens [B] int32, copy_pairs [B * W, 2] int64;
 * free_blocks and free_state as for pa_step_plan.  tables_out may be block_tables,
 * context_lens_out context_lens, and free_state_out free_state.
 * W at most 32, block_size in {4, 8, 16, 32} (else PA_ERR_UNSUPPORTED);
 * max_blocks_per_seq * block_size below 2^31 - 64.  workspace: at least
 * pa_beam_reorder_workspace_size(...) bytes (0 for small batches), 16-byte aligned.
 * ------------------------------------------------------------------------- */
size_t pa_beam_reorder_workspace_size(int B, int W, int max_blocks_per_seq);

pa_status pa_beam_reorder(const int32_t *parents, const int32_t *block_tables,
                          const int32_t *context_lens, const int32_t *shared_lens, int B,
                          int W, int block_size, int num_blocks, int max_blocks_per_seq,
                          int32_t *free_blocks, const int64_t *free_state,
                          int32_t *tables_out, int32_t *context_lens_out,
                          int64_t *free_state_out, int64_t *copy_pairs, void *workspace,
                          size_t workspace_bytes, int32_t *status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Beam backtrack: hypotheses' tokens from the steps' tokens and parents.
 *
 * Hypothesis k of request b has n = lengths[b][k] tokens and ends in beam beams[b][k]:
 *     beam(n - 1) = beams[b][k],  beam(s - 1) = parents[s][b][beam(s)],
 *     out[b][k][s] = tokens[s][b][beam(s)] for s < n, pad_token behind
 * (one that ended with eos_token at step s, by ended_scores of its beam w, has length s
 * and beam w; its end is no token of it).
 *
 * tokens, parents [S, B, W] int32; lengths, beams [B, K] int32; out [B, K, S] int32.
 * A length outside [0, S] or, where there are tokens, a beam outside [0, W) gives
 * pad_token alone, a parent outside [0, W) pad_token in the steps before it; both flagged
 * PA_DEV_BAD_BEAM.  W and K at most 32 (else PA_ERR_UNSUPPORTED), S below 2^26 - 1024.
 * ------------------------------------------------------------------------- */
pa_status pa_beam_backtrack(const int32_t *tokens, const int32_t *parents,
                            const int32_t *lengths, const int32_t *beams, int S, int B,
                            int W, int K, int pad_token, int32_t *out, int32_t *status,
                            pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
