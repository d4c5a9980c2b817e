"""A serving step with grouped K/V heads (include/pagedkv.h): step plan, rotary
cache write, prompt attention, chunk attention and grouped decode, on packed
tokens in fp16 or bf16.

Argument marshalling only, as in ``_lib``: every step runs in the library's
CUDA kernels.  The kernels of a single-token step take 2 to 6 us, less than
checking and passing ten to seventeen tensors from Python (7 to 9 us), so these
calls go through a compiled binding (``csrc/py_grouped.cpp``) that checks the
arguments, allocates a workspace that was left out and makes the call; the
functions here allocate outputs and say which argument did not fit.
"""
from typing import NamedTuple

import torch

from ._lib import _check, _ptr, lib

_HALF = (torch.float16, torch.bfloat16)
_UNFIT = -1  # the binding found an argument that does not fit


class StepPlan(NamedTuple):
    """What pa_step_plan writes besides the block tables."""
    context_lens: torch.Tensor  # [B] int32
    q_offsets: torch.Tensor     # [B + 1] int32
    slot_mapping: torch.Tensor  # [max_tokens] int64
    positions: torch.Tensor     # [max_tokens] int32
    free_state: torch.Tensor    # [2] int64

    @classmethod
    def empty(cls, batch, max_tokens, device):
        def new(n, dtype):
            return torch.empty(n, dtype=dtype, device=device)
        return cls(new(batch, torch.int32), new(batch + 1, torch.int32),
                   new(max_tokens, torch.int64), new(max_tokens, torch.int32),
                   new(2, torch.int64))


_grouped = None


def _binding():
    """The compiled binding; raises if the library has not been built."""
    global _grouped
    if _grouped is None:
        lib()
        try:
            from . import _grouped as module
        except ImportError as e:
            raise RuntimeError("the grouped binding is not built: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        _grouped = module
    return _grouped


def _handle(name, stream, tensor):
    """What the binding takes for a stream: its handle, or None for the current one."""
    if stream is None:
        return None
    if isinstance(tensor, torch.Tensor) and stream.device != tensor.device:
        raise ValueError(f"{name}: stream on {stream.device}, tensors on {tensor.device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor from the pool of the stream that the call runs on: one of
    another stream's pool could still be in use there, or be handed out again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _failed(rc, name, q, dense, strided=(), status=None):
    """Raises the error behind a call's return code.  dense, strided: (name, tensor,
    dtype or None for q's, shape; None: any size) of the arguments in order; q:
    the tensor that the others go by, first of its list."""
    if rc != _UNFIT:
        _check(rc, name)
    for is_strided, group in ((True, strided), (False, dense)):
        for what, t, dtype, shape in group:
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: {what} must be a torch.Tensor")
            if dtype is None and q.dtype not in _HALF:
                raise TypeError(f"{name}: {what} must be fp16 or bf16, got {q.dtype}")
            if t.dtype != (dtype or q.dtype):
                raise TypeError(f"{name}: {what} must be {dtype or q.dtype}, got {t.dtype}")
            if not t.is_cuda:
                raise ValueError(f"{name}: {what} must be on a CUDA device")
            if t.device != q.device:
                raise ValueError(f"{name}: {what} is on {t.device}, others on {q.device}")
            if t.dim() != len(shape) or any(n not in (None, m) for n, m in zip(shape, t.shape)):
                raise ValueError(f"{name}: {what} must be {list(shape)} (None: any), got "
                                 f"{list(t.shape)}")
            if not is_strided and not t.is_contiguous():
                raise ValueError(f"{name}: {what} must be contiguous")
            if is_strided and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
                raise ValueError(f"{name}: a token's heads must be contiguous in {what}")
    if status is not None and (status.dtype != torch.int32 or status.device != q.device):
        raise TypeError(f"{name}: status must be int32 on the tensors' device")
    raise ValueError(f"{name}: bad arguments")


def _size(t, dim):
    """A size that other arguments go by, None where there is none to read."""
    return t.shape[dim] if isinstance(t, torch.Tensor) and t.dim() > dim else None


def pa_step_plan(cached_lens, new_lens, block_tables, free_blocks, free_state, block_size,
                 max_tokens, out=None, status=None, stream=None):
    """Block tables, slots and positions of a step, from its lengths on the GPU.

    cached_lens, new_lens [B] int32: tokens in the cache and tokens this step
    adds; block_tables [B, max_blocks] int32, extended in place; free_blocks
    [num_blocks] int32 and free_state [2] int64: the ring of free blocks (blocks
    taken and put so far; the ring itself is only read).  Returns a StepPlan, in
    ``out`` when given (``StepPlan.empty``): context_lens [B], q_offsets [B+1],
    slot_mapping and positions [max_tokens] (-1 and 0 behind the last token) and
    the new free_state (out's may be the one passed in, as context_lens may be
    cached_lens).  A bad sequence (a negative length, or one past its table row) is
    flagged PA_DEV_BAD_CONTEXT and gets context 0, or keeps its length in place.  A step that does not fit
    the ring (PA_DEV_NO_BLOCKS) or max_tokens (PA_DEV_BAD_CONTEXT) plans nothing."""
    name = "pa_step_plan"
    if out is None:
        if not isinstance(cached_lens, torch.Tensor):
            raise TypeError(f"{name}: cached_lens must be a torch.Tensor")
        with torch.cuda.stream(stream):  # (None: the current one)
            out = StepPlan.empty(cached_lens.numel(), int(max_tokens), cached_lens.device)
    rc = _binding().step_plan(cached_lens, new_lens, block_tables, free_blocks, free_state, *out,
                              status, block_size, max_tokens, _handle(name, stream, free_state))
    if rc:
        i32, i64, B = torch.int32, torch.int64, _size(cached_lens, 0)
        _failed(rc, name, cached_lens,
                (("cached_lens", cached_lens, i32, (None,)), ("new_lens", new_lens, i32, (B,)),
                 ("block_tables", block_tables, i32, (B, None)),
                 ("free_blocks", free_blocks, i32, (None,)),
                 ("free_state", free_state, i64, (2,)),
                 ("out.context_lens", out[0], i32, (B,)),
                 ("out.q_offsets", out[1], i32, (None if B is None else B + 1,)),
                 ("out.slot_mapping", out[2], i64, (max_tokens,)),
                 ("out.positions", out[3], i32, (max_tokens,)),
                 ("out.free_state", out[4], i64, (2,))), status=status)
    return out


def pa_rope_table(inv_freq, axes=None, device=None):
    """The table pa_rope_cache_write turns pairs by: int64 [rotary_dim / 2] on
    ``device`` from inv_freq (radians a position, float64) and the axis of each
    pair (0..3; None: all 0).  Built on the host, once for a model."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64).cpu().contiguous()
    ax = None if axes is None else torch.as_tensor(axes).to("cpu", torch.int32).contiguous()
    if f.dim() != 1 or (ax is not None and ax.shape != f.shape):
        raise ValueError("inv_freq and axes must be one-dimensional and of the same length")
    table = torch.empty(f.shape[0], dtype=torch.int64)
    _check(lib().pa_rope_table(_ptr(f), _ptr(ax), f.shape[0], _ptr(table)), "pa_rope_table")
    return table if device is None else table.to(device)


def pa_rope_cache_write(q, k, v, positions, table, slot_mapping, k_cache=None, v_cache=None,
                        interleaved=False, q_out=None, k_out=None, status=None, stream=None):
    """Rotates q [T,H,D] and k [T,Hkv,D] and writes the rotated k and v to the
    paged cache [num_blocks, block_size, Hkv, D] at slot_mapping [T] int64 (-1:
    not written).  positions [n_axes, T] (or [T]) int32; table from pa_rope_table;
    pairs are (i, i + rotary_dim/2), or (2i, 2i+1) with ``interleaved``.  q, k, v
    may be views of one projection's output (a token's heads contiguous).  Returns
    (q_out, k_out); q_out is allocated when not given and may be q; k_out, given
    or with no cache allocated, receives the rotated keys and may be k."""
    name = "pa_rope_cache_write"
    cache = k_cache is not None or v_cache is not None
    if q_out is None:
        if not isinstance(q, torch.Tensor):
            raise TypeError(f"{name}: q must be a torch.Tensor")
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    if not cache:
        v = slot_mapping = None
        if k_out is None:
            if not isinstance(k, torch.Tensor):
                raise TypeError(f"{name}: k must be a torch.Tensor")
            k_out = _empty(k.shape, k.dtype, k.device, stream)
    rc = _binding().rope_cache_write(q, k, v, positions, table, slot_mapping, k_cache, v_cache,
                                     q_out, k_out, status, interleaved, _handle(name, stream, q))
    if rc:
        T, D, Hkv = _size(q, 0), _size(q, 2), _size(k, 1)
        one = isinstance(positions, torch.Tensor) and positions.dim() == 1
        dense = [("positions", positions, torch.int32, (T,) if one else (None, T)),
                 ("table", table, torch.int64, (None,))]
        strided = [("q", q, None, (None, None, None)), ("k", k, None, (T, None, D)),
                   ("q_out", q_out, None, (T, _size(q, 1), D))]
        if k_out is not None:
            strided.append(("k_out", k_out, None, (T, Hkv, D)))
        if cache:
            pool = (_size(k_cache, 0), _size(k_cache, 1), Hkv, D)
            strided.append(("v", v, None, (T, Hkv, D)))
            dense += [("k_cache", k_cache, None, pool), ("v_cache", v_cache, None, pool),
                      ("slot_mapping", slot_mapping, torch.int64, (T,))]
        _failed(rc, name, q, dense, strided, status)
    return q_out, k_out


def pa_prompt_attention(q, k, v, q_offsets, scale, out=None, status=None, stream=None):
    """Causal attention of packed prompts over their own rows.  q [T,H,D], k and
    v [T,Hkv,D] (views of one projection's output are fine), q_offsets [B+1]
    int32: sequence b is rows q_offsets[b] .. q_offsets[b+1]-1.  Returns ``out``
    [T,H,D]; rows outside the sequences are left as they were (undefined when
    ``out`` is allocated here)."""
    name = "pa_prompt_attention"
    if out is None:
        if not isinstance(q, torch.Tensor):
            raise TypeError(f"{name}: q must be a torch.Tensor")
        out = _empty(q.shape, q.dtype, q.device, stream)
    rc = _binding().prompt_attention(q, k, v, q_offsets, out, status, scale,
                                     _handle(name, stream, q))
    if rc:
        T, H, D, Hkv = _size(q, 0), _size(q, 1), _size(q, 2), _size(k, 1)
        _failed(rc, name, q, (("q_offsets", q_offsets, torch.int32, (None,)),
                              ("out", out, None, (T, H, D))),
                (("q", q, None, (None, None, None)), ("k", k, None, (T, None, D)),
                 ("v", v, None, (T, Hkv, D))), status)
    return out


def pa_chunk_attention_workspace_size(B, T, H, Hkv, D, max_context_len):
    """Bytes of workspace pa_chunk_attention uses on the current device."""
    return lib().pa_chunk_attention_workspace_size(B, T, H, Hkv, D, max_context_len)


def pa_chunk_attention(q, k_cache, v_cache, block_tables, context_lens, q_offsets, scale,
                       max_context_len=None, out=None, workspace=None, split=True, status=None,
                       stream=None):
    """Attention of packed chunks over the paged cache with grouped heads.  q
    [T,H,D]; caches [NB,bs,Hkv,D]; sequence b's rows q_offsets[b] ..
    q_offsets[b+1]-1 are its last positions of context_lens[b] and attend to
    everything up to themselves.  ``max_context_len`` bounds the contexts (None:
    what the tables hold).  A workspace for the split of long contexts is
    allocated when not given; split=False passes none.  Returns ``out``
    [T,H,D]; rows outside the sequences are left as they were."""
    name = "pa_chunk_attention"
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"{name}: q must be a torch.Tensor")
    if max_context_len is None:
        max_context_len = (_size(block_tables, 1) or 0) * (_size(k_cache, 1) or 0)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    own = split and workspace is None  # (allocated by the binding)
    if not split:
        workspace = None
    rc = _binding().chunk_attention(q, k_cache, v_cache, block_tables, context_lens, q_offsets,
                                    out, own or workspace, status, max_context_len, scale,
                                    _handle(name, stream, q))
    if rc:
        B = None if _size(q_offsets, 0) is None else q_offsets.shape[0] - 1
        _failed(rc, name, q,
                (("q_offsets", q_offsets, torch.int32, (None,)),
                 *_cache_args(q, k_cache, v_cache, block_tables, context_lens, B),
                 ("out", out, None, tuple(q.shape)), *_workspace_arg(workspace)),
                (("q", q, None, (None, None, None)),), status)
    return out


def _cache_args(q, k_cache, v_cache, block_tables, context_lens, B):
    pool = (_size(k_cache, 0), _size(k_cache, 1), _size(k_cache, 2), _size(q, 2))
    return (("k_cache", k_cache, None, pool), ("v_cache", v_cache, None, pool),
            ("block_tables", block_tables, torch.int32, (B, None)),
            ("context_lens", context_lens, torch.int32, (B,)))


def _workspace_arg(workspace):
    if workspace is None:
        return ()
    if not isinstance(workspace, torch.Tensor):
        return (("workspace", workspace, None, ()),)
    return (("workspace", workspace, workspace.dtype, tuple(workspace.shape)),)


def pa_decode_grouped_workspace_size(B, H, Hkv, D, block_size, max_context_len,
                                     partition_tokens=0):
    """Bytes of workspace pa_decode_grouped needs on the current device."""
    return lib().pa_decode_grouped_workspace_size(B, H, Hkv, D, block_size, max_context_len,
                                                  partition_tokens)


def pa_decode_grouped(q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                      out=None, partition_tokens=0, workspace=None, status=None, stream=None):
    """Paged decode attention with grouped heads: q [B,H,D] (fp16 or bf16), caches
    [NB,bs,Hkv,D] of the same type, ``max_context_len`` a host-side bound on
    context_lens.  Returns ``out`` [B,H,D]."""
    name = "pa_decode_grouped"
    if out is None:
        if not isinstance(q, torch.Tensor):
            raise TypeError(f"{name}: q must be a torch.Tensor")
        out = _empty(q.shape, q.dtype, q.device, stream)
    rc = _binding().decode_grouped(q, k_cache, v_cache, block_tables, context_lens, out,
                                   workspace, status, max_context_len, partition_tokens, scale,
                                   _handle(name, stream, q))
    if rc:
        _failed(rc, name, q,
                (("q", q, None, (None, None, None)),
                 *_cache_args(q, k_cache, v_cache, block_tables, context_lens, _size(q, 0)),
                 ("out", out, None, tuple(_size(q, i) for i in range(3))),
                 *_workspace_arg(workspace)), (), status)
    return out
