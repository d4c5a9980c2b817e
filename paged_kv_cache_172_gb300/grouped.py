"""ctypes binding of a serving step with grouped K/V heads (include/pagedkv.h):
step plan, rotary cache write, prompt attention, chunk attention and grouped
decode, on packed tokens in fp16 or bf16.

Argument marshalling only, as in ``_lib``: every step runs in the library's
CUDA kernels.  Single-token calls are as short as their launches, so the
checks here are kept to plain attribute reads.
"""
import ctypes
from typing import NamedTuple

import torch

from ._lib import _check, _ptr, _stream, lib

_DTYPE = {torch.float16: 0, torch.bfloat16: 1}  # pa_dtype


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


def _same_device(name, first, *rest):
    dev = first.device
    for t in rest:
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: tensors on different devices: {dev}, {t.device}")
    return dev


def _run(fn, name, dev, stream, *args):
    """Calls the library with the tensors' device current (its launches go to the
    current device) on ``stream`` or that device's current stream."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"{name}: stream on {stream.device}, tensors on {dev}")
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(stream, dev))
    else:
        rc = fn(*args, _stream(stream, dev))
    if rc:
        _check(rc, name)


def _dense(t, dtype, name, *shape):
    """A contiguous CUDA tensor of that type; -1 in ``shape`` takes any size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != len(shape) or any(n not in (-1, m) for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {list(shape)} (-1: any), got {list(t.shape)}")


def _rows(t, dtype, name, *shape):
    """A [T, heads, D] CUDA tensor whose tokens' heads are contiguous; the
    distance between tokens in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or dtype not in _DTYPE:
        raise TypeError(f"{name} must be {dtype if dtype in _DTYPE else 'fp16 or bf16'}, "
                        f"got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dim() != 3 or any(n not in (-1, m) for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {list(shape)} (-1: any), got {list(t.shape)}")
    T, heads, D = t.shape
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return st[0] if T > 1 else heads * D


def _status(status):
    if status is not None and (status.dtype != torch.int32 or not status.is_cuda):
        raise TypeError("status must be a CUDA int32 tensor")
    return _ptr(status)


def pa_step_plan(cached_lens, new_lens, block_tables, free_blocks, free_state, block_size,
                 max_tokens, out=None, status=None, stream=None):
    """Block tables, slots and positions of a step, from its lengths on the GPU.

    cached_lens, new_lens [B] int32: tokens in the cache and tokens this step
    adds; block_tables [B, max_blocks] int32, extended in place; free_blocks
    [num_blocks] int32 and free_state [2] int64: the ring of free blocks (blocks
    taken and put so far; the ring itself is only read).  Returns a StepPlan, in
    ``out`` when given (``StepPlan.empty``): context_lens [B], q_offsets [B+1],
    slot_mapping and positions [max_tokens] (-1 and 0 behind the last token) and
    the new free_state (out's may be the one passed in).  A step that does not fit
    the ring (PA_DEV_NO_BLOCKS) or max_tokens (PA_DEV_BAD_CONTEXT) plans nothing."""
    _dense(cached_lens, torch.int32, "cached_lens", -1)
    B = cached_lens.shape[0]
    _dense(new_lens, torch.int32, "new_lens", B)
    _dense(block_tables, torch.int32, "block_tables", B, -1)
    _dense(free_blocks, torch.int32, "free_blocks", -1)
    _dense(free_state, torch.int64, "free_state", 2)
    max_tokens = int(max_tokens)
    if out is None:
        out = StepPlan.empty(B, max_tokens, cached_lens.device)
    else:
        _dense(out.context_lens, torch.int32, "out.context_lens", B)
        _dense(out.q_offsets, torch.int32, "out.q_offsets", B + 1)
        _dense(out.slot_mapping, torch.int64, "out.slot_mapping", max_tokens)
        _dense(out.positions, torch.int32, "out.positions", max_tokens)
        _dense(out.free_state, torch.int64, "out.free_state", 2)
    dev = _same_device("pa_step_plan", cached_lens, new_lens, block_tables, free_blocks,
                       free_state, *out, status)
    _run(lib().pa_step_plan, "pa_step_plan", dev, stream, _ptr(cached_lens), _ptr(new_lens), B,
         int(block_size), free_blocks.shape[0], block_tables.shape[1], max_tokens,
         _ptr(free_blocks), _ptr(free_state), _ptr(block_tables), _ptr(out.context_lens),
         _ptr(out.q_offsets), _ptr(out.slot_mapping), _ptr(out.positions), _ptr(out.free_state),
         _status(status))
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
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dt = q.dtype
    qs = _rows(q, dt, "q", -1, -1, -1)
    T, H, D = q.shape
    ks = _rows(k, dt, "k", T, -1, D)
    Hkv = k.shape[1]
    if positions.dim() == 1:
        positions = positions[None]
    _dense(positions, torch.int32, "positions", -1, T)
    _dense(table, torch.int64, "table", -1)
    NB = bs = vs = 0
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache are given together")
    if k_cache is not None:
        vs = _rows(v, dt, "v", T, Hkv, D)
        _dense(k_cache, dt, "k_cache", -1, -1, Hkv, D)
        NB, bs = k_cache.shape[:2]
        _dense(v_cache, dt, "v_cache", NB, bs, Hkv, D)
        _dense(slot_mapping, torch.int64, "slot_mapping", T)
    else:
        v = slot_mapping = None
        if k_out is None:
            k_out = torch.empty((T, Hkv, D), dtype=dt, device=q.device)
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=dt, device=q.device)
    qos = _rows(q_out, dt, "q_out", T, H, D)
    kos = 0 if k_out is None else _rows(k_out, dt, "k_out", T, Hkv, D)
    dev = _same_device("pa_rope_cache_write", q, k, v, positions, table, slot_mapping, k_cache,
                       v_cache, q_out, k_out, status)
    _run(lib().pa_rope_cache_write, "pa_rope_cache_write", dev, stream, _ptr(q), _ptr(k), _ptr(v),
         _ptr(positions), _ptr(table), _ptr(slot_mapping), T, H, Hkv, D, 2 * table.shape[0],
         positions.shape[0], int(bool(interleaved)), _DTYPE[dt], qs, ks, vs, bs, NB, _ptr(q_out),
         qos, _ptr(k_out), kos, _ptr(k_cache), _ptr(v_cache), _status(status))
    return q_out, k_out


def pa_prompt_attention(q, k, v, q_offsets, scale, out=None, status=None, stream=None):
    """Causal attention of packed prompts over their own rows.  q [T,H,D], k and
    v [T,Hkv,D] (views of one projection's output are fine), q_offsets [B+1]
    int32: sequence b is rows q_offsets[b] .. q_offsets[b+1]-1.  Returns ``out``
    [T,H,D]; rows outside the sequences are left as they were (undefined when
    ``out`` is allocated here)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dt = q.dtype
    qs = _rows(q, dt, "q", -1, -1, -1)
    T, H, D = q.shape
    ks = _rows(k, dt, "k", T, -1, D)
    Hkv = k.shape[1]
    vs = _rows(v, dt, "v", T, Hkv, D)
    _dense(q_offsets, torch.int32, "q_offsets", -1)
    B = q_offsets.shape[0] - 1
    if out is None:
        out = torch.empty((T, H, D), dtype=dt, device=q.device)
    else:
        _dense(out, dt, "out", T, H, D)
    dev = _same_device("pa_prompt_attention", q, k, v, q_offsets, out, status)
    _run(lib().pa_prompt_attention, "pa_prompt_attention", dev, stream, _ptr(q), _ptr(k),
         _ptr(v), _ptr(q_offsets), B, T, H, Hkv, D, _DTYPE[dt], qs, ks, vs, float(scale),
         _ptr(out), _status(status))
    return out


def _cache(dt, D, k_cache, v_cache, block_tables, context_lens, B):
    """(num_blocks, block_size, Hkv, max_blocks) of a checked paged cache."""
    _dense(k_cache, dt, "k_cache", -1, -1, -1, D)
    NB, bs, Hkv, _ = k_cache.shape
    _dense(v_cache, dt, "v_cache", NB, bs, Hkv, D)
    _dense(block_tables, torch.int32, "block_tables", B, -1)
    _dense(context_lens, torch.int32, "context_lens", B)
    return NB, bs, Hkv, block_tables.shape[1]


def _workspace(workspace, nbytes, device):
    """(tensor, bytes) of the given workspace, or of a new one where one is needed."""
    if workspace is None:
        if nbytes == 0:
            return None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


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
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dt = q.dtype
    qs = _rows(q, dt, "q", -1, -1, -1)
    T, H, D = q.shape
    _dense(q_offsets, torch.int32, "q_offsets", -1)
    B = q_offsets.shape[0] - 1
    NB, bs, Hkv, M = _cache(dt, D, k_cache, v_cache, block_tables, context_lens, B)
    cap = M * bs if max_context_len is None else int(max_context_len)
    if out is None:
        out = torch.empty((T, H, D), dtype=dt, device=q.device)
    else:
        _dense(out, dt, "out", T, H, D)
    dev = _same_device("pa_chunk_attention", q, k_cache, v_cache, block_tables, context_lens,
                       q_offsets, out, workspace, status)
    ws, ws_bytes = None, 0
    if split:
        need = 0
        if workspace is None:
            with torch.cuda.device(dev):
                need = pa_chunk_attention_workspace_size(B, T, H, Hkv, D, cap)
        ws, ws_bytes = _workspace(workspace, need, dev)
    _run(lib().pa_chunk_attention, "pa_chunk_attention", dev, stream, _ptr(q), _ptr(k_cache),
         _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), _ptr(q_offsets), B, T, H, Hkv, D,
         _DTYPE[dt], qs, bs, NB, M, cap, float(scale), _ptr(out), _ptr(ws), ws_bytes,
         _status(status))
    return out


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
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dt = q.dtype
    if dt not in _DTYPE:
        raise TypeError(f"q must be fp16 or bf16, got {dt}")
    _dense(q, dt, "q", -1, -1, -1)
    B, H, D = q.shape
    NB, bs, Hkv, M = _cache(dt, D, k_cache, v_cache, block_tables, context_lens, B)
    cap = int(max_context_len)
    if out is None:
        out = torch.empty_like(q)
    else:
        _dense(out, dt, "out", B, H, D)
    dev = _same_device("pa_decode_grouped", q, k_cache, v_cache, block_tables, context_lens, out,
                       workspace, status)
    need = 0
    if workspace is None:
        with torch.cuda.device(dev):
            need = pa_decode_grouped_workspace_size(B, H, Hkv, D, bs, cap, partition_tokens)
    ws, ws_bytes = _workspace(workspace, need, dev)
    _run(lib().pa_decode_grouped, "pa_decode_grouped", dev, stream, _ptr(q), _ptr(k_cache),
         _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), B, H, Hkv, D, _DTYPE[dt], bs, NB,
         M, cap, int(partition_tokens), float(scale), _ptr(out), _ptr(ws), ws_bytes,
         _status(status))
    return out
