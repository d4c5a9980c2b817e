"""ctypes binding of a serving step with grouped K/V heads (include/pagedkv.h):
step plan, rotary cache write, prompt attention, chunk attention and grouped
decode, on packed tokens in fp16 or bf16.

Argument marshalling only, as in ``_lib``: every step runs in the library's
CUDA kernels.  The kernels of a single-token step take 2 to 6 us, less than
a call's argument checks written out one by one (about 20 us of host time), so
each call tests all its arguments in one expression and looks for the one to
complain about only when that fails.
"""
from typing import NamedTuple

import torch

from ._lib import _check, _ptr, lib

_DTYPE = {torch.float16: 0, torch.bfloat16: 1}  # pa_dtype
# The current stream's handle without a torch.cuda.Stream object around it, and
# the current device (tensors on one exist: CUDA is initialised).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


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


def _run(fn, name, dev, stream, *args):
    """Calls the library with the tensors' device current (its launches go to the
    current device) on ``stream`` or that device's current stream."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{name}: stream on {stream.device}, tensors on cuda:{dev}")
        handle = stream.cuda_stream
    else:
        handle = _raw_stream(dev)
    if dev == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        _check(rc, name)


def _empty(shape, dtype, device, stream):
    """A new tensor from the pool of the stream that the call runs on: one of
    another stream's pool could still be in use there, or be handed out again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dense(t, dtype, shape, dev):
    """Whether t is a contiguous tensor of that type and shape on device dev."""
    return (t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev)


def _rows(t, dtype, shape, dev):
    """Whether t is [T, heads, D] on device dev with a token's heads contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        return False
    st = t.stride()
    return st[2] == 1 and (st[1] == shape[2] or shape[1] == 1)


def _stride(t):
    """Distance between tokens in elements (any for a single token)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _status_ok(status, dev):
    return status is None or (status.dtype is torch.int32 and status.get_device() == dev)


def _misshaped(name, *tensors):
    """The error behind sizes that could not be read off: (name, tensor, dims)."""
    for what, t, dims in tensors:
        if not isinstance(t, torch.Tensor):
            return TypeError(f"{name}: {what} must be a torch.Tensor")
        if t.dim() != dims:
            return ValueError(f"{name}: {what} must have {dims} dims, got {list(t.shape)}")
    return ValueError(f"{name}: bad shapes")


def _complain(name, dev, dense, rows=(), status=None):
    """Raises the error of the first argument that a call's test found wrong.
    dense, rows: (name, tensor or None, dtype, shape)."""
    for strided, group in ((False, dense), (True, rows)):
        for what, t, dtype, shape in group:
            if t is None:
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: {what} must be a torch.Tensor")
            if t.dtype != dtype:
                raise TypeError(f"{name}: {what} must be {dtype}, got {t.dtype}")
            if not t.is_cuda:
                raise ValueError(f"{name}: {what} must be on a CUDA device")
            if t.get_device() != dev:
                raise ValueError(f"{name}: {what} is on {t.device}, others on cuda:{dev}")
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name}: {what} must be {list(shape)}, got {list(t.shape)}")
            if not strided and not t.is_contiguous():
                raise ValueError(f"{name}: {what} must be contiguous")
            if strided and not _rows(t, dtype, shape, dev):
                raise ValueError(f"{name}: a token's heads must be contiguous in {what}")
    if not _status_ok(status, dev):
        raise TypeError(f"{name}: status must be int32 on the tensors' device")
    raise ValueError(f"{name}: bad arguments")


def _float16(name, q):
    """pa_dtype of q, the tensor that sets a call's type."""
    if q.dtype not in _DTYPE:
        raise TypeError(f"{name}: q must be fp16 or bf16, got {q.dtype}")
    return _DTYPE[q.dtype]


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
    i32, i64 = torch.int32, torch.int64
    try:
        (B,), (_, M), (NB,), T = (cached_lens.shape, block_tables.shape, free_blocks.shape,
                                  int(max_tokens))
    except (AttributeError, ValueError):
        raise _misshaped("pa_step_plan", ("cached_lens", cached_lens, 1),
                         ("block_tables", block_tables, 2),
                         ("free_blocks", free_blocks, 1)) from None
    dev = cached_lens.get_device()
    if out is None:
        with torch.cuda.stream(stream):  # (None: the current one)
            out = StepPlan.empty(B, T, cached_lens.device)
    ctx, offs, slots, pos, state = out
    one = (B,)
    if not (dev >= 0 and _dense(cached_lens, i32, one, dev) and _dense(new_lens, i32, one, dev)
            and _dense(block_tables, i32, (B, M), dev) and _dense(free_blocks, i32, (NB,), dev)
            and _dense(free_state, i64, (2,), dev) and _dense(ctx, i32, one, dev)
            and _dense(offs, i32, (B + 1,), dev) and _dense(slots, i64, (T,), dev)
            and _dense(pos, i32, (T,), dev) and _dense(state, i64, (2,), dev)
            and _status_ok(status, dev)):
        _complain("pa_step_plan", dev,
                  (("cached_lens", cached_lens, i32, one), ("new_lens", new_lens, i32, one),
                   ("block_tables", block_tables, i32, (B, M)),
                   ("free_blocks", free_blocks, i32, (NB,)), ("free_state", free_state, i64, (2,)),
                   ("out.context_lens", ctx, i32, one), ("out.q_offsets", offs, i32, (B + 1,)),
                   ("out.slot_mapping", slots, i64, (T,)), ("out.positions", pos, i32, (T,)),
                   ("out.free_state", state, i64, (2,))), status=status)
    _run(lib().pa_step_plan, "pa_step_plan", dev, stream, cached_lens.data_ptr(),
         new_lens.data_ptr(), B, int(block_size), NB, M, T, free_blocks.data_ptr(),
         free_state.data_ptr(), block_tables.data_ptr(), ctx.data_ptr(), offs.data_ptr(),
         slots.data_ptr(), pos.data_ptr(), state.data_ptr(),
         None if status is None else status.data_ptr())
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
    try:
        (T, H, D), (_, Hkv, _), (n,) = q.shape, k.shape, table.shape
    except (AttributeError, ValueError):
        raise _misshaped(name, ("q", q, 3), ("k", k, 3), ("table", table, 1)) from None
    code, dt, dev = _float16(name, q), q.dtype, q.get_device()
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    pos_shape = (T,) if positions.dim() == 1 else (axes, T)
    kv, caches = (T, Hkv, D), ()
    NB = bs = 0
    if k_cache is not None or v_cache is not None:
        try:
            (NB, bs, _, _), (_, _, _) = k_cache.shape, v.shape
        except (AttributeError, ValueError):
            raise _misshaped(name, ("k_cache", k_cache, 4), ("v", v, 3)) from None
        caches = (NB, bs, Hkv, D)
    else:
        v = slot_mapping = None
        if k_out is None:
            k_out = _empty(kv, dt, q.device, stream)
    if q_out is None:
        q_out = _empty((T, H, D), dt, q.device, stream)
    if not (dev >= 0 and _rows(q, dt, (T, H, D), dev) and _rows(k, dt, kv, dev)
            and _dense(positions, torch.int32, pos_shape, dev)
            and _dense(table, torch.int64, (n,), dev) and _rows(q_out, dt, (T, H, D), dev)
            and (k_out is None or _rows(k_out, dt, kv, dev))
            and (not caches or (_rows(v, dt, kv, dev) and _dense(k_cache, dt, caches, dev)
                                and v_cache is not None and _dense(v_cache, dt, caches, dev)
                                and slot_mapping is not None
                                and _dense(slot_mapping, torch.int64, (T,), dev)))
            and _status_ok(status, dev)):
        if caches and (v_cache is None or slot_mapping is None):
            raise ValueError(f"{name}: the cache write needs k_cache, v_cache and slot_mapping")
        _complain(name, dev,
                  (("positions", positions, torch.int32, pos_shape),
                   ("table", table, torch.int64, (n,)), ("k_cache", k_cache, dt, caches),
                   ("v_cache", v_cache, dt, caches),
                   ("slot_mapping", slot_mapping, torch.int64, (T,))),
                  (("q", q, dt, (T, H, D)), ("k", k, dt, kv), ("v", v, dt, kv),
                   ("q_out", q_out, dt, (T, H, D)), ("k_out", k_out, dt, kv)), status)
    _run(lib().pa_rope_cache_write, name, dev, stream, q.data_ptr(), k.data_ptr(),
         v.data_ptr() if caches else None, positions.data_ptr(), table.data_ptr(),
         slot_mapping.data_ptr() if caches else None, T, H, Hkv, D, 2 * n, axes,
         1 if interleaved else 0, code, _stride(q), _stride(k), _stride(v) if caches else 0, bs,
         NB, q_out.data_ptr(), _stride(q_out), None if k_out is None else k_out.data_ptr(),
         0 if k_out is None else _stride(k_out), k_cache.data_ptr() if caches else None,
         v_cache.data_ptr() if caches else None, None if status is None else status.data_ptr())
    return q_out, k_out


def pa_prompt_attention(q, k, v, q_offsets, scale, out=None, status=None, stream=None):
    """Causal attention of packed prompts over their own rows.  q [T,H,D], k and
    v [T,Hkv,D] (views of one projection's output are fine), q_offsets [B+1]
    int32: sequence b is rows q_offsets[b] .. q_offsets[b+1]-1.  Returns ``out``
    [T,H,D]; rows outside the sequences are left as they were (undefined when
    ``out`` is allocated here)."""
    name = "pa_prompt_attention"
    try:
        (T, H, D), (_, Hkv, _), (_, _, _), (n,) = q.shape, k.shape, v.shape, q_offsets.shape
    except (AttributeError, ValueError):
        raise _misshaped(name, ("q", q, 3), ("k", k, 3), ("v", v, 3),
                         ("q_offsets", q_offsets, 1)) from None
    code, dt, dev = _float16(name, q), q.dtype, q.get_device()
    if out is None:
        out = _empty((T, H, D), dt, q.device, stream)
    if not (dev >= 0 and _rows(q, dt, (T, H, D), dev) and _rows(k, dt, (T, Hkv, D), dev)
            and _rows(v, dt, (T, Hkv, D), dev) and _dense(q_offsets, torch.int32, (n,), dev)
            and _dense(out, dt, (T, H, D), dev) and _status_ok(status, dev)):
        _complain(name, dev, (("q_offsets", q_offsets, torch.int32, (n,)),
                              ("out", out, dt, (T, H, D))),
                  (("q", q, dt, (T, H, D)), ("k", k, dt, (T, Hkv, D)),
                   ("v", v, dt, (T, Hkv, D))), status)
    _run(lib().pa_prompt_attention, name, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
         q_offsets.data_ptr(), n - 1, T, H, Hkv, D, code, _stride(q), _stride(k), _stride(v),
         scale, out.data_ptr(), None if status is None else status.data_ptr())
    return out


def _workspace(name, workspace, nbytes, dev, stream):
    """(address, bytes, owner) of the given workspace, or of a new one of nbytes."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = _empty(nbytes, torch.uint8, f"cuda:{dev}", stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be contiguous and on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _sized(fn, dev, *args):
    """A workspace size, which depends on the device, with that device current."""
    if dev == _current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


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
    try:
        (T, H, D), (NB, bs, Hkv, _), (_, M), (n,) = (q.shape, k_cache.shape, block_tables.shape,
                                                     q_offsets.shape)
    except (AttributeError, ValueError):
        raise _misshaped(name, ("q", q, 3), ("k_cache", k_cache, 4),
                         ("block_tables", block_tables, 2), ("q_offsets", q_offsets, 1)) from None
    code, dt, dev = _float16(name, q), q.dtype, q.get_device()
    B, pool = n - 1, (NB, bs, Hkv, D)
    cap = M * bs if max_context_len is None else int(max_context_len)
    if out is None:
        out = _empty((T, H, D), dt, q.device, stream)
    if not (dev >= 0 and _rows(q, dt, (T, H, D), dev) and _dense(k_cache, dt, pool, dev)
            and _dense(v_cache, dt, pool, dev) and _dense(block_tables, torch.int32, (B, M), dev)
            and _dense(context_lens, torch.int32, (B,), dev)
            and _dense(q_offsets, torch.int32, (n,), dev) and _dense(out, dt, (T, H, D), dev)
            and _status_ok(status, dev)):
        _complain(name, dev, (("k_cache", k_cache, dt, pool), ("v_cache", v_cache, dt, pool),
                              ("block_tables", block_tables, torch.int32, (B, M)),
                              ("context_lens", context_lens, torch.int32, (B,)),
                              ("q_offsets", q_offsets, torch.int32, (n,)),
                              ("out", out, dt, (T, H, D))), (("q", q, dt, (T, H, D)),), status)
    ws, ws_bytes = None, 0
    if split:
        need = 0 if workspace is not None else _sized(pa_chunk_attention_workspace_size, dev, B,
                                                      T, H, Hkv, D, cap)
        ws, ws_bytes, workspace = _workspace(name, workspace, need, dev, stream)
    _run(lib().pa_chunk_attention, name, dev, stream, q.data_ptr(), k_cache.data_ptr(),
         v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
         q_offsets.data_ptr(), B, T, H, Hkv, D, code, _stride(q), bs, NB, M, cap, scale,
         out.data_ptr(), ws, ws_bytes, None if status is None else status.data_ptr())
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
    name = "pa_decode_grouped"
    try:
        (B, H, D), (NB, bs, Hkv, _), (_, M) = q.shape, k_cache.shape, block_tables.shape
    except (AttributeError, ValueError):
        raise _misshaped(name, ("q", q, 3), ("k_cache", k_cache, 4),
                         ("block_tables", block_tables, 2)) from None
    code, dt, dev = _float16(name, q), q.dtype, q.get_device()
    pool, cap = (NB, bs, Hkv, D), int(max_context_len)
    if out is None:
        out = _empty((B, H, D), dt, q.device, stream)
    if not (dev >= 0 and _dense(q, dt, (B, H, D), dev) and _dense(k_cache, dt, pool, dev)
            and _dense(v_cache, dt, pool, dev) and _dense(block_tables, torch.int32, (B, M), dev)
            and _dense(context_lens, torch.int32, (B,), dev) and _dense(out, dt, (B, H, D), dev)
            and _status_ok(status, dev)):
        _complain(name, dev, (("q", q, dt, (B, H, D)), ("k_cache", k_cache, dt, pool),
                              ("v_cache", v_cache, dt, pool),
                              ("block_tables", block_tables, torch.int32, (B, M)),
                              ("context_lens", context_lens, torch.int32, (B,)),
                              ("out", out, dt, (B, H, D))), (), status)
    need = 0 if workspace is not None else _sized(pa_decode_grouped_workspace_size, dev, B, H,
                                                  Hkv, D, bs, cap, partition_tokens)
    ws, ws_bytes, workspace = _workspace(name, workspace, need, dev, stream)
    _run(lib().pa_decode_grouped, name, dev, stream, q.data_ptr(), k_cache.data_ptr(),
         v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), B, H, Hkv, D, code,
         bs, NB, M, cap, partition_tokens, scale, out.data_ptr(), ws, ws_bytes,
         None if status is None else status.data_ptr())
    return out
