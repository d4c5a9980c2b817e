"""Beam search over the paged cache (include/pagedkv.h): the best continuations over
beams and vocabulary, block tables that follow the beams, and the way back to the
hypotheses' tokens.

Argument marshalling only, through the compiled binding of ``grouped``: every step
runs in the library's CUDA kernels.
"""
from typing import NamedTuple

import torch

from ._lib import lib
from .grouped import _HALF, _binding, _empty, _failed, _handle, _size, _workspace_arg


class BeamStep(NamedTuple):
    """What pa_beam_select writes, [batch, beams] each."""
    tokens: torch.Tensor        # int32
    parents: torch.Tensor       # int32
    scores: torch.Tensor        # float32
    ended_scores: torch.Tensor  # float32, by beam before the step

    @classmethod
    def empty(cls, batch, beams, device):
        def new(dtype):
            return torch.empty(batch, beams, dtype=dtype, device=device)
        return cls(new(torch.int32), new(torch.int32), new(torch.float32), new(torch.float32))


class BeamTables(NamedTuple):
    """What pa_beam_reorder writes besides the ring."""
    block_tables: torch.Tensor  # [batch * beams, max_blocks] int32
    context_lens: torch.Tensor  # [batch * beams] int32
    free_state: torch.Tensor    # [2] int64
    copy_pairs: torch.Tensor    # [batch * beams, 2] int64

    @classmethod
    def empty(cls, rows, max_blocks, device):
        def new(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=device)
        return cls(new(rows, max_blocks, dtype=torch.int32), new(rows, dtype=torch.int32),
                   new(2, dtype=torch.int64), new(rows, 2, dtype=torch.int64))


def pa_beam_select_workspace_size(B, W, V):
    """Bytes of workspace pa_beam_select needs on the current device."""
    return lib().pa_beam_select_workspace_size(B, W, V)


def pa_beam_select(logits, scores, eos_token=-1, pad_token=0, out=None, workspace=None,
                   status=None, stream=None):
    """The W best continuations of each request's W beams: logits [B*W, V] (fp32, fp16
    or bf16; rows may be apart), scores [B, W] float32 (-inf: no beam).  Returns a
    BeamStep, in ``out`` when given (its scores may be the ones passed in, tokens and
    parents slices of a history): tokens and parents of the next beams, best first,
    their scores, and by beam the score of its end with ``eos_token`` where that is
    better than the last of them (-inf elsewhere).  Places that nothing fills hold
    ``pad_token``, their own index and -inf.  A beam with NaN or +inf among its logits
    gives no candidate and is flagged."""
    name = "pa_beam_select"
    if out is None:
        if not isinstance(scores, torch.Tensor):
            raise TypeError(f"{name}: scores must be a torch.Tensor")
        if scores.dim() != 2:
            raise ValueError(f"{name}: scores must be [batch, beams], got {list(scores.shape)}")
        with torch.cuda.stream(stream):  # (None: the current one)
            out = BeamStep.empty(*scores.shape, scores.device)
    rc = _binding().beam_select(logits, scores, *out, workspace, status, eos_token, pad_token,
                                _handle(name, stream, logits))
    if rc:
        B, W = _size(scores, 0), _size(scores, 1)
        if not isinstance(logits, torch.Tensor):
            raise TypeError(f"{name}: logits must be a torch.Tensor")
        if logits.dtype != torch.float32 and logits.dtype not in _HALF:
            raise TypeError(f"{name}: logits must be fp32, fp16 or bf16, got {logits.dtype}")
        if not logits.is_cuda or logits.dim() != 2:
            raise ValueError(f"{name}: logits must be [batch * beams, vocabulary] on a CUDA device")
        if logits.shape[1] > 1 and logits.stride(1) != 1:
            raise ValueError(f"{name}: a row of logits must be contiguous")
        if B is not None and W is not None and logits.shape[0] != B * W:
            raise ValueError(f"{name}: logits must have {B * W} rows, got {logits.shape[0]}")
        f32, i32 = torch.float32, torch.int32
        _failed(rc, name, logits,
                (("scores", scores, f32, (None, None)), ("out.tokens", out[0], i32, (B, W)),
                 ("out.parents", out[1], i32, (B, W)), ("out.scores", out[2], f32, (B, W)),
                 ("out.ended_scores", out[3], f32, (B, W)), *_workspace_arg(workspace)), (),
                status)
    return out


def pa_beam_reorder_workspace_size(B, W, max_blocks):
    """Bytes of workspace pa_beam_reorder needs (0 for small batches)."""
    return lib().pa_beam_reorder_workspace_size(B, W, max_blocks)


def pa_beam_reorder(parents, block_tables, context_lens, free_blocks, free_state, block_size,
                    shared_lens=None, out=None, workspace=None, status=None, stream=None):
    """Block tables that follow the beams: row b*W + w becomes that of beam
    parents[b, w] (-1: the beam ends).  parents [B, W], block_tables [B*W, max_blocks],
    context_lens [B*W] int32; free_blocks [num_blocks] int32 and free_state [2] int64 the
    ring of pa_step_plan, which blocks that no beam holds any more go back to and copies
    of half-full last blocks are taken from; columns that hold the first shared_lens [B]
    tokens stay out of it.  Returns a BeamTables, in ``out`` when given (its tables,
    lengths and state may be the ones passed in); its copy_pairs [B*W, 2] go to
    pa_block_copy before the next token is written.  The beams of a request are of one
    length (of others, a half-full last block that a longer beam holds as a full one is
    not copied)."""
    name = "pa_beam_reorder"
    if out is None:
        if not isinstance(block_tables, torch.Tensor):
            raise TypeError(f"{name}: block_tables must be a torch.Tensor")
        if block_tables.dim() != 2:
            raise ValueError(f"{name}: block_tables must have 2 dims, got {block_tables.dim()}")
        with torch.cuda.stream(stream):
            out = BeamTables.empty(*block_tables.shape, block_tables.device)
    rc = _binding().beam_reorder(parents, block_tables, context_lens, free_blocks, free_state,
                                 shared_lens, *out, workspace, status, block_size,
                                 _handle(name, stream, parents))
    if rc:
        i32, i64, B, W = torch.int32, torch.int64, _size(parents, 0), _size(parents, 1)
        n = None if B is None or W is None else B * W
        M = _size(block_tables, 1)
        dense = [("parents", parents, i32, (None, None)),
                 ("block_tables", block_tables, i32, (n, None)),
                 ("context_lens", context_lens, i32, (n,)),
                 ("free_blocks", free_blocks, i32, (None,)), ("free_state", free_state, i64, (2,)),
                 ("out.block_tables", out[0], i32, (n, M)),
                 ("out.context_lens", out[1], i32, (n,)), ("out.free_state", out[2], i64, (2,)),
                 ("out.copy_pairs", out[3], i64, (n, 2)), *_workspace_arg(workspace)]
        if shared_lens is not None:
            dense.append(("shared_lens", shared_lens, i32, (B,)))
        _failed(rc, name, parents, dense, (), status)
    return out


def pa_beam_backtrack(tokens, parents, lengths, beams, pad_token=0, out=None, status=None,
                      stream=None):
    """The tokens of hypotheses: tokens and parents [S, B, W] int32 of the steps,
    lengths and beams [B, K] int32, how many tokens hypothesis k has and the beam of its
    last one.  Returns ``out`` [B, K, S] int32, ``pad_token`` behind each."""
    name = "pa_beam_backtrack"
    if out is None:
        for what, t, dims in (("tokens", tokens, 3), ("lengths", lengths, 2)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: {what} must be a torch.Tensor")
            if t.dim() != dims:
                raise ValueError(f"{name}: {what} must have {dims} dims, got {t.dim()}")
        out = _empty((*lengths.shape, tokens.shape[0]), torch.int32, tokens.device, stream)
    rc = _binding().beam_backtrack(tokens, parents, lengths, beams, out, status, pad_token,
                                   _handle(name, stream, tokens))
    if rc:
        i32 = torch.int32
        S, B, W, K = (_size(tokens, 0), _size(tokens, 1), _size(tokens, 2), _size(lengths, 1))
        _failed(rc, name, tokens,
                (("tokens", tokens, i32, (None, None, None)), ("parents", parents, i32, (S, B, W)),
                 ("lengths", lengths, i32, (B, None)), ("beams", beams, i32, (B, K)),
                 ("out", out, i32, (B, K, S))), (), status)
    return out
