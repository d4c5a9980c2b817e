"""The step plan directly followed by chunk attention, with nothing between them: the
attention starts while the plan still runs, and has to see the table entries that the
plan writes, in lines that also hold older ones."""
import numpy as np
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import attend, check
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B", [3, 40])
def test_fresh_entries_are_seen(B, captured):
    # the pool is filled beforehand, so that only the tables decide what is read; every step
    # takes other blocks, and the entries behind the last one hold a bad id until then
    H, Hkv, D, bs, M, steps = 8, 2, 64, 8, 40, 24
    n = 9  # a fresh entry or two a step
    NB = B * M
    g = torch.Generator(device=DEV).manual_seed(B)
    kc, vc = (torch.randn(NB, bs, Hkv, D, generator=g, device=DEV).half() for _ in range(2))
    q = torch.randn(B * n, H, D, generator=g, device=DEV).half()
    ring = torch.randperm(NB, generator=g, device=DEV).int()
    tables = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    state = torch.tensor([0, NB], dtype=torch.int64, device=DEV)
    new = torch.full((B,), n, dtype=torch.int32, device=DEV)
    plan = pk.StepPlan.empty(B, B * n, DEV)._replace(context_lens=lens, free_state=state)
    status = zero_status(DEV)
    outs = [torch.empty_like(q) for _ in range(steps)]

    def step(out):
        p = pk.pa_step_plan(lens, new, tables, ring, state, bs, B * n, out=plan, status=status)
        pk.pa_chunk_attention(q, kc, vc, tables, p.context_lens, p.q_offsets, D ** -0.5, out=out,
                              status=status)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for out in outs:
                step(out)
        graph.replay()
    else:
        for out in outs:
            step(out)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = tables.long().cpu().numpy()
    for i in range(0, steps, 5):
        for b in range(0, B, 7):
            ctx = (i + 1) * n
            j = np.arange(ctx)
            blk = torch.as_tensor(rows[b, j // bs], device=DEV)
            at = torch.as_tensor(j % bs, device=DEV)
            ref, tol = attend(q[b * n:(b + 1) * n], kc[blk, at], vc[blk, at], D ** -0.5, ctx - n)
            check(outs[i][b * n:(b + 1) * n], ref, tol, f"step {i} sequence {b}")


@pytest.mark.parametrize("bs", [4, 16])
def test_fresh_entries_are_seen_by_padded_chunks(bs):
    # pa_prefill_chunk, directly behind the plan: one K/V head a query head, padded rows
    B, H, D, n, steps = 12, 2, 64, 9, 12
    M = 128 // bs
    NB = B * M
    g = torch.Generator(device=DEV).manual_seed(bs)
    kc, vc = (torch.randn(NB, bs, H, D, generator=g, device=DEV).half() for _ in range(2))
    q = torch.randn(B, H, n, D, generator=g, device=DEV).half()
    ring = torch.randperm(NB, generator=g, device=DEV).int()
    tables = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    state = torch.tensor([0, NB], dtype=torch.int64, device=DEV)
    new = torch.full((B,), n, dtype=torch.int32, device=DEV)
    plan = pk.StepPlan.empty(B, B * n, DEV)._replace(context_lens=lens, free_state=state)
    status = zero_status(DEV)
    outs = []
    for _ in range(steps):
        p = pk.pa_step_plan(lens, new, tables, ring, state, bs, B * n, out=plan, status=status)
        outs.append(pk.pa_prefill_chunk(q, kc, vc, tables, p.context_lens, D ** -0.5,
                                        status=status))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = tables.long().cpu().numpy()
    for i in range(0, steps, 3):
        for b in range(0, B, 5):
            ctx = (i + 1) * n
            j = np.arange(ctx)
            blk = torch.as_tensor(rows[b, j // bs], device=DEV)
            at = torch.as_tensor(j % bs, device=DEV)
            ref, tol = attend(q[b].transpose(0, 1), kc[blk, at], vc[blk, at], D ** -0.5, ctx - n)
            check(outs[i][b].transpose(0, 1), ref, tol, f"step {i} sequence {b}")
