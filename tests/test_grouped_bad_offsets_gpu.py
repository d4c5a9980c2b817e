"""Packed attention where some of the offsets are bad: the sequences that break no
rule are computed as if they were alone (bound: grouped_ref)."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import Paged, attend, check
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


# (offsets in 60 rows, the sequence that breaks no rule)
@pytest.mark.parametrize("offsets,good", [
    ([0, 40, -1], 0), ([0, 40, 20], 0), ([70, 20, 60], 1), ([0, 500, 20, 60], 2),
    ([20, 60, 59, 70], 0), ([-3, 20, 60], 1), ([0, 40, 61], 0),
])
@pytest.mark.parametrize("D", [64, 128])
def test_split_rows_beside_bad_offsets_are_merged(offsets, good, D):
    B = len(offsets) - 1
    n = 40
    qlens = [n if b == good else 0 for b in range(B)]
    p = Paged([3000] * B, qlens, 8, 2, D, 16, torch.bfloat16, seed=B, before=offsets[good],
              behind=60 - n - offsets[good])
    p.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    ref, tol = attend(p.q[offsets[good]:offsets[good] + n], p.keys[good], p.values[good], p.scale,
                      3000 - n)
    ws = pk.pa_chunk_attention_workspace_size(B, 60, 8, 2, D, p.tables.shape[1] * 16)
    assert ws > 0  # long contexts: cut into key ranges and merged
    for split in (True, False):
        status = zero_status(DEV)
        out = torch.full_like(p.q, 7.0)
        pk.pa_chunk_attention(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.offsets, p.scale,
                              out=out, split=split, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == pk.PA_DEV_BAD_CONTEXT
        rows = slice(offsets[good], offsets[good] + n)
        check(out[rows], ref, tol, f"split {split}")
        out[rows] = 7.0
        assert (out == 7).all()  # nobody else's rows are touched


@pytest.mark.parametrize("paged", [False, True])
def test_overlapping_sequences_are_flagged_and_bounded(paged):
    # sequences over the same rows have more units than T rows can: the call ends (with what
    # it leaves in their rows undefined), keeps to its rows and harms no later call
    T, n, H, Hkv, D, bs = 3000, 40, 8, 2, 64, 8
    M = T // bs
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).half() for h in (H, Hkv, Hkv))
    for offsets in ([n] + [T, n] * 50, [0, n]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        B = len(offsets) - 1
        status = zero_status(DEV)
        out = torch.full_like(q, 7.0)
        if paged:  # every sequence on the same blocks
            tables = torch.arange(M, dtype=torch.int32, device=DEV).repeat(B, 1)
            context = torch.full((B,), T if B > 1 else n, dtype=torch.int32, device=DEV)
            pk.pa_chunk_attention(q, k.view(M, bs, Hkv, D), v.view(M, bs, Hkv, D), tables, context,
                                  off, D ** -0.5, out=out, status=status)
        else:
            pk.pa_prompt_attention(q, k, v, off, D ** -0.5, out=out, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == (pk.PA_DEV_BAD_CONTEXT if B > 1 else 0)
        assert (out[:n] == 7).all() if B > 1 else (out[n:] == 7).all()
    ref, tol = attend(q[:n], k[:n], v[:n], D ** -0.5, 0)
    check(out[:n], ref, tol)
