"""pa_step_plan at its limits: rings of nearly 2^31 blocks, bad lengths kept in place."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


@pytest.mark.parametrize("NB", [2 ** 30 + 1, 2 ** 31 - 1])
def test_rings_that_end_past_31_bits(NB):
    # the blocks of the step lie across the ring's end: head + i passes 2^31
    head, n, bs = NB - 3, 10, 4
    ring = torch.empty(NB, dtype=torch.int32, device=DEV)  # (only the entries below are read)
    ids = [11, 22, 33, 44, 55, 66, 77, 88, 99, NB - 1]
    ring[head:] = ints(ids[:3])
    ring[:n - 3] = ints(ids[3:])
    state = ints([head, head + n], torch.int64)
    tables = torch.full((1, 16), -7, dtype=torch.int32, device=DEV)
    status = zero_status(DEV)
    p = pk.pa_step_plan(ints([0]), ints([n * bs]), tables, ring, state, bs, n * bs, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert tables[0].tolist() == ids + [-7] * 6
    assert p.slot_mapping.tolist() == [i * bs + j for i in ids for j in range(bs)]
    assert p.free_state.tolist() == [head + n, head + n]


@pytest.mark.parametrize("B", [3, 300, 2000])
@pytest.mark.parametrize("cached,new", [(40, 9), (-5, 2), (12, -3), (48, 1)])
def test_a_bad_sequence_keeps_its_length_in_place(B, cached, new):
    # lengths updated in place over steps: a sequence that breaks a rule is flagged each
    # time, and its table row is never handed out anew
    at = B // 2
    bs, M, NB = 16, 3, 3 * B + 4
    lens = ints([16 if b != at else cached for b in range(B)])
    n = ints([1 if b != at else new for b in range(B)])
    tables = torch.arange(3 * B, dtype=torch.int32, device=DEV).view(B, M)
    tables[:, 1:] = -7
    tables[at] = torch.arange(3 * at, 3 * at + 3, dtype=torch.int32, device=DEV)
    row = tables[at].clone()
    left = [3 * b + e for b in range(B) for e in (1, 2) if b != at] + list(range(3 * B, NB))
    ring = torch.full((NB,), -9, dtype=torch.int32, device=DEV)
    ring[:len(left)] = ints(left)
    state = ints([0, len(left)], torch.int64)
    out = pk.StepPlan.empty(B, 2 * B, DEV)._replace(context_lens=lens, free_state=state)
    for step in range(3):
        status = zero_status(DEV)
        p = pk.pa_step_plan(lens, n, tables, ring, state, bs, 2 * B, out=out, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == pk.PA_DEV_BAD_CONTEXT, step
        assert lens.tolist() == [17 + step if b != at else cached for b in range(B)]
        assert torch.equal(tables[at], row)
        assert state.tolist() == [B - 1, len(left)]  # one block each, in the first step
        assert int(p.q_offsets[at + 1]) - int(p.q_offsets[at]) == 0
        assert int(p.q_offsets[B]) == B - 1
