"""pa_step_plan at its limits: rings of nearly 2^31 blocks."""
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
