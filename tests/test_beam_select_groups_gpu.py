"""pa_beam_select with a request's rows shared out among several clusters, in uneven parts:
equal rows tie whichever cluster they are in."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,W,V,stride", [(1, 16, 140000, 140000), (1, 16, 140001, 140003),
                                          (1, 32, 260000, 260000), (2, 31, 60001, 60001),
                                          (3, 15, 120000, 120000), (2, 24, 100000, 100000),
                                          (4, 13, 128256, 128256), (1, 5, 90000, 90000),
                                          (8, 32, 128000, 128000), (2, 7, 200000, 200000)])
def test_equal_rows(B, W, V, stride, dtype):
    """All rows alike, some beams dead: the lowest (beam, token), and equal scores."""
    g = torch.Generator(device="cuda").manual_seed(V + W)
    row = (torch.randn(1, V, device="cuda", generator=g) * 3).to(dtype)
    x = torch.empty(B * W, stride, dtype=dtype, device="cuda")[:, :V]
    x.copy_(row.expand(B * W, V))
    eos = 3
    order = torch.sort(row[0].double(), descending=True, stable=True)
    best = [i for i in order.indices[:W + 1].tolist() if i != eos][:W]
    for dead in ([], [0], [W - 1], [0, 1], list(range(1, W, 3)), list(range(W // 2)),
                 list(range(2, W))):
        live = [w for w in range(W) if w not in dead]
        s = torch.full((B, W), -2.0, device="cuda")
        s[:, dead] = -INF
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pk.pa_beam_select(x, s, eos, -7, status=status)
        assert status.item() == 0
        want = [(w, v) for v in best for w in live]
        # (values that are equal in the row's type: beams first, then places)
        values = row[0].double()
        want = sorted(want, key=lambda c: (-values[c[1]].item(), *c))[:W]
        for b in range(B):
            got = list(zip(out.parents[b].tolist(), out.tokens[b].tolist()))
            assert got == want, (dead, b)
            assert len(set(out.scores[b].tolist())) == len({values[v].item() for _, v in want})


def test_uneven_parts_are_tested():
    """Of the sizes above some are shared out among clusters."""
    sizes = [pk.pa_beam_select_workspace_size(*a) for a in
             ((1, 16, 140000), (1, 32, 260000), (2, 31, 60001), (3, 15, 120000), (2, 24, 100000))]
    assert all(n > 0 for n in sizes), sizes
