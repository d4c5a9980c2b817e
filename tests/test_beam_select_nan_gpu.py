"""pa_beam_select on rows of which much is NaN: flagged, no candidate of that beam, the other
beams as ever."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from beam_ref import compare

pytestmark = pytest.mark.gpu
NAN = float("nan")


def patterns(V):
    """Where a row is NaN, [n, V]."""
    at = torch.arange(V, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(V)
    out = [at < V // 3, at >= V // 2, (at > V // 4) & (at < V // 2), at != V // 2, at >= 0]
    out += [at % 512 < n for n in (264, 288, 320, 388, 400, 416, 440, 511)]
    out += [at % 512 >= n for n in (70, 100, 200)]
    out += [at % p < n for p, n in ((16, 15), (32, 27), (128, 100), (8, 7), (1000, 800))]
    out += [torch.rand(V, device="cuda", generator=g) < share for share in (0.5, 0.8, 0.85, 0.97)]
    return torch.stack(out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("W", [1, 2, 4, 8, 9, 16])
@pytest.mark.parametrize("V,stride", [(512, 512), (513, 515), (4000, 4000), (9001, 9001),
                                      (65537, 65539)])
def test_much_that_is_none(V, stride, W, dtype):
    nan = patterns(V)
    B = len(nan)
    g = torch.Generator(device="cuda").manual_seed(W + V)
    x = torch.randn(B * W, stride, generator=g, device="cuda").mul_(3).to(dtype)[:, :V]
    s = -torch.rand(B, W, generator=g, device="cuda") * 5
    row = torch.arange(B, device="cuda") * W + torch.arange(B, device="cuda") % W
    x[row] = x[row].masked_fill(nan, NAN)
    # all requests, then one of them, whose rows are cut finer
    for b0, b1 in ((0, B), (0, 1), (9, 10), (B - 3, B - 2)):
        logits, scores = x[b0 * W:b1 * W], s[b0:b1]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pk.pa_beam_select(logits, scores, V - 1, -7, status=status)
        assert status.item() == pk.PA_DEV_BAD_LOGITS
        compare(out, logits, scores, V - 1, -7)
        bad = torch.arange(b0, b1, device="cuda") % W
        filled = torch.isfinite(out.scores)
        assert not ((out.parents == bad[:, None]) & filled).any()
        assert (out.ended_scores.gather(1, bad[:, None]) == -float("inf")).all()


def test_bad_beams_of_a_dead_place():
    """A beam that is not there may hold nothing else."""
    x = torch.randn(8, 5000, device="cuda")
    x[3] = NAN
    x[5, :400] = NAN
    s = torch.zeros(2, 4, device="cuda")
    s[0, 3] = s[1, 1] = -float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.pa_beam_select(x, s, 4, -7, status=status)
    assert status.item() == 0
    compare(out, x, s, 4, -7)
