"""pa_beam_select against a plain implementation in 64 bits (beam_ref)."""
import math

import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from beam_ref import compare

pytestmark = pytest.mark.gpu
F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


def run(logits, scores, eos=-1, pad=-7, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.pa_beam_select(logits, scores, eos, pad, status=status, **kw)
    return out, status.item()


def check(logits, scores, eos=-1, pad=-7, flags=0, rises=24, **kw):
    out, got = run(logits, scores, eos, pad, **kw)
    assert got == flags
    compare(out, logits, scores, eos, pad, rises)
    return out


def made(B, W, V, dtype, seed, stride=None, first=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B * W, stride or V, generator=g, device="cuda").mul_(3).to(dtype)
    s = -torch.rand(B, W, generator=g, device="cuda") * 5
    if first:
        s[: max(1, int(B * first)), 1:] = -INF
    return x[:, :V], s


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8, 16, 31, 32])
def test_beams(W, dtype):
    for V in (1, 2, 31, 64, 1000, 8191, 8192, 8193, 20001):
        x, s = made(2, W, V, dtype, seed=W + V, first=0.5)
        check(x, s, eos=V // 2)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("B,W,V,stride", [(1, 4, 32000, None), (7, 4, 50001, None),
                                         (2, 5, 50001, 50048), (2, 3, 128000, 128001),
                                         (1, 1, 300000, None), (1, 32, 100003, None),
                                         (2, 16, 140001, None), (1, 24, 260000, None),
                                         (40, 16, 4099, None), (300, 2, 513, 520)])
def test_vocabularies(B, W, V, stride, dtype):
    """One row cut into ranges, rows of several chunks, rows that begin anywhere."""
    x, s = made(B, W, V, dtype, seed=V, stride=stride, first=0.1)
    check(x, s, eos=V - 1)
    check(x, s)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ends(dtype):
    """Ends of every rank, in the first and the last place of the vocabulary."""
    B, W, V = 64, 4, 2000
    for eos in (0, 777, V - 1):
        x, s = made(B, W, V, dtype, seed=eos)
        x[:, eos] = x.amax(1) + torch.linspace(-6, 3, B * W, device="cuda").to(dtype)
        out = check(x, s, eos=eos)
        assert (out.tokens != eos).all()
        assert torch.isfinite(out.ended_scores).any() and (out.ended_scores == -INF).any()


@pytest.mark.parametrize("V", [50, 8192, 30000])
def test_equal_values(V):
    """All logits equal, of all beams: the lowest (beam, token); ends among them."""
    for W in (1, 4, 32):
        x = torch.full((2 * W, V), 1.5, device="cuda")
        s = torch.full((2, W), -2.0, device="cuda")
        out, _ = run(x, s)
        n = min(W, V)
        assert out.tokens[0, :n].tolist() == list(range(n))
        assert (out.parents[:, :n] == 0).all()
        # equal rows at other places, of other alignment, tie all the same
        g = torch.Generator(device="cuda").manual_seed(V)
        x = torch.randn(1, V, device="cuda", generator=g).repeat(2 * W, 1).contiguous()
        out, _ = run(x, s, eos=3)
        order = torch.sort(x[0].double(), descending=True, stable=True)
        best = [i for i in order.indices.tolist() if i != 3][:W]
        want = [(w, v) for v in best for w in range(W)][:W]
        for b in range(2):
            assert list(zip(out.parents[b].tolist(), out.tokens[b].tolist())) == want
        check(x, s, eos=3)
    # zeros of either sign are equal
    x = torch.zeros(1, V, device="cuda")
    x[0, ::2] = -0.0
    out, _ = run(x, torch.zeros(1, 1, device="cuda"))
    assert out.tokens.item() == 0


def test_equal_candidates_and_ends():
    """The end ties with the last candidate chosen: the lower index is ahead."""
    for eos, ahead in ((0, True), (9, False)):
        x = torch.full((2, 10), -INF, device="cuda")
        x[:, [0, 4, 9]] = 1.0
        s = torch.tensor([[0.0, -INF]], device="cuda")
        out, _ = run(x, s, eos=eos)
        left = [i for i in (0, 4, 9) if i != eos]
        assert out.tokens[0].tolist() == left and out.parents[0].tolist() == [0, 0]
        assert math.isfinite(out.ended_scores[0, 0].item()) == ahead
        compare(out, x, s, eos, -7)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
def test_orders_that_fill_the_list(dtype):
    """Logits that rise or fall along the row, steps, and few values over all of it."""
    V = 40000
    ramp = torch.arange(V, device="cuda", dtype=torch.float64)
    rows = torch.stack([ramp / V * 20, -ramp / V * 20, (ramp // 4096), -(ramp // 4096),
                        ramp % 2, ramp % 7 - 3, (ramp > V - 3).double() * 5,
                        torch.sin(ramp)]).to(dtype)
    for W in (2, 4, 8):
        s = -torch.arange(8, device="cuda").float().reshape(8 // W, W) * 0.0137
        check(rows, s, eos=V - 1, rises=V)
    for W in (1, 32):
        for r in rows:
            x = r.repeat(W, 1)
            s = torch.full((1, W), -INF, device="cuda")
            s[0, W - 1] = -1.0
            check(x, s, eos=17, rises=V)


@pytest.mark.parametrize("V", [40, 20000])
def test_masked(V):
    """Few tokens allowed, or none: places that nothing fills."""
    W = 4
    for allowed in ([], [7], [0, V - 1], [1, 2, 3, 4, 5, 9]):
        x, s = made(3, W, V, F32, seed=len(allowed))
        mask = torch.ones(V, dtype=torch.bool, device="cuda")
        mask[allowed] = False
        x = x.masked_fill(mask, -INF)
        s[1, 1:] = -INF
        s[2] = -INF
        out = check(x, s, eos=7)
        assert (out.tokens[2] == -7).all() and out.parents[2].tolist() == [0, 1, 2, 3]
        assert (out.scores[2] == -INF).all() and (out.ended_scores[2] == -INF).all()
    lowest = torch.finfo(F32).min
    x, s = made(2, W, V, F32, seed=5)
    x[:, 5:] = lowest  # the type's lowest value is a value
    check(x, s, eos=2)
    for dtype in (F32, BF16, FP16):  # a row of nothing else is one of equal values
        x[:] = torch.finfo(dtype).min
        x[1, V // 2] = torch.finfo(dtype).max
        check(x.to(dtype), s, eos=2)


def test_no_numbers():
    """NaN and +inf: of a dead beam unseen, of a live one flagged, the others as ever."""
    for v in (float("nan"), INF):
        x, s = made(3, 4, 9000, F32, seed=3)
        s[0, 1] = -INF
        x[1, 8999] = v
        check(x, s, eos=4)
        x[4 + 2, 100] = v
        out = check(x, s, eos=4, flags=pk.PA_DEV_BAD_LOGITS)
        assert (out.parents[1] != 2).all()
        x[8:, 0] = v
        x[9, :] = v
        out = check(x, s, eos=4, flags=pk.PA_DEV_BAD_LOGITS)
        assert (out.scores[2] == -INF).all()
    for v in (float("nan"), INF):  # scores that are none
        x, s = made(2, 3, 100, F32, seed=4)
        s[0, 1] = v
        out, flags = run(x, s)
        assert flags == 0 and (out.parents[0] != 1).all()


def test_far_scores():
    """Scores of long sequences: candidates that fp32 does not tell apart."""
    x, s = made(8, 4, 500, F32, seed=6)
    check(x, s - 3e6, eos=1)


def test_large_and_tiny_logits():
    for scale in (1e30, 1e-3, 80.0):
        x, s = made(4, 4, 3001, F32, seed=7)
        check(x * scale, s, eos=1)


def test_in_place_and_history():
    """Scores replaced, tokens and parents slices of a history, in a captured graph."""
    B, W, V, S = 3, 4, 5000, 4
    x, s = made(B, W, V, F32, seed=8, first=1.0)
    s[:, 0] = 0
    tok = torch.zeros(S, B, W, dtype=torch.int32, device="cuda")
    par = torch.zeros_like(tok)
    end = torch.zeros(S, B, W, device="cuda")
    live = s.clone()
    ws = torch.empty(pk.pa_beam_select_workspace_size(B, W, V), dtype=torch.uint8, device="cuda")

    def step(i):
        pk.pa_beam_select(x, live, 11, 0, out=pk.BeamStep(tok[i], par[i], live, end[i]),
                          workspace=ws)

    step(0)
    live.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(S):
            step(i)
    for seed in (1, 2):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        live.copy_(s)
        g.replay()
        torch.cuda.synchronize()
        now = s
        for i in range(S):
            out, _ = run(x, now, 11, 0)
            assert torch.equal(out.tokens, tok[i]) and torch.equal(out.parents, par[i])
            assert torch.equal(out.ended_scores, end[i])
            now = out.scores
        assert torch.equal(now, live)


def test_groups_of_rows():
    """Few requests, many beams: rows shared out among clusters, some of them dead."""
    B, W, V = 1, 16, 140000
    need = pk.pa_beam_select_workspace_size(B, W, V)
    assert need > 0
    for dead in ([], [0], [15], [3, 4, 7, 8, 11], list(range(1, 16)), list(range(16))):
        x, s = made(B, W, V, BF16, seed=len(dead))
        s[0, dead] = -INF
        check(x, s, eos=7)
    with pytest.raises(pk.PagedKVError) as e:
        run(x, s, workspace=torch.empty(need - 8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pk.PA_ERR_WORKSPACE


@pytest.mark.parametrize("B,W,V", [(1, 32, 33000), (2, 16, 60001), (8, 32, 20001), (5, 8, 40000),
                                   (12, 8, 30000), (18, 4, 64000), (20, 5, 50257), (40, 8, 20000),
                                   (80, 16, 5001), (100, 3, 9000)])
def test_shares_of_the_device(B, W, V):
    """Requests that take clusters of different sizes, several or a part of one each, and more
    than the device holds at once."""
    x, s = made(B, W, V, BF16 if B % 2 else F32, seed=B + W, first=0.3)
    check(x, s, eos=V - 2)


def test_deterministic_and_streams():
    x, s = made(16, 8, 60001, BF16, seed=9)
    first, _ = run(x, s, eos=5)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for stream in (None, other):
        for _ in range(5):
            out, _ = run(x, s, eos=5, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_far_rows():
    """Rows whose offset passes 2^32 elements."""
    V, W, stride = 1000, 4, 2 ** 31
    buf = torch.empty(3 * stride + V, dtype=FP16, device="cuda")
    x = buf.as_strided((W, V), (stride, 1))
    x.copy_(torch.randn(W, V, device="cuda"))
    check(x, torch.zeros(1, W, device="cuda"), eos=5)


def test_refusals():
    x, s = made(2, 4, 100, F32, seed=1)
    for args, err in (((x.double(), s), TypeError), ((x[:7], s), ValueError),
                      ((x, s.double()), TypeError), ((x, s[0]), ValueError),
                      ((x.cpu(), s), ValueError), ((x, s.cpu()), ValueError),
                      ((None, s), TypeError), ((x, None), TypeError),
                      ((x.t().contiguous().t(), s), ValueError),
                      ((x[:1].expand(8, 100), s), pk.PagedKVError)):
        with pytest.raises(err):
            pk.pa_beam_select(*args)
    for kw, err in ((dict(eos_token=100), pk.PagedKVError), (dict(eos_token=-2), pk.PagedKVError),
                    (dict(out=pk.BeamStep.empty(2, 3, "cuda")), ValueError),
                    (dict(out=pk.BeamStep.empty(2, 4, "cpu")), ValueError),
                    (dict(workspace=4), TypeError),
                    (dict(status=s), TypeError)):
        with pytest.raises(err):
            pk.pa_beam_select(x, s, **kw)
    x, s = made(1, 33, 100, F32, seed=1)
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_beam_select(x, s)
    assert e.value.code == pk.PA_ERR_UNSUPPORTED
    empty = torch.zeros(0, 4, device="cuda")
    assert pk.pa_beam_select(torch.zeros(0, 9, device="cuda"), empty).tokens.shape == (0, 4)
