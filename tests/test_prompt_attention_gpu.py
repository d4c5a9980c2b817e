"""pa_prompt_attention against attention in 64 bits (bound: grouped_ref)."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import Packed, attend, check
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def run(p, out=None, **kw):
    status = zero_status(DEV)
    out = torch.full_like(p.q.contiguous(), 7.0) if out is None else out
    pk.pa_prompt_attention(p.q, p.k, p.v, p.offsets, p.scale, out=out, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check_all(p, out, only=None, what=""):
    for b in range(len(p.lens)) if only is None else only:
        r = p.rows(b)
        ref, tol = attend(p.q[r], p.k[r], p.v[r], p.scale, 0)
        check(out[r], ref, tol, f"{what} sequence {b} of {p.lens[b]}")


LENS = [1, 0, 2, 127, 128, 129, 31, 33, 255, 256, 257, 63, 64, 65, 300, 0]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,fused", [(8, 2, True), (3, 3, False), (14, 2, True), (5, 1, True),
                                         (16, 1, False), (20, 4, False), (24, 2, True)])
def test_lengths_around_tiles(dtype, D, H, Hkv, fused):
    p = Packed(LENS, H, Hkv, D, dtype, seed=H + D, fused=fused)
    out, st = run(p)
    assert st == 0
    check_all(p, out, what=f"{H}/{Hkv}")


@pytest.mark.parametrize("n", [1, 5, 600, 1111])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (32, 8)])
def test_one_sequence(n, H, Hkv):
    p = Packed([n], H, Hkv, 128, torch.bfloat16, seed=n)
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_long_sequence_beside_short_ones():
    p = Packed([17, 4100, 1, 900], 8, 2, 128, torch.bfloat16, seed=3, fused=True)
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_many_sequences():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    p = Packed(lens, 8, 2, 64, torch.float16, seed=4)
    out, st = run(p)
    assert st == 0
    check_all(p, out, only=range(0, 700, 23))
    # every sequence, against itself alone
    for b in (1, 350, 699):
        if lens[b]:
            q = Packed([lens[b]], 8, 2, 64, torch.float16)
            q.q, q.k, q.v = (x[p.rows(b)].contiguous() for x in (p.q, p.k, p.v))
            alone, _ = run(q)
            assert torch.equal(alone, out[p.rows(b)])


@pytest.mark.parametrize("H,Hkv", [(128, 1), (43, 1), (65, 1), (96, 2)])
def test_large_groups(H, Hkv):
    p = Packed([130, 1, 77], H, Hkv, 64, torch.bfloat16, seed=H)
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_rows_outside_the_sequences_stay_and_nan_does_not_leak():
    p = Packed([40, 130], 8, 2, 128, torch.float16, seed=6, before=5, behind=9)
    for x in (p.q, p.k, p.v):
        x[:5] = float("nan")
        x[175:] = float("inf")
    out, st = run(p)
    assert st == 0
    assert (out[:5] == 7).all() and (out[175:] == 7).all()
    check_all(p, out)
    # the next sequence's rows hold NaN: the one before is not touched by them
    for x in (p.q, p.k, p.v):
        x[45:175] = float("nan")
    out, _ = run(p)
    check_all(p, out, only=[0])
    assert torch.isnan(out[45:175]).all()


def test_scores_far_apart():
    # the running maximum jumps by up to 70 nats, upwards, downwards and across tiles
    p = Packed([700, 300], 4, 2, 128, torch.float16, seed=7)
    p.q.copy_((1 + 0.25 * torch.randn(p.q.shape, device=DEV)).half())
    nat = 1.0 / (128 * p.scale)
    for at, nats in ((0, 20), (100, 35), (140, -40), (400, 70), (701, 60), (900, 15)):
        p.k[at] = nats * nat
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_values_of_one_give_one():
    p = Packed([513], 8, 2, 128, torch.bfloat16, seed=8)
    p.v.fill_(1.0)
    out, _ = run(p)
    assert (out.float() - 1).abs().max() <= 2.0 ** -7


def test_bad_offsets_are_flagged_and_skipped():
    p = Packed([50, 60, 70], 4, 2, 64, torch.float16, seed=9)
    for offs, live in (([0, 50, 110, 181], [0, 1]), ([-1, 50, 110, 180], [1, 2])):
        p.offsets.copy_(torch.tensor(offs, dtype=torch.int32))
        out, st = run(p)
        assert st == pk.PA_DEV_BAD_CONTEXT
        check_all(p, out, only=live)
    # falling offsets: the last sequence is rows 40 .. 179 and shares 40 .. 49 with
    # the first, whose other rows are its own
    p.offsets.copy_(torch.tensor([0, 50, 40, 180], dtype=torch.int32))
    out, st = run(p)
    assert st == pk.PA_DEV_BAD_CONTEXT
    ref, tol = attend(p.q[:40], p.k[:40], p.v[:40], p.scale, 0)
    check(out[:40], ref, tol, "rows of one sequence alone")
    p.offsets.copy_(torch.tensor([0, 50, 110, 181], dtype=torch.int32))
    out, _ = run(p)
    assert (out[110:] == 7).all()


def test_other_stream_and_captured():
    p = Packed([100, 333], 8, 2, 128, torch.bfloat16, seed=10)
    want, _ = run(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    pk.pa_prompt_attention(p.q, p.k, p.v, p.offsets, p.scale, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_prompt_attention(p.q, p.k, p.v, p.offsets, p.scale, out=out)
    p.offsets.copy_(torch.tensor([0, 200, 433], dtype=torch.int32))  # other lengths, same graph
    p.lens, p.start[1] = [200, 233], 200
    graph.replay()
    torch.cuda.synchronize()
    check_all(p, out)


def test_same_call_twice_gives_the_same_bits():
    p = Packed([900, 31, 256], 16, 4, 128, torch.float16, seed=11)
    a, _ = run(p)
    b, _ = run(p)
    assert torch.equal(a, b)


def test_empty_and_refusals():
    p = Packed([0, 0], 8, 2, 64, torch.float16)
    out, st = run(p)
    assert st == 0 and out.shape[0] == 0
    p = Packed([9], 8, 2, 64, torch.float16)
    with pytest.raises(TypeError):
        pk.pa_prompt_attention(p.q.float(), p.k, p.v, p.offsets, 0.1)
    with pytest.raises(TypeError):
        pk.pa_prompt_attention(p.q, p.k.bfloat16(), p.v, p.offsets, 0.1)
    with pytest.raises(ValueError):
        pk.pa_prompt_attention(p.q, p.k, p.v[:5], p.offsets, 0.1)
    with pytest.raises(ValueError):
        pk.pa_prompt_attention(p.q, p.k, p.v, p.offsets, 0.1, out=torch.empty_like(p.k))
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(pk.PagedKVError):
            pk.pa_prompt_attention(p.q, p.k, p.v, p.offsets, scale)
    with pytest.raises(pk.PagedKVError):  # 129 query heads on one K/V head
        wide = Packed([3], 129, 1, 64, torch.float16)
        run(wide)
