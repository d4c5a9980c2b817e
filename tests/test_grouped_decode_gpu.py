"""pa_decode_grouped against attention in 64 bits (bound: grouped_ref).  Every
slot that no sequence holds is NaN."""
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


def run(p, max_ctx=None, **kw):
    status = zero_status(DEV)
    out = torch.full_like(p.q, float("nan"))
    pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale,
                         max(p.ctx) if max_ctx is None else max_ctx, out=out, status=status,
                         **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check_all(p, out, only=None, what=""):
    for b in range(len(p.ctx)) if only is None else only:
        if p.ctx[b] == 0:
            assert (out[b] == 0).all()
            continue
        ref, tol = p.ref(b)
        check(out[p.rows(b)], ref, tol, f"{what} context {p.ctx[b]}")


CTX = [1, 0, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1025]


def batch(ctx, H, Hkv, D, bs, dtype, seed):
    return Paged(ctx, [1] * len(ctx), H, Hkv, D, bs, dtype, seed=seed)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (14, 2), (3, 3), (24, 2), (17, 1), (40, 1)])
def test_lengths_and_groups(dtype, D, bs, H, Hkv):
    p = batch(CTX, H, Hkv, D, bs, dtype, seed=D + bs + H)
    for pt in (0, 64, 192, 2048):
        out, st = run(p, partition_tokens=pt)
        assert st == 0
        check_all(p, out, what=f"partition {pt}")


@pytest.mark.parametrize("B,hi", [(1, 1000), (1, 9001), (3, 20000), (150, 700)])
def test_chosen_partitions(B, hi):
    g = torch.Generator().manual_seed(B)
    ctx = [hi] + torch.randint(1, hi, (B - 1,), generator=g).tolist()
    p = batch(ctx, 16, 2, 128, 16, torch.bfloat16, seed=B)
    out, st = run(p)
    assert st == 0
    check_all(p, out, only=range(0, B, 7))
    loose, st = run(p, max_ctx=p.tables.shape[1] * 16)  # a looser bound, other partitions
    assert st == 0
    check_all(p, loose, only=range(0, B, 7))


def test_stale_workspace_and_repeated_calls():
    p = batch([5000, 64, 1, 700], 8, 2, 128, 16, torch.float16, seed=4)
    n = pk.pa_decode_grouped_workspace_size(4, 8, 2, 128, 16, 5000)
    assert n > 0
    ws = torch.full((n // 4,), float("nan"), device=DEV)
    a, st = run(p, workspace=ws)
    assert st == 0
    check_all(p, a)
    b, _ = run(p, workspace=ws)
    assert torch.equal(a, b)


def test_scores_far_apart():
    p = batch([1500, 900, 700], 8, 2, 128, 16, torch.float16, seed=5)
    p.q.copy_((1 + 0.25 * torch.randn(p.q.shape, device=DEV)).half())
    nat = 1.0 / (128 * p.scale)
    for b, at, nats in ((0, 0, 20), (0, 700, 45), (0, 1499, 70), (1, 0, 60), (2, 100, -40)):
        p.keys[b][at] = nats * nat
        p.store(b)
    for pt in (0, 64, 2048):
        out, st = run(p, partition_tokens=pt)
        assert st == 0
        check_all(p, out)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_any_finite_scale(scale):
    p = batch([300, 20], 8, 2, 64, 16, torch.bfloat16, seed=6)
    p.scale = scale
    out, st = run(p, partition_tokens=64)
    assert st == 0
    check_all(p, out)


def test_nan_of_a_held_key_shows():
    p = batch([300, 300], 8, 2, 64, 16, torch.float16, seed=7)
    p.keys[0][200] = float("nan")
    p.store(0)
    for pt in (64, 2048):
        out, st = run(p, partition_tokens=pt)
        assert torch.isnan(out[0]).all()
        check_all(p, out, only=[1])


def test_bad_contexts_and_blocks_are_flagged():
    p = batch([100, 90, 200], 4, 2, 64, 16, torch.float16, seed=8)
    p.context[1] = -2
    out, st = run(p)
    assert st == pk.PA_DEV_BAD_CONTEXT and (out[1] == 0).all()
    check_all(p, out, only=[0, 2])
    p.context[1] = 90
    out, st = run(p, max_ctx=100)  # sequence 2 is cut to 100 keys
    assert st == pk.PA_DEV_BAD_CONTEXT
    cut = batch([100, 90, 200], 4, 2, 64, 16, torch.float16, seed=8)
    cut.context[2], cut.ctx[2] = 100, 100
    cut.keys[2], cut.values[2] = cut.keys[2][:100], cut.values[2][:100]
    check_all(cut, out)
    for bad in (-1, p.k_cache.shape[0], 2 ** 30):
        p.tables[1, 2] = bad
        out, st = run(p)
        assert st == pk.PA_DEV_BAD_BLOCK_ID
        p.keys[1][32:48] = 0
        p.values[1][32:48] = 0
        check_all(p, out)


def test_graph_and_streams():
    p = batch([3000, 10], 8, 2, 128, 16, torch.bfloat16, seed=9)
    want, _ = run(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    with torch.cuda.stream(side):
        pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale, 3000,
                             out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale, 3000,
                             out=out)
    p.context[0], p.ctx[0] = 2500, 2500
    p.keys[0], p.values[0] = p.keys[0][:2500], p.values[0][:2500]
    graph.replay()
    torch.cuda.synchronize()
    check_all(p, out)


def test_matches_pa_decode_with_a_head_each():
    p = batch([700, 33, 1], 4, 4, 128, 16, torch.float16, seed=10)
    a, _ = run(p)
    b = pk.pa_decode(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale, 700)
    assert (a.float() - b.float()).abs().max() <= 2e-3


def test_refusals():
    p = batch([1000], 4, 2, 64, 16, torch.float16, seed=1)
    for kw in (dict(partition_tokens=60), dict(partition_tokens=4096), dict(partition_tokens=-64),
               dict(max_ctx=p.tables.shape[1] * 16 + 1),
               dict(partition_tokens=64, workspace=torch.empty(16, device=DEV))):
        with pytest.raises(pk.PagedKVError):
            run(p, **kw)
    with pytest.raises(TypeError):
        pk.pa_decode_grouped(p.q, p.k_cache.bfloat16(), p.v_cache, p.tables, p.context, 0.1, 9)
    with pytest.raises(ValueError):
        pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context[:0], 0.1, 9)
    empty = pk.pa_decode_grouped(p.q[:0], p.k_cache, p.v_cache, p.tables[:0], p.context[:0], 0.1,
                                 9)
    assert empty.shape[0] == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gone", [range(0, 16), range(0, 64), range(64, 128), range(16, 300)])
def test_infinite_scores_weigh_nothing(dtype, gone):
    p = batch([300, 300], 8, 2, 128, 16, dtype, seed=9)
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.keys[0][gone.start:gone.stop, :, 5] = -float("inf")  # scores of -inf, whole stages of them
    p.store(0)
    kept = torch.tensor([j for j in range(300) if j not in gone], device=DEV)
    ref, tol = attend(p.q[:1], p.keys[0][kept], p.values[0][kept], p.scale, len(kept) - 1)
    for pt in (0, 64, 2048):
        out, st = run(p, partition_tokens=pt)
        assert st == 0
        check(out[:1], ref, tol, f"partition {pt}")
        check_all(p, out, only=[1])
