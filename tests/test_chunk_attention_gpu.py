"""pa_chunk_attention against attention in 64 bits (bound: grouped_ref).  Every
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


def run(p, out=None, **kw):
    status = zero_status(DEV)
    out = torch.full_like(p.q, 7.0) if out is None else out
    pk.pa_chunk_attention(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.offsets, p.scale,
                          out=out, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check_all(p, out, only=None, what=""):
    for b in range(len(p.ctx)) if only is None else only:
        ref, tol = p.ref(b)
        check(out[p.rows(b)], ref, tol, f"{what} sequence {b}")


CTX = [1, 129, 128, 700, 40, 256, 5, 0, 1000, 333, 64]
QL = [1, 1, 128, 70, 40, 0, 3, 0, 257, 33, 64]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (14, 2), (3, 3), (20, 1)])
def test_lengths_around_tiles(dtype, D, bs, H, Hkv):
    p = Paged(CTX, QL, H, Hkv, D, bs, dtype, seed=D + bs + H)
    for split in (True, False):
        out, st = run(p, split=split)
        assert st == 0
        check_all(p, out, what=f"split {split}")


def test_split_contexts_merge():
    # few units, long contexts: up to eight key ranges, some of them all masked
    # for the first rows of a tile
    p = Paged([8192, 1025, 513, 4000, 600], [3, 1, 200, 130, 100], 8, 2, 128, 16, torch.bfloat16,
              seed=5)
    n = pk.pa_chunk_attention_workspace_size(5, 434, 8, 2, 128, p.tables.shape[1] * 16)
    assert n >= 8 * 434 * 8 * 130 * 4
    ws = torch.full((n // 4,), float("nan"), device=DEV)
    out, st = run(p, workspace=ws)
    assert st == 0
    check_all(p, out)
    whole, _ = run(p, split=False)
    check_all(p, whole)
    again, _ = run(p, workspace=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("first", [510, 511, 512, 600, 640])
def test_ranges_that_end_at_the_diagonal(first):
    # one chunk over a short cache: the last range of a unit is partly masked
    p = Paged([first + 100], [100], 4, 1, 64, 8, torch.float16, seed=first)
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_rows_outside_the_sequences_stay():
    p = Paged([300, 50], [20, 50], 8, 2, 128, 16, torch.float16, seed=6, before=3, behind=11)
    p.q[:3] = float("nan")
    p.q[73:] = float("nan")
    out, st = run(p)
    assert st == 0
    assert (out[:3] == 7).all() and (out[73:] == 7).all()
    check_all(p, out)


def test_scores_far_apart_across_ranges():
    p = Paged([4096, 2000], [16, 40], 4, 2, 128, 16, torch.float16, seed=7)
    p.q.copy_((1 + 0.25 * torch.randn(p.q.shape, device=DEV)).half())
    nat = 1.0 / (128 * p.scale)
    for b, at, nats in ((0, 0, 15), (0, 600, 45), (0, 3000, 30), (0, 4090, 60), (1, 1999, 70),
                        (1, 513, -40)):
        p.keys[b][at] = nats * nat
        p.store(b)
    out, st = run(p)
    assert st == 0
    check_all(p, out)


def test_bad_contexts_and_blocks_are_flagged():
    p = Paged([100, 90, 200], [20, 30, 10], 4, 2, 64, 16, torch.float16, seed=8)
    for bad in (29, -5, p.tables.shape[1] * 16 + 1):
        p.context.copy_(torch.tensor([100, bad, 200], dtype=torch.int32))
        for split in (True, False):
            out, st = run(p, split=split)
            assert st == pk.PA_DEV_BAD_CONTEXT
            assert (out[p.rows(1)] == 0).all()
            check_all(p, out, only=[0, 2])
    p.context.copy_(torch.tensor([100, 90, 200], dtype=torch.int32))
    p.offsets.copy_(torch.tensor([0, 20, 50, 61], dtype=torch.int32))
    out, st = run(p)
    assert st == pk.PA_DEV_BAD_CONTEXT
    check_all(p, out, only=[0, 1])
    assert (out[50:] == 7).all()
    p.offsets.copy_(torch.tensor([0, 20, 50, 60], dtype=torch.int32))
    for bad in (-1, p.k_cache.shape[0], 2 ** 30):
        p.tables[1, 2] = bad
        out, st = run(p)
        assert st == pk.PA_DEV_BAD_BLOCK_ID
        p.keys[1][32:48] = 0
        p.values[1][32:48] = 0
        check_all(p, out)
    # max_context_len bounds the contexts too
    out, st = run(p, max_context_len=100)
    assert st & pk.PA_DEV_BAD_CONTEXT
    assert (out[p.rows(2)] == 0).all()


def test_two_streams_share_nothing_and_a_graph_follows_lengths():
    a = Paged([2000, 900], [10, 40], 8, 2, 128, 16, torch.bfloat16, seed=9)
    b = Paged([1500, 3000], [33, 5], 8, 2, 128, 16, torch.bfloat16, seed=10)
    wa, wb = run(a)[0], run(b)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    for _ in range(5):
        for p, o, s in ((a, oa, s1), (b, ob, s2)):
            with torch.cuda.stream(s):
                pk.pa_chunk_attention(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.offsets,
                                      p.scale, out=o)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_chunk_attention(a.q, a.k_cache, a.v_cache, a.tables, a.context, a.offsets, a.scale,
                              out=oa)
    a.offsets.copy_(torch.tensor([0, 45, 50], dtype=torch.int32))
    a.qlens, a.start[1] = [45, 5], 45
    graph.replay()
    torch.cuda.synchronize()
    check_all(a, oa)


def test_own_buffers_come_from_the_stream_of_the_call():
    # out and workspace left to the call on another stream, while the current one
    # keeps taking and dropping blocks of the same size
    p = Paged([4000, 900], [10, 40], 8, 2, 128, 16, torch.bfloat16, seed=12)
    want = run(p)[0]
    side = torch.cuda.Stream()
    n = pk.pa_chunk_attention_workspace_size(2, 50, 8, 2, 128, p.tables.shape[1] * 16)
    assert n > 0
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append(pk.pa_chunk_attention(p.q, p.k_cache, p.v_cache, p.tables, p.context,
                                          p.offsets, p.scale, stream=side))
        for size in (n, want.numel() * 2):  # scribbles on whatever the pool hands out
            torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_refusals():
    p = Paged([100], [10], 4, 2, 64, 16, torch.float16)
    with pytest.raises(pk.PagedKVError):
        run(p, max_context_len=p.tables.shape[1] * 16 + 1)
    long = Paged([6000], [4], 4, 2, 64, 16, torch.float16)
    with pytest.raises(pk.PagedKVError):
        run(long, workspace=torch.empty(16, device=DEV))
    p4 = Paged([100], [10], 4, 2, 64, 4, torch.float16)
    with pytest.raises(pk.PagedKVError):
        run(p4)  # 4-token blocks
    with pytest.raises(TypeError):
        pk.pa_chunk_attention(p.q, p.k_cache.bfloat16(), p.v_cache, p.tables, p.context,
                              p.offsets, p.scale)
    with pytest.raises(ValueError):
        pk.pa_chunk_attention(p.q, p.k_cache, p.v_cache, p.tables, p.context[:0], p.offsets,
                              p.scale)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gone", [range(0, 128), range(0, 1300), range(512, 3000)])
def test_infinite_scores_weigh_nothing(dtype, gone):
    p = Paged([3100, 600], [40, 9], 8, 2, 128, 16, dtype, seed=12)
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    gone = range(gone.start, min(gone.stop, p.ctx[0] - 40))
    p.keys[0][gone.start:gone.stop, :, 5] = -float("inf")  # whole key tiles and ranges of them
    p.store(0)
    kept = torch.tensor([j for j in range(p.ctx[0]) if j not in gone], device=DEV)
    ref, tol = attend(p.q[p.rows(0)], p.keys[0][kept], p.values[0][kept], p.scale,
                      len(kept) - 40)
    for split in (True, False):
        out, st = run(p, split=split)
        assert st == 0
        check(out[p.rows(0)], ref, tol, f"split {split}")
        check_all(p, out, only=[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_bad", [1, 2, 3, 5])
def test_bad_sequences_among_short_ones(D, n_bad):
    # rows of zeros take a place in the ring, but no product: units of one to three key
    # tiles before and behind up to five of them
    ctx, good = [], []
    for i in range(80):
        good.append(len(ctx))
        ctx += [[130, 200, 256, 300, 100, 3, 384][i % 7]] + [60] * n_bad
    p = Paged(ctx, [1 + b % 3 for b in range(len(ctx))], 8, 4, D, 16, torch.bfloat16, seed=n_bad)
    bad = [b for b in range(len(ctx)) if b not in good]
    p.context[bad] = 1 << 20
    first = None
    for _ in range(5):
        out, st = run(p, split=False)
        assert st == pk.PA_DEV_BAD_CONTEXT
        check_all(p, out, only=good)
        for b in bad:
            assert (out[p.rows(b)] == 0).all()
        first = out if first is None else first
        assert torch.equal(out, first)
