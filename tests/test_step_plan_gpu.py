"""pa_step_plan against a token-by-token replay on the host.

The replay takes blocks from a queue, first in first out, as the allocator of
the pages does, and appends every new token's slot one at a time; all results
are whole numbers and have to be equal.
"""
import collections

import numpy as np
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


def make(cached, new, bs, M, NB, T_max, head=0, seed=0):
    """Host state of a step: shuffled ids, cached blocks mapped, the rest in the ring."""
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached, np.int64), np.asarray(new, np.int64)
    ids = rng.permutation(NB).astype(np.int32)
    bt = np.full((len(cached), M), -7, np.int32)  # entries that nothing may touch
    at = 0
    for b, c in enumerate(cached):
        have = -(-int(max(c, 0)) // bs) if 0 <= c <= M * bs else 0
        bt[b, :have] = ids[at:at + have]
        at += have
    ring = np.full(NB, -9, np.int32)
    left = ids[at:]
    ring[(head + np.arange(len(left))) % NB] = left
    return dict(cached=cached, new=new, bs=bs, M=M, NB=NB, T_max=T_max, bt=bt, ring=ring,
                state=np.array([head, head + len(left)], np.int64))


def replay(h):
    """(tables, context, offsets, slots, positions, state) of a step that fits."""
    bt = h["bt"].copy()
    head, tail = (int(x) for x in h["state"])
    queue = collections.deque(int(h["ring"][i % h["NB"]]) for i in range(head, tail))
    slots, pos, offs = [], [], [0]
    for b, (c, n) in enumerate(zip(h["cached"], h["new"])):
        held = -(-int(c) // h["bs"])
        for p in range(int(c), int(c + n)):
            if p >= held * h["bs"]:
                bt[b, held] = queue.popleft()
                held += 1
                head += 1
            slots.append(int(bt[b, p // h["bs"]]) * h["bs"] + p % h["bs"])
            pos.append(p)
        offs.append(len(pos))
    pad = h["T_max"] - len(pos)
    return (bt, h["cached"] + h["new"], np.array(offs), np.array(slots + [-1] * pad, np.int64),
            np.array(pos + [0] * pad, np.int64), np.array([head, tail]))


def call(h, out=None, in_place=False, stream=None):
    g = {k: torch.from_numpy(np.ascontiguousarray(h[k])).to(DEV) for k in ("bt", "ring", "state")}
    g["cached"] = torch.from_numpy(h["cached"].astype(np.int32)).to(DEV)
    g["new"] = torch.from_numpy(h["new"].astype(np.int32)).to(DEV)
    status = zero_status(DEV)
    if in_place:
        out = pk.StepPlan.empty(len(h["cached"]), h["T_max"], DEV)._replace(free_state=g["state"])
    p = pk.pa_step_plan(g["cached"], g["new"], g["bt"], g["ring"], g["state"], h["bs"],
                        h["T_max"], out=out, status=status, stream=stream)
    torch.cuda.synchronize()
    return g, p, int(status.item())


def check(h, g, p):
    bt, ctx, offs, slots, pos, state = replay(h)
    assert np.array_equal(g["bt"].cpu().numpy(), bt)
    assert np.array_equal(p.context_lens.cpu().numpy(), ctx)
    assert np.array_equal(p.q_offsets.cpu().numpy(), offs)
    assert np.array_equal(p.slot_mapping.cpu().numpy(), slots)
    assert np.array_equal(p.positions.cpu().numpy(), pos)
    assert np.array_equal(p.free_state.cpu().numpy(), state)
    assert np.array_equal(g["ring"].cpu().numpy(), h["ring"])


@pytest.mark.parametrize("bs", [4, 8, 16, 32])
@pytest.mark.parametrize("B,hi,qhi,pad,head", [
    (1, 0, 1, 0, 0), (1, 5000, 5000, 3, 11), (7, 40, 1, 57, 10 ** 9), (33, 300, 70, 0, 1),
    (1000, 100, 5, 100, 999), (1025, 60, 3, 1, 5), (2500, 40, 9, 500, 77),
])
def test_plan_matches_replay(bs, B, hi, qhi, pad, head):
    rng = np.random.default_rng(B * 100 + bs)
    cached = rng.integers(0, hi + 1, B)
    new = rng.integers(0, qhi + 1, B)
    new[-1] = qhi  # at least one token
    M = int((-(-(cached + new) // bs)).max()) + 1
    NB = int((-(-(cached + new) // bs)).sum()) + 3
    h = make(cached, new, bs, M, NB, int(new.sum()) + pad, head=head, seed=B)
    g, p, st = call(h)
    assert st == 0
    check(h, g, p)


def test_largest_batch_with_idle_sequences():
    rng = np.random.default_rng(5)
    B = 16384
    cached = rng.integers(0, 50, B)
    new = np.where(rng.random(B) < 0.7, 0, rng.integers(1, 4, B))
    need = -(-(cached + new) // 16)
    h = make(cached, new, 16, 4, int(need.sum()) + 1, int(new.sum()) + 9, head=3)
    g, p, st = call(h)
    assert st == 0
    check(h, g, p)


def test_exactly_the_last_block_and_in_place_state():
    h = make([15, 0, 16], [2, 17, 0], 16, 4, 5, 19, head=4)  # 2 cached blocks, 3 more: all 5
    g, p, st = call(h, in_place=True)
    assert st == 0 and int(p.free_state[1] - p.free_state[0]) == 0
    check(h, g, p)


def refused(h, bit):
    g, p, st = call(h)
    assert st == bit
    assert np.array_equal(g["bt"].cpu().numpy(), h["bt"])
    assert np.array_equal(p.context_lens.cpu().numpy(), h["cached"])
    assert (p.q_offsets == 0).all() and (p.slot_mapping == -1).all() and (p.positions == 0).all()
    assert np.array_equal(p.free_state.cpu().numpy(), h["state"])


def test_steps_that_do_not_fit_change_nothing():
    cached, new = [16, 3, 0], [1, 14, 30]  # 1 + 1 + 2 blocks of 16
    h = make(cached, new, 16, 4, 6, 45)    # 2 mapped, 4 free: fits
    g, p, st = call(h)
    assert st == 0
    check(h, g, p)
    refused(make(cached, new, 16, 4, 5, 45), pk.PA_DEV_NO_BLOCKS)       # 3 free
    refused(make(cached, new, 16, 4, 6, 44), pk.PA_DEV_BAD_CONTEXT)     # one token too many
    big = 2 ** 30  # sums past 32 bits
    h = make([0] * 6, [big] * 6, 16, 2 ** 26, 8, 64)
    h["bt"] = np.zeros((6, 1), np.int32)  # 6 * 2^30 tokens do not fit any table: all bad
    g, p, st = call(h)
    assert st == pk.PA_DEV_BAD_CONTEXT and (p.q_offsets == 0).all()


@pytest.mark.parametrize("state", [(-1, 3), (5, 4), (0, 100)])
def test_impossible_ring_state_holds_nothing(state):
    h = make([0], [1], 16, 2, 4, 4)
    h["state"] = np.array(state, np.int64)
    refused(h, pk.PA_DEV_NO_BLOCKS)


def test_bad_sequences_and_ids_are_flagged_and_skipped():
    good = make([20, 5, 31], [3, 1, 2], 16, 3, 12, 16, seed=9)
    want = replay(good)
    for bad_c, bad_n in ((-1, 2), (4, -3), (40, 9)):  # negative, or past the table row
        h = make([20, 5, 31], [3, 1, 2], 16, 3, 12, 16, seed=9)
        h["cached"] = np.insert(h["cached"], 1, bad_c)
        h["new"] = np.insert(h["new"], 1, bad_n)
        h["bt"] = np.insert(h["bt"], 1, -7, axis=0)
        g, p, st = call(h)
        assert st == pk.PA_DEV_BAD_CONTEXT
        assert p.context_lens.tolist() == [23, 0, 6, 33]
        assert p.q_offsets.tolist() == [0, 3, 3, 4, 6]
        assert np.array_equal(p.slot_mapping.cpu().numpy(), want[3])
        assert (g["bt"][1] == -7).all()
    h = make([20, 5], [3, 28], 16, 3, 12, 40, seed=2)
    h["ring"][0] = 12  # an id past the pool, taken by sequence 1's second block
    h["bt"][0, 1] = -1  # the block that sequence 0 continues
    g, p, st = call(h)
    assert st == pk.PA_DEV_BAD_BLOCK_ID
    s = p.slot_mapping.cpu().numpy()
    assert (s[:3] == -1).all() and (s[3:14] >= 0).all()
    assert (s[14:30] == -1).all() and s[30] >= 0 and int(g["bt"][1, 1]) == -1


def test_captured_plan_follows_new_lengths():
    # two replays of one graph, the second on new lengths and on the ring that
    # the first left (updated in place)
    h = make([10, 0, 33], [1, 20, 1], 16, 8, 40, 64, seed=3)
    g = {k: torch.from_numpy(np.ascontiguousarray(h[k])).to(DEV) for k in ("bt", "ring", "state")}
    cached = torch.from_numpy(h["cached"].astype(np.int32)).to(DEV)
    new = torch.from_numpy(h["new"].astype(np.int32)).to(DEV)
    status = zero_status(DEV)
    out = pk.StepPlan.empty(3, 64, DEV)._replace(free_state=g["state"])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pk.pa_step_plan(cached, new, g["bt"], g["ring"], g["state"], 16, 64, out=out,
                        status=status)
    for step_new in ([1, 20, 1], [30, 0, 2]):
        new.copy_(torch.tensor(step_new, dtype=torch.int32))
        h["new"] = np.array(step_new)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        check(h, g, out)
        h["bt"], h["cached"], h["state"] = (g["bt"].cpu().numpy(), h["cached"] + h["new"],
                                            g["state"].cpu().numpy())
        cached.copy_(out.context_lens)


def test_empty_step():
    h = make([], [], 16, 1, 4, 5)
    h["bt"] = np.zeros((0, 1), np.int32)
    g, p, st = call(h)
    assert st == 0 and p.q_offsets.tolist() == [0] and (p.slot_mapping == -1).all()
    assert p.free_state.tolist() == h["state"].tolist()
    h = make([5], [0], 16, 1, 4, 0)
    g, p, st = call(h)
    assert st == 0 and p.q_offsets.tolist() == [0, 0] and p.context_lens.tolist() == [5]


@pytest.mark.parametrize("B,hi,qhi", [(3, 90, 40), (200, 60, 1), (700, 90, 3), (64, 900, 200),
                                      (4000, 100, 2)])
def test_context_lengths_may_replace_the_cached_ones(B, hi, qhi):
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, hi + 1, B), rng.integers(0, qhi + 1, B)
    M = (hi + qhi + 7) // 8 + 1
    T = int(new.sum()) + 5
    h = make(cached, new, 8, M, B * M, T, seed=B)
    g = {k: torch.from_numpy(np.ascontiguousarray(h[k])).to(DEV) for k in ("bt", "ring", "state")}
    lens = torch.from_numpy(cached.astype(np.int32)).to(DEV)
    out = pk.StepPlan.empty(B, T, DEV)._replace(context_lens=lens, free_state=g["state"])
    status = zero_status(DEV)
    p = pk.pa_step_plan(lens, torch.from_numpy(new.astype(np.int32)).to(DEV), g["bt"], g["ring"],
                        g["state"], 8, T, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(h, g, p)
