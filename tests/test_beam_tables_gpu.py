"""pa_beam_reorder and pa_beam_backtrack against a replay element by element (beam_ref)."""
import numpy as np
import pytest
import torch

import beam_ref
import paged_kv_cache_172_gb300 as pk

pytestmark = pytest.mark.gpu
FLAGS = {"beam": pk.PA_DEV_BAD_BEAM, "context": pk.PA_DEV_BAD_CONTEXT,
         "blocks": pk.PA_DEV_NO_BLOCKS, "id": pk.PA_DEV_BAD_BLOCK_ID}


def whole(x, t=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)


class Beams:
    """Requests whose beams have parted block by block; a ring with the ids left."""

    def __init__(self, B, W, lens, bs, M=None, seed=0, spare=None, ragged=False):
        rng = np.random.default_rng(seed)
        lens = np.broadcast_to(np.asarray(lens), (B,))
        need = -(-lens // bs)
        self.B, self.W, self.bs = B, W, bs
        self.M = M or int(need.max()) + 1
        rows = np.full((B, W, self.M), -1, np.int64)
        at = 0
        for b in range(B):
            prompt = int(rng.integers(0, need[b] + 1)) if need[b] else 0
            for i in range(need[b]):
                if i < prompt:
                    rows[b, :, i] = at
                    at += 1
                    continue
                if rng.random() < 0.3:
                    rows[b, :, :i] = rows[b, rng.integers(0, W, W), :i]
                rows[b, :, i] = at + np.arange(W)
                at += W
        spare = B * W + 2 if spare is None else spare
        self.NB = at + spare
        ids = rng.permutation(self.NB)
        rows = np.where(rows >= 0, ids[rows], -1)
        if ragged:  # beams of other lengths: the rows' ends are dropped unseen
            lens = np.maximum(0, lens[:, None] - rng.integers(0, 2 * bs, (B, W)))
        else:
            lens = np.repeat(lens[:, None], W, 1)
        self.tables, self.lens = rows.reshape(B * W, self.M), lens.reshape(-1)
        head = int(rng.integers(0, 5 * self.NB))
        self.ring = np.full(self.NB, -1, np.int64)
        self.ring[(head + np.arange(spare)) % self.NB] = ids[at:]
        self.state = np.array([head, head + spare])
        self.rng = rng

    def parents(self):
        p = self.rng.integers(0, self.W, (self.B, self.W))
        kind = self.rng.random(self.B)
        p[kind < 0.3] = np.arange(self.W)
        p[kind < 0.1] = -1
        p[(kind > 0.9)[:, None] & (self.rng.random(p.shape) < 0.5)] = -1
        return p

    def check(self, parents, shared=None, in_place=False, flags=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = dict(p=whole(parents), bt=whole(self.tables), ctx=whole(self.lens),
                 ring=whole(self.ring), st=whole(self.state, torch.int64))
        out = None
        if in_place:
            out = pk.BeamTables(t["bt"], t["ctx"], t["st"],
                                torch.full((self.B * self.W, 2), 9, device="cuda"))
        got = pk.pa_beam_reorder(t["p"], t["bt"], t["ctx"], t["ring"], t["st"], self.bs,
                                 shared_lens=None if shared is None else whole(shared), out=out,
                                 status=status)
        ref = beam_ref.reorder(np.asarray(parents), self.tables, self.lens, self.ring, self.state,
                               self.bs, shared)
        for name, g, r in (("tables", got.block_tables, ref[0]), ("lens", got.context_lens, ref[1]),
                           ("ring", t["ring"], ref[2]), ("state", got.free_state, ref[3]),
                           ("pairs", got.copy_pairs, ref[4])):
            g = g.cpu().numpy()
            r = np.asarray(r).reshape(g.shape)
            d = np.argwhere(g != r)
            assert len(d) == 0, (name, d[:4].tolist(), g[tuple(d[0])], r[tuple(d[0])])
        assert status.item() == sum(FLAGS[f] for f in ref[5]), (status.item(), ref[5])
        if flags is not None:
            assert ref[5] == flags
        return ref


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bs", [4, 8, 16, 32])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8, 9, 16, 32])
def test_reorder(W, bs, in_place):
    rng = np.random.default_rng(W * bs)
    for seed, B in enumerate((1, 3, 17)):
        for ragged in (False, True):
            c = Beams(B, W, rng.integers(0, 9 * bs, B), bs, seed=seed, ragged=ragged)
            shared = rng.integers(0, 3 * bs, B) if seed else None
            c.check(c.parents(), shared, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,longest,M", [(64, 4, 2000, None), (1, 8, 80000, 6000),
                                          (300, 2, 300, 40), (1100, 1, 40, 4),
                                          (40, 32, 1000, None), (1024, 8, 30, 4),
                                          (1025, 8, 30, 4), (511, 2, 700, 50),
                                          (512, 2, 700, 50), (2500, 4, 100, 9),
                                          (20000, 1, 40, 3)])
def test_reorder_by_requests(B, W, longest, M, in_place):
    """Batches past one CTA, and at its border."""
    rng = np.random.default_rng(B)
    c = Beams(B, W, rng.integers(0, longest + 1, B), 16, M=M, seed=B)
    c.check(c.parents(), in_place=in_place)
    c.check(c.parents(), shared=rng.integers(0, 64, B), in_place=in_place)


def test_first_step():
    """All rows alike after the prompt, its last block half full: one keeps it."""
    for n in (16, 17, 31, 1, 0):
        c = Beams(2, 4, n, 16, seed=n)
        k = -(-n // 16)
        for b in range(2):
            c.tables[b * 4:(b + 1) * 4, :k] = c.tables[b * 4, :k]
        for p in ([[0] * 4] * 2, [[0, 1, 2, 3]] * 2, [[3, 2, 2, 1], [1, -1, -1, 1]]):
            ref = c.check(p)
            if p[0] == [0] * 4:
                assert len({r[max(0, k - 1)] for r in ref[0][:4]}) == (4 if n % 16 else 1)


@pytest.mark.parametrize("B", [5, 700])
def test_too_few_blocks(B):
    """All or nothing, up to the last block; states that no ring can have."""
    c = Beams(B, 8, 24, 16, seed=2, spare=B * 7)
    p = np.zeros((B, 8), int)
    c.check(p, flags=set())
    for in_place in (False, True):
        c.state[1] -= 1
        c.check(p, in_place=in_place, flags={"blocks"})
        c.state[1] += 1
    for state in ([-1, 5], [9, 8], [0, c.NB + 1], [2 ** 62, -2 ** 62]):
        c.state = np.array(state)
        c.check(p, flags={"blocks"})


@pytest.mark.parametrize("many", [False, True])
def test_bad_requests(many):
    """What does not fit leaves its request as it was, and the others as ever."""
    B, W = (600 if many else 6), 8
    for what in ("parent", "parent low", "length", "long", "shared", "tail", "held", "ring",
                 "full"):
        c = Beams(B, W, 40, 16, seed=3, M=8)
        p, shared = c.parents(), np.zeros(B, int)
        p[2] = [0, 0, 1, 1, 2, 2, 3, 3]
        if what == "parent":
            p[2, 5] = W
        elif what == "parent low":
            p[2, 5] = -2
        elif what == "length":
            c.lens[2 * W + 1] = -1
        elif what == "long":
            c.lens[2 * W + 1] = 2 ** 31 - 1
        elif what == "shared":
            shared[2] = -1
        elif what == "tail":
            c.tables[2 * W:3 * W, 2] = [c.NB, -1, -2 ** 31, 2 ** 31 - 1] * 2
        elif what == "held":
            c.tables[2 * W + 4:3 * W, 1] = [c.NB, -1, -2 ** 31, 2 ** 31 - 1]
        elif what == "ring":
            c.ring[(c.state[0] + np.arange(2)) % c.NB] = [-1, c.NB]
        else:  # more come back than there can be
            c.state[1] = c.state[0] + c.NB - 2
            c.ring[:] = c.rng.permutation(c.NB)
        flag = {"parent": "beam", "parent low": "beam", "length": "context", "long": "context",
                "shared": "context"}.get(what, "id")
        for in_place in (False, True):
            c.check(p, shared, in_place, flags={flag})


def test_a_search():
    """Steps of plan, reorder and copies: every beam's cache holds its own history, and all
    blocks come back."""
    B, W, bs, NB, M = 5, 4, 8, 400, 24
    rng = np.random.default_rng(4)
    kc = torch.zeros(NB, bs, 1, 64, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    ring = whole(rng.permutation(NB))
    state = whole([0, NB], torch.int64)
    tables = whole(np.full((B * W, M), -1))
    lens = whole(np.zeros(B * W))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(B * W)]
    pairs = torch.zeros(B * W, 2, dtype=torch.int64, device="cuda")
    new = whole(np.ones(B * W))
    for step in range(60):
        plan = pk.pa_step_plan(lens, new, tables, ring, state, bs, B * W, status=status)
        lens, state = plan.context_lens, plan.free_state
        k = torch.from_numpy(rng.standard_normal((B * W, 1, 64))).half().cuda()
        pk.pa_kv_cache_write(k, -k, plan.slot_mapping, kc, vc, status=status)
        for i in range(B * W):
            history[i] = history[i] + [k[i, 0]]
        p = rng.integers(0, W, (B, W)) if step % 3 else np.tile(np.arange(W), (B, 1))
        t = pk.BeamTables(tables, lens, state, pairs)
        pk.pa_beam_reorder(whole(p), tables, lens, ring, state, bs, out=t, status=status)
        pk.pa_block_copy(kc, vc, pairs, status=status)
        history = [history[b * W + p[b, w]] for b in range(B) for w in range(W)]
        if step % 10 == 9:
            assert status.item() == 0
            for i in range(B * W):
                at = torch.arange(len(history[i]), device="cuda")
                got = kc[tables[i, at // bs].long(), at % bs, 0]
                assert torch.equal(got, torch.stack(history[i])), (step, i)
            held = state.tolist()
            used = {int(x) for r, n in zip(tables.tolist(), lens.tolist()) for x in r[:-(-n // bs)]}
            free = [int(ring[i % NB]) for i in range(*held)]
            assert len(free) == len(set(free)) and not used & set(free)
            assert len(used) + len(free) == NB
    pk.pa_beam_reorder(whole(np.full((B, W), -1)), tables, lens, ring, state, bs,
                       out=pk.BeamTables(tables, lens, state, pairs), status=status)
    free = [int(ring[i % NB]) for i in range(*state.tolist())]
    assert sorted(free) == list(range(NB)) and status.item() == 0
    assert (tables == -1).all() and (lens == 0).all()


@pytest.mark.parametrize("W,K", [(1, 1), (2, 2), (4, 1), (4, 4), (8, 3), (16, 16), (32, 32),
                                 (3, 32)])
def test_backtrack(W, K):
    rng = np.random.default_rng(W + K)
    for S in (1, 2, 31, 32, 33, 64, 100, 1000, 2560, 2561, 6000):
        B = 3
        tok, par = rng.integers(0, 10 ** 6, (S, B, W)), rng.integers(0, W, (S, B, W))
        n, beam = rng.integers(0, S + 1, (B, K)), rng.integers(0, W, (B, K))
        n[0, 0], n[1, 0], n[2, 0] = S, 0, 1
        par[0] = -5  # of nothing
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pk.pa_beam_backtrack(whole(tok), whole(par), whole(n), whole(beam), -3, status=status)
        ref, bad = beam_ref.backtrack(tok, par, n, beam, -3)
        assert not bad and status.item() == 0
        assert (out.cpu().numpy() == ref).all(), S


@pytest.mark.parametrize("S", [5, 300, 7000])
def test_backtrack_what_is_off(S):
    rng = np.random.default_rng(S)
    B, W, K = 4, 5, 6
    for what in ("parent", "parent high", "beam", "length", "short"):
        tok, par = rng.integers(0, 99, (S, B, W)), rng.integers(0, W, (S, B, W))
        n, beam = np.full((B, K), S), rng.integers(0, W, (B, K))
        if what.startswith("parent"):
            par[S // 2, 1] = W if what == "parent high" else -1
            par[1, 2] = 2 ** 31 - 1
        elif what == "beam":
            beam[2] = [-1, 0, W, 1, 2 ** 31 - 1, 2]
        elif what == "length":
            n[2] = [-1, 0, S + 1, S, 2 ** 31 - 1, 1]
        else:
            n[2], beam[2] = 0, -9  # nothing asked for: the beam is not looked at
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((B, K, S), 77, dtype=torch.int32, device="cuda")
        pk.pa_beam_backtrack(whole(tok), whole(par), whole(n), whole(beam), -1, out=out,
                             status=status)
        ref, bad = beam_ref.backtrack(tok, par, n, beam, -1)
        assert (out.cpu().numpy() == ref).all(), what
        assert status.item() == (pk.PA_DEV_BAD_BEAM if bad else 0)
        assert bad == (what != "short")


def test_captured():
    """Reorder in place by requests, replayed with other parents."""
    c = Beams(600, 8, 200, 16, seed=5, spare=600 * 8 * 8)
    t = [whole(c.tables), whole(c.lens), whole(c.state, torch.int64),
         torch.zeros(4800, 2, dtype=torch.int64, device="cuda")]
    ring, p = whole(c.ring), whole(c.parents())
    ws = torch.empty(pk.pa_beam_reorder_workspace_size(600, 8, c.M), dtype=torch.uint8,
                     device="cuda")
    first = [x.clone() for x in (*t, ring)]

    def step():
        pk.pa_beam_reorder(p, t[0], t[1], ring, t[2], 16, out=pk.BeamTables(*t), workspace=ws)

    step()
    for x, y in zip((*t, ring), first):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        parents = c.parents()
        p.copy_(whole(parents))
        ref = beam_ref.reorder(parents, c.tables, c.lens, c.ring, c.state, 16)
        g.replay()
        torch.cuda.synchronize()
        for x, r in zip((t[0], t[1], ring, t[2], t[3]), ref):
            assert (x.cpu().numpy() == np.asarray(r)).all()
        c.tables, c.lens, c.ring, c.state = (np.asarray(r) for r in ref[:4])


def test_refusals():
    c = Beams(2, 4, 40, 16)
    a = [whole(c.parents()), whole(c.tables), whole(c.lens), whole(c.ring),
         whole(c.state, torch.int64), 16]
    for i, x, err in ((0, a[0].long(), TypeError), (0, a[0][0], ValueError),
                      (1, a[1][:7], ValueError), (1, a[1].long(), TypeError),
                      (2, a[2][:7], ValueError), (3, a[3].cpu(), ValueError),
                      (4, a[4].int(), TypeError), (4, a[4][:1], ValueError), (0, None, TypeError),
                      (5, 12, pk.PagedKVError), (1, a[1][:, ::2], ValueError)):
        args = list(a)
        args[i] = x
        with pytest.raises(err):
            pk.pa_beam_reorder(*args)
    for kw, err in ((dict(shared_lens=a[2]), ValueError), (dict(shared_lens=3), TypeError),
                    (dict(out=pk.BeamTables.empty(8, c.M + 1, "cuda")), ValueError),
                    (dict(status=a[4]), TypeError)):
        with pytest.raises(err):
            pk.pa_beam_reorder(*a, **kw)
    big = Beams(2000, 4, 40, 16)
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_beam_reorder(whole(big.parents()), whole(big.tables), whole(big.lens),
                           whole(big.ring), whole(big.state, torch.int64), 16,
                           workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pk.PA_ERR_WORKSPACE
    t = torch.zeros(6, 2, 3, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    b = [t, t, n, n]
    for i, x, err in ((0, t.long(), TypeError), (1, t[:5], ValueError), (2, n[:1], ValueError),
                      (3, n[:, :1].contiguous(), ValueError), (1, t.cpu(), ValueError),
                      (0, t[0], ValueError), (2, None, TypeError),
                      (0, t.transpose(0, 1), ValueError)):
        args = list(b)
        args[i] = x
        with pytest.raises(err):
            pk.pa_beam_backtrack(*args)
    assert pk.pa_beam_backtrack(t[:0], t[:0], n, n).shape == (2, 2, 0)
    assert pk.pa_beam_backtrack(t, t, n[:, :0], n[:, :0]).shape == (2, 0, 6)
    many = torch.zeros(2, 33, dtype=torch.int32, device="cuda")
    with pytest.raises(pk.PagedKVError):
        pk.pa_beam_backtrack(t, t, many, many)
