"""Beam search with an encoder through all its calls: the encoder's attention over its own
rows, prompts, then steps of plan, rotation with the cache write, single-token decode of all
beams, cross attention with the beams as queries, selection, reorder and block copies, and
the way back at the end; eagerly, checked at every step, and captured as one graph.

The host keeps the keys, values and tokens of every beam and moves them by the parents.
Attention is compared with attention in 64 bits over these (bound: grouped_ref), what is
selected with a selection in 64 bits from the same logits (bound: beam_ref), and the
hypotheses with the host's."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from beam_ref import compare
from grouped_ref import attend, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EOS, PAD, LAYERS = 3, 0, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def ints(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device=DEV)


class Search:
    """Random weights, the encoder's states of one batch, and the decoder's state."""

    def __init__(self, W, H, Hkv, D, bs, dtype, prompts, states, steps, end, V=700, seed=0):
        self.B, self.W, self.H, self.Hkv, self.D, self.bs = len(prompts), W, H, Hkv, D, bs
        self.dtype, self.prompts, self.states, self.steps, self.V = dtype, prompts, states, steps, V
        self.S, self.scale, self.E = max(steps), D ** -0.5, 96
        g = torch.Generator(device=DEV).manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device=DEV) * n ** -0.5).to(dtype)
        E, HD, KD = self.E, H * D, Hkv * D
        self.emb = weight(V, E) * E ** 0.5
        self.qkv = [weight(E, HD + 2 * KD) for _ in range(LAYERS)]
        self.o = [weight(HD, E) for _ in range(LAYERS)]
        self.cq = [weight(E, HD) for _ in range(LAYERS)]
        self.ckv = [weight(E, 2 * KD) for _ in range(LAYERS)]
        self.co = [weight(HD, E) for _ in range(LAYERS)]
        self.enc_qkv, self.enc_o = weight(E, HD + 2 * KD), weight(HD, E)
        self.out = weight(E, V).float() * 2
        self.out[:, EOS] *= end
        self.src = weight(sum(states), E) * E ** 0.5
        self.starts = ints(np.cumsum([0] + states)[:-1])
        self.lens = ints(states)
        self.src_offs = ints(np.cumsum([0] + states))
        self.table = pk.pa_rope_table(1e4 ** (-np.arange(D // 2) * 2 / D), device=DEV)
        n = self.B * W
        self.M = -(-(max(prompts) + self.S) // bs) + 1
        self.NB = n * self.M
        self.order = torch.randperm(self.NB, generator=torch.Generator().manual_seed(seed))
        self.start = torch.randint(4, V, (sum(prompts),), generator=g, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.tokens = torch.empty(self.S, self.B, W, dtype=torch.int32, device=DEV)
        self.parents = torch.empty_like(self.tokens)
        self.ended = torch.empty(self.S, self.B, W, device=DEV)
        self.limit = ints(steps)

    def heads(self, x, w, parts):
        return torch.split((x @ w).view(x.shape[0], -1, self.D), parts, 1)

    def attended(self, x, o, w):
        return x + o.reshape(o.shape[0], -1) @ w

    def encode(self, seen):
        H, Hkv = self.H, self.Hkv
        q, k, v = self.heads(self.src, self.enc_qkv, (H, Hkv, Hkv))
        o = pk.pa_cross_attention(q, k, v, self.src_offs, self.starts, self.lens, self.scale,
                                  status=self.status)
        seen("encoder", q, k, v, o)
        x = self.attended(self.src, o, self.enc_o)
        return [self.heads(x, w, (Hkv, Hkv)) for w in self.ckv]

    def layers(self, x, plan, cross, offs, longest, seen, prompt):
        """The decoder's layers over the rows of a step; its logits."""
        H, Hkv = self.H, self.Hkv
        for i in range(LAYERS):
            q, k, v = self.heads(x, self.qkv[i], (H, Hkv, Hkv))
            q, k = pk.pa_rope_cache_write(q, k, v, plan.positions, self.table, plan.slot_mapping,
                                          self.kc[i], self.vc[i], status=self.status,
                                          k_out=k.new_empty(k.shape))
            if prompt:
                o = pk.pa_prompt_attention(q, k, v, plan.q_offsets, self.scale,
                                           status=self.status)
            else:
                o = pk.pa_decode_grouped(q, self.kc[i], self.vc[i], self.tables, self.context,
                                         self.scale, self.M * self.bs, status=self.status)
            seen("self", i, q, k, v, o)
            x = self.attended(x, o, self.o[i])
            q = self.heads(x, self.cq[i], (H,))[0]
            o = pk.pa_cross_attention(q, *cross[i], offs, self.starts, self.lens, self.scale,
                                      longest, max(self.states), status=self.status)
            seen("cross", i, q, o)
            x = self.attended(x, o, self.co[i])
        return x.float() @ self.out

    def run(self, seen=lambda *a: None):
        """The whole search, on the device alone (so that it can be captured)."""
        B, W, bs, n = self.B, self.W, self.bs, self.B * self.W
        shape = (self.NB, bs, self.Hkv, self.D)
        self.kc, self.vc = ([torch.full(shape, math.nan, dtype=self.dtype, device=DEV)
                             for _ in range(LAYERS)] for _ in range(2))
        self.tables = torch.full((n, self.M), -1, dtype=torch.int32, device=DEV)
        ring, state = self.ring0.clone(), self.state0.clone()
        self.context = torch.zeros(n, dtype=torch.int32, device=DEV)
        cross = self.encode(seen)
        pairs = torch.empty(n, 2, dtype=torch.int64, device=DEV)
        scores = self.scores0.clone()
        for s in range(self.S):
            new, T = (self.first, sum(self.prompts)) if s == 0 else (self.ones, n)
            plan = pk.StepPlan.empty(n, T, DEV)._replace(context_lens=self.context,
                                                         free_state=state)
            pk.pa_step_plan(self.context, new, self.tables, ring, state, bs, T, out=plan,
                            status=self.status)
            if s == 0:  # a prompt is beam 0's; the other beams have no rows yet
                offs = plan.q_offsets[::W].contiguous()
                x = self.layers(self.emb[self.start], plan, cross, offs, max(self.prompts), seen,
                                True)
                logits = torch.full((n, self.V), math.nan, device=DEV)
                logits[::W] = x[(offs[1:] - 1).long()]
            else:
                logits = self.layers(self.emb[self.tokens[s - 1].flatten().long()], plan, cross,
                                     self.beams, W, seen, False)
            step = pk.BeamStep(self.tokens[s], self.parents[s], torch.empty_like(scores),
                               self.ended[s])
            pk.pa_beam_select(logits, scores, EOS, PAD, out=step, status=self.status)
            seen("select", s, logits, scores, step)
            done = (self.limit <= s + 1)[:, None]
            moved = step.parents.masked_fill(done, -1)
            pk.pa_beam_reorder(moved, self.tables, self.context, ring, state, bs,
                               out=pk.BeamTables(self.tables, self.context, state, pairs),
                               status=self.status)
            for kc, vc in zip(self.kc, self.vc):
                pk.pa_block_copy(kc, vc, pairs, status=self.status)
            seen("moved", s, moved, step)
            scores = step.scores.masked_fill(done, -math.inf)
        self.state, self.ring = state, ring

    def before(self):
        """What a run begins from, made outside of it."""
        self.ring0, self.state0 = self.order.int().to(DEV), ints([0, self.NB], torch.int64)
        self.scores0 = torch.full((self.B, self.W), -math.inf, device=DEV)
        self.scores0[:, 0] = 0
        self.ones = torch.ones(self.B * self.W, dtype=torch.int32, device=DEV)
        self.first = torch.zeros_like(self.ones)
        self.first[::self.W] = ints(self.prompts)
        self.beams = ints(np.arange(self.B + 1) * self.W)


class Host:
    """What every beam holds, as the host has it; called with all that a run computes."""

    def __init__(self, s):
        self.s = s
        self.n = s.B * s.W
        self.kv = [[[] for _ in range(LAYERS)] for _ in range(self.n)]  # beam, layer: (k, v)
        self.said = [[] for _ in range(self.n)]
        self.finished = [[] for _ in range(s.B)]  # (score, length, beam, tokens)
        self.step = 0

    def rows(self):
        """The row or rows of each beam in this step."""
        s = self.s
        if self.step:
            return [range(i, i + 1) for i in range(self.n)]
        at, out = 0, []
        for i in range(self.n):
            m = s.prompts[i // s.W] if i % s.W == 0 else 0
            out.append(range(at, at + m))
            at += m
        return out

    def __call__(self, what, *a):
        getattr(self, "see_" + what)(*a)

    def full(self, q, k, v, what, got):
        ref, tol = attend(q, k, v, self.s.scale, len(k))  # (every query sees all keys)
        check(got, ref, tol, what)

    def see_encoder(self, q, k, v, o):
        at = 0
        for m in self.s.states:
            r = slice(at, at + m)
            self.full(q[r], k[r], v[r], "encoder", o[r])
            at += m
        self.cross = None

    def see_self(self, layer, q, k, v, o):
        for i, r in enumerate(self.rows()):
            if len(r) == 0:
                continue
            r = slice(r.start, r.stop)
            held = self.kv[i][layer]
            held.extend(zip(k[r], v[r]))
            K, V = (torch.stack(x) for x in zip(*held))
            ref, tol = attend(q[r], K, V, self.s.scale, len(held) - (r.stop - r.start))
            check(o[r], ref, tol, f"step {self.step} beam {i}")

    def see_cross(self, layer, q, o):
        s, at = self.s, 0
        rows = self.rows()
        for b, m in enumerate(s.states):
            r = slice(rows[b * s.W].start, rows[b * s.W + s.W - 1].stop)
            k, v = (x[at:at + m] for x in self.states[layer])
            self.full(q[r], k, v, f"step {self.step} cross {b}", o[r])
            at += m

    def see_select(self, step, logits, scores, out):
        s = self.s
        fine = torch.isfinite(scores).reshape(-1, 1)
        compare(out, torch.where(fine, logits, 0.0), scores, EOS, PAD)
        for b, w in torch.isfinite(out.ended_scores).nonzero().tolist():
            i = b * s.W + w
            self.finished[b].append((out.ended_scores[b, w].item(), step, w, self.said[i][:]))

    def see_moved(self, step, moved, out):
        s = self.s
        p, t = moved.tolist(), out.tokens.tolist()
        kv, said = [], []
        for b in range(s.B):
            for w in range(s.W):
                i = b * s.W + p[b][w]
                kv.append([x[:] for x in self.kv[i]] if p[b][w] >= 0 else
                          [[] for _ in range(LAYERS)])
                said.append(self.said[i] + [t[b][w]] if p[b][w] >= 0 else [])
                if s.steps[b] == step + 1:  # the request's last step: its beams end as they are
                    i = b * s.W + out.parents[b, w].item()
                    self.finished[b].append((out.scores[b, w].item(), step + 1, w,
                                             self.said[i] + [t[b][w]]))
        self.kv, self.said, self.step = kv, said, step + 1
        held = s.context.tolist()
        assert held == [len(x[0]) for x in kv]
        for i, m in enumerate(held):  # every cache has the beam's own history
            at = torch.arange(m, device=DEV)
            blk = s.tables[i].long()[at // s.bs]
            for layer in range(LAYERS):
                if m:
                    K, V = (torch.stack(x) for x in zip(*kv[i][layer]))
                    assert torch.equal(s.kc[layer][blk, at % s.bs], K), (step, i)
                    assert torch.equal(s.vc[layer][blk, at % s.bs], V), (step, i)
        assert s.status.item() == 0


CASES = [
    (4, 8, 2, 64, 16, torch.bfloat16, [5, 1, 18], [70, 1, 33], [20, 13, 20], 1.5),
    (5, 4, 4, 128, 8, torch.float16, [8, 16], [300, 129], [19, 19], 8.0),
    (8, 16, 4, 64, 32, torch.bfloat16, [31, 2, 9, 40, 1], [5, 64, 128, 200, 17], [6, 9, 12, 1, 2],
     8.0),
    (1, 4, 1, 64, 8, torch.float16, [3], [40], [10], 1.5),
]  # (the last number: the weight of the end, with 8 some hypotheses end early)


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{len(c[6])}" for c in CASES])
def test_search(case):
    W, H, Hkv, D, bs, dtype, prompts, states, steps, end = case
    s = Search(W, H, Hkv, D, bs, dtype, prompts, states, steps, end, seed=W)
    s.before()
    host = Host(s)
    encode = s.encode

    def keep(seen):
        host.states = encode(seen)
        return host.states
    s.encode = keep
    s.run(host)
    s.encode = encode
    # every block is free again
    head, tail = s.state.tolist()
    assert sorted(s.ring[i % s.NB].item() for i in range(head, tail)) == list(range(s.NB))
    if end > 2:
        assert any(n < steps[b] for b, f in enumerate(host.finished) for _, n, _, _ in f)
    # the best hypotheses of each request
    best = [sorted(f, key=lambda h: -h[0])[:W] for f in host.finished]
    K = min(len(f) for f in best)
    said = pk.pa_beam_backtrack(s.tokens, s.parents, ints([[h[1] for h in f[:K]] for f in best]),
                                ints([[h[2] for h in f[:K]] for f in best]), PAD,
                                status=s.status).tolist()
    for b, f in enumerate(best):
        for k, (_, n, _, tokens) in enumerate(f[:K]):
            assert said[b][k] == tokens + [PAD] * (s.S - n), (b, k)
    assert s.status.item() == 0
    # the same as one graph, twice, on a stream of its own
    want = [x.clone() for x in (s.tokens, s.parents, s.ended, s.state, s.ring)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()  # (what is allocated or set up once)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    for _ in range(2):
        for x in (s.tokens, s.parents, s.ended):
            x.fill_(-9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, (s.tokens, s.parents, s.ended, s.state, s.ring)):
            assert torch.equal(x, y)
        assert s.status.item() == 0


def test_block_copy_of_bf16_pools():
    k = torch.randn(6, 8, 2, 64, device=DEV).bfloat16()
    v, before = -k, k.clone()
    pk.pa_block_copy(k, v, ints([[0, 5], [2, 2], [3, 1]], torch.int64))
    for to, of in ((0, 0), (1, 3), (2, 2), (3, 3), (4, 4), (5, 0)):
        assert torch.equal(k[to], before[of]) and torch.equal(v[to], -before[of])
    with pytest.raises(TypeError):
        pk.pa_block_copy(k, v.half(), ints([[0, 5]], torch.int64))
    with pytest.raises(TypeError):
        pk.pa_block_copy(k.float(), v.float(), ints([[0, 5]], torch.int64))


def test_two_calls_at_once():
    """Calls on two streams at a time, each with outputs and a workspace of its own, give what
    they give alone."""
    g = torch.Generator(device=DEV).manual_seed(5)
    sides = []
    for i in range(2):
        W, V, bs = 16, 140000, 16
        logits = torch.randn(W, V, generator=g, device=DEV)
        scores = -torch.rand(1, W, generator=g, device=DEV)
        q = torch.randn(700, 8, 64, generator=g, device=DEV).half()
        k, v = (torch.randn(9000, 4, 64, generator=g, device=DEV).half() for _ in range(2))
        B, M = 300, 40
        tables = torch.randperm(B * 4 * M, generator=torch.Generator().manual_seed(i)).int()
        tables = tables.view(B * 4, M).to(DEV)
        lens = torch.randint(1, M * bs, (B,), generator=g, device=DEV).int().repeat_interleave(4)
        ring, state = ints(np.arange(B * 4 * M)), ints([0, 0], torch.int64)
        parents = torch.randint(0, 4, (B, 4), generator=g, device=DEV).int()
        # blocks of other rows for the copies: all of them are held, so the ring is empty
        lens = lens // bs * bs

        def call(out, stream, logits=logits, scores=scores, q=q, k=k, v=v, tables=tables,
                 lens=lens, ring=ring, state=state, parents=parents):
            step, att, few, moved, ws = out
            pk.pa_beam_select(logits, scores, 3, out=step, workspace=ws[0], stream=stream)
            for x, n, w in ((att, 700, ws[1]), (few, 2, ws[2])):
                pk.pa_cross_attention(q[:n], k, v, ints([0, n]), ints([0]), ints([9000]), 0.125,
                                      n, 9000, out=x, workspace=w, stream=stream)
            pk.pa_beam_reorder(parents, tables, lens, ring.clone(), state, bs, out=moved,
                               workspace=ws[3], stream=stream)

        def room():
            sizes = (pk.pa_beam_select_workspace_size(1, W, V),
                     pk.pa_cross_attention_workspace_size(1, 700, 8, 4, 64, 700, 9000),
                     pk.pa_cross_attention_workspace_size(1, 2, 8, 4, 64, 2, 9000),
                     pk.pa_beam_reorder_workspace_size(B, 4, M))
            return (pk.BeamStep.empty(1, W, DEV), torch.empty_like(q), torch.empty_like(q[:2]),
                    pk.BeamTables.empty(B * 4, M, DEV),
                    [torch.empty(max(16, n), dtype=torch.uint8, device=DEV) for n in sizes])
        sides.append((call, room(), room(), torch.cuda.Stream()))

    def results(out):
        return [*out[0], out[1], out[2], *out[3]]
    for call, alone, _, _ in sides:
        call(alone, None)
    torch.cuda.synchronize()
    for _ in range(8):
        for call, _, out, stream in sides:
            with torch.cuda.stream(stream):
                call(out, stream)
    torch.cuda.synchronize()
    for _, alone, out, _ in sides:
        for x, y in zip(results(alone), results(out)):
            assert torch.equal(x, y)
