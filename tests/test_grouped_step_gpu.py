"""A serving loop with grouped heads through all its calls: plan, rotation with the
cache write, prompt attention, chunk attention and single-token decode.

The host keeps every sequence's raw queries, keys and values.  What the calls
leave is compared with it at each step: the plan's slots with the tables, the
cache with keys rotated in 64 bits (bound: test_rope_write_gpu), and attention
with attention in 64 bits over the rows the cache holds (bound: grouped_ref).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import attend, check
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


class Server:
    """Device state of the loop; one buffer of each kind, as a captured step has."""

    def __init__(self, B, H, Hkv, D, bs, NB, M, T_max, dtype, seed):
        self.H, self.Hkv, self.D, self.bs, self.NB, self.T_max = H, Hkv, D, bs, NB, T_max
        g = torch.Generator().manual_seed(seed)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.dtype = dtype
        self.k_cache = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dtype, device=DEV)
        self.v_cache = torch.full_like(self.k_cache, float("nan"))
        self.tables = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.randperm(NB, generator=g).int().to(DEV)
        self.state = torch.tensor([0, NB], dtype=torch.int64, device=DEV)
        self.context = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.inv = 10000.0 ** (-np.arange(D // 2) * 2.0 / D)
        self.axis = np.arange(D // 2) % 3
        self.table = pk.pa_rope_table(self.inv, self.axis, device=DEV)
        self.plan = pk.StepPlan.empty(B, T_max, DEV)._replace(free_state=self.state)
        self.status = zero_status(DEV)
        self.scale = D ** -0.5

    def begin(self, new):
        """Plans a step and writes its keys and values; returns (plan, rotated q, k, raw)."""
        n = torch.tensor(new, dtype=torch.int32, device=DEV)
        p = pk.pa_step_plan(self.context, n, self.tables, self.ring, self.state, self.bs,
                            self.T_max, out=self.plan, status=self.status)
        H, Hkv, D = self.H, self.Hkv, self.D
        qkv = torch.randn(self.T_max, H + 2 * Hkv, D, generator=self.gen, device=DEV).to(
            self.dtype)
        pos = torch.stack([p.positions, p.positions // 3, p.positions % 7])  # t, h, w
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        qr, kr = pk.pa_rope_cache_write(q, k, v, pos, self.table, p.slot_mapping, self.k_cache,
                                        self.v_cache, k_out=torch.empty_like(k.contiguous()),
                                        status=self.status)
        self.context = p.context_lens.clone()
        return p, qr, kr, (q, k, v, pos)

    def rows(self, b):
        """(keys, values) of sequence b as the cache holds them."""
        n = int(self.context[b])
        j = torch.arange(n, device=DEV)
        blk = self.tables[b].long()[j // self.bs]
        return self.k_cache[blk, j % self.bs], self.v_cache[blk, j % self.bs]


def check_rotation(s, x, pos, got):
    angle = pos.double().cpu().numpy()[s.axis].T * s.inv
    c = torch.from_numpy(np.cos(angle)).to(DEV)[:, None]
    n = torch.from_numpy(np.sin(angle)).to(DEV)[:, None]
    a, b = x.double().chunk(2, -1)
    ref = torch.cat([a * c - b * n, b * c + a * n], -1)
    mag = torch.cat([a.abs() + b.abs()] * 2, -1)
    tol = torch.finfo(x.dtype).eps / 2 * ref.abs() + 6e-7 * mag + 2.0 ** -25
    assert ((got.double() - ref).abs() <= tol).all()


def check_step(s, p, new, kr, raw, before):
    """The plan, the rotated rows and the cache against the host's view of the step."""
    q, k, v, pos = raw
    offs = np.concatenate([[0], np.cumsum(new)])
    assert p.q_offsets.tolist() == offs.tolist()
    assert s.context.tolist() == [c + n for c, n in zip(before, new)]
    T = int(offs[-1])
    check_rotation(s, k[:T], pos[:, :T], kr[:T])
    for b, n in enumerate(new):
        r = slice(int(offs[b]), int(offs[b + 1]))
        if n:
            assert p.positions[r].tolist() == list(range(before[b], before[b] + n))
        kc, vc = s.rows(b)
        assert not torch.isnan(kc).any() and not torch.isnan(vc).any()
        assert torch.equal(kc[before[b]:], kr[r]) and torch.equal(vc[before[b]:], v[r])
    assert (p.slot_mapping[T:] == -1).all()
    used = [x for x in s.tables.flatten().tolist() if x >= 0]
    assert len(used) == len(set(used))  # no block twice
    assert s.status.item() == 0


@pytest.mark.parametrize("dtype,H,Hkv,D,bs", [
    (torch.bfloat16, 8, 2, 128, 16), (torch.float16, 14, 2, 64, 32), (torch.bfloat16, 4, 4, 64, 8),
    (torch.float16, 20, 1, 128, 16),
])
def test_serving_loop(dtype, H, Hkv, D, bs):
    B = 6
    s = Server(B, H, Hkv, D, bs, NB=400, M=100, T_max=900, dtype=dtype, seed=H + D)
    before = [0] * B
    # step 1: prompts (two slots idle), attended to from their own rows
    new = [300, 0, 17, 129, 1, 0]
    p, qr, kr, raw = s.begin(new)
    out = pk.pa_prompt_attention(qr, kr, raw[2], p.q_offsets, s.scale, status=s.status)
    check_step(s, p, new, kr, raw, before)
    o = np.concatenate([[0], np.cumsum(new)])
    for b in range(B):
        r = slice(int(o[b]), int(o[b + 1]))
        ref, tol = attend(qr[r], kr[r], raw[2][r], s.scale, 0)
        check(out[r], ref, tol, f"prompt {b}")
    # the same prompts through the cache: a chunk that is the whole context
    again = pk.pa_chunk_attention(qr, s.k_cache, s.v_cache, s.tables, s.context, p.q_offsets,
                                  s.scale, status=s.status)
    for b in range(B):
        r = slice(int(o[b]), int(o[b + 1]))
        ref, tol = attend(qr[r], kr[r], raw[2][r], s.scale, 0)
        check(again[r], ref, tol, f"prompt {b} through the cache")
    before = s.context.tolist()
    # step 2: chunks on what is cached, a new prompt, a single token, an idle sequence
    new = [64, 200, 5, 0, 1, 33]
    p, qr, kr, raw = s.begin(new)
    out = pk.pa_chunk_attention(qr, s.k_cache, s.v_cache, s.tables, s.context, p.q_offsets,
                                s.scale, status=s.status)
    check_step(s, p, new, kr, raw, before)
    o = np.concatenate([[0], np.cumsum(new)])
    for b in range(B):
        r = slice(int(o[b]), int(o[b + 1]))
        kc, vc = s.rows(b)
        ref, tol = attend(qr[r], kc, vc, s.scale, before[b])
        check(out[r], ref, tol, f"chunk {b}")
    before = s.context.tolist()
    # steps 3 to 6: one token each
    for _ in range(4):
        new = [1] * B
        p, qr, kr, raw = s.begin(new)
        q1 = qr[:B].contiguous()
        out = pk.pa_decode_grouped(q1, s.k_cache, s.v_cache, s.tables, s.context, s.scale,
                                   max_context_len=100 * bs, status=s.status)
        check_step(s, p, new, kr, raw, before)
        for b in range(B):
            kc, vc = s.rows(b)
            ref, tol = attend(q1[b:b + 1], kc, vc, s.scale, before[b])
            check(out[b:b + 1], ref, tol, f"decode {b}")
        before = s.context.tolist()
    assert int(s.state[1] - s.state[0]) == 400 - sum(-(-c // bs) for c in before)


def test_captured_decode_step_replayed():
    # plan, rotation and decode in one graph, the state carried from replay to replay
    B, H, Hkv, D, bs, dtype = 5, 8, 2, 128, 16, torch.bfloat16
    s = Server(B, H, Hkv, D, bs, NB=200, M=30, T_max=512, dtype=dtype, seed=3)
    p, qr, kr, raw = s.begin([100, 15, 16, 250, 1])
    check_step(s, p, [100, 15, 16, 250, 1], kr, raw, [0] * B)
    q = torch.empty(B, H, D, dtype=dtype, device=DEV)
    k, v = (torch.empty(B, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
    ones = torch.ones(B, dtype=torch.int32, device=DEV)
    cached = s.context.clone()
    plan = pk.StepPlan.empty(B, B, DEV)._replace(free_state=s.state)
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    ws = torch.empty(pk.pa_decode_grouped_workspace_size(B, H, Hkv, D, bs, 30 * bs) or 16,
                     dtype=torch.uint8, device=DEV)

    def step():
        pk.pa_step_plan(cached, ones, s.tables, s.ring, s.state, bs, B, out=plan,
                        status=s.status)
        pk.pa_rope_cache_write(q, k, v, plan.positions.expand(3, B).contiguous(), s.table,
                               plan.slot_mapping, s.k_cache, s.v_cache, q_out=qr, k_out=kr,
                               status=s.status)
        pk.pa_decode_grouped(qr, s.k_cache, s.v_cache, s.tables, plan.context_lens, s.scale,
                             30 * bs, out=out, workspace=ws, status=s.status)
        cached.copy_(plan.context_lens)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):  # past block ends
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=s.gen, device=DEV))
        before = s.context.tolist()
        graph.replay()
        torch.cuda.synchronize()
        s.context = cached.clone()
        assert s.status.item() == 0 and s.context.tolist() == [c + 1 for c in before]
        for b in range(B):
            kc, vc = s.rows(b)
            assert torch.equal(kc[-1], kr[b]) and torch.equal(vc[-1], v[b])
            ref, tol = attend(qr[b:b + 1], kc, vc, s.scale, before[b])
            check(out[b:b + 1], ref, tol, f"replay {i}, sequence {b}")
