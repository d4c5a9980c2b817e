"""Cases of the grouped-head serving operators: step plan, rotary cache write, prompt
attention, chunk attention and grouped decode, with their plain forms in torch.

A serving loop with grouped key/value heads runs them in this order each step: the plan
gives every sequence its blocks and every new token its slot; queries and keys are rotated
and the keys and values stored; new prompts attend to themselves, chunks and single tokens
to the paged cache.  ``run`` computes one of them, in its plain form or (``own``) through
this package.  The lengths of a case come from the case itself (``mix`` seeds them), the
data from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- lengths of a case
def _lens(case):
    """(cached, new) lengths of the case's sequences, two int64 arrays."""
    rng = np.random.default_rng(case["mix"])
    B, op = case["B"], case["op"]
    if op == "prompt":
        new = _spread(rng, B, case["lo"], case["hi"])
        return np.zeros(B, np.int64), new
    if op == "chunk":
        new = _spread(rng, B, case["qlo"], case["qhi"])
        return _spread(rng, B, case["lo"], case["hi"]), new
    if op == "decode":
        total = _spread(rng, B, case["lo"], case["hi"])
        return total - 1, np.ones(B, np.int64)
    cached = _spread(rng, B, case["lo"], case["hi"])  # plan
    new = _spread(rng, B, case["qlo"], case["qhi"])
    fresh = rng.random(B) < case["fresh"]  # prompts that begin in this step
    return np.where(fresh, 0, cached), new


def _spread(rng, B, lo, hi):
    """B lengths in [lo, hi], the first one hi, so that the case's size is what it says."""
    x = rng.integers(lo, hi + 1, B)
    x[0] = hi
    return x.astype(np.int64)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the 38-sequence decode batch of the benchmark: one new token for each sequence
        dict(name="plan_decode", op="plan", B=38, lo=128, hi=2048, qlo=1, qhi=1, fresh=0.0, bs=16,
             mix=1),
        # a step of new prompts and chunks beside running sequences
        dict(name="plan_mixed", op="plan", B=200, lo=1, hi=2048, qlo=0, qhi=160, fresh=0.5, bs=16,
             mix=2),
        # single tokens of the same batch: latency counts
        dict(name="rope_decode", op="rope", T=38, H=40, Hkv=8, D=128, R=128, axes=1,
             interleaved=False, fused=True, k_out=False, far=2048, dtype="fp16", bs=16, mix=3),
        # a long image-and-text prompt: three axes, an odd number of tokens
        dict(name="rope_prompt_3axes", op="rope", T=16001, H=32, Hkv=8, D=128, R=128, axes=3,
             interleaved=False, fused=True, k_out=True, far=32768, dtype="bf16", bs=16, mix=4),
        # many short prompts of different lengths packed together, small heads
        dict(name="prompt_short_ragged", op="prompt", B=24, lo=1, hi=512, H=16, Hkv=4, D=64,
             fused=True, dtype="fp16", mix=5),
        # an ordinary batch of prompts
        dict(name="prompt_batch", op="prompt", B=8, lo=500, hi=4096, H=32, Hkv=8, D=128,
             fused=True, dtype="bf16", mix=6),
        # one long prompt of odd length
        dict(name="prompt_long", op="prompt", B=1, lo=16001, hi=16001, H=32, Hkv=8, D=128,
             fused=False, dtype="bf16", mix=7),
        # the benchmark's chunk (512 queries on 3,584 cached tokens, eight sequences), grouped
        dict(name="chunk_8x512", op="chunk", B=8, lo=3584, hi=3584, qlo=512, qhi=512, H=40, Hkv=8,
             D=128, bs=16, dtype="fp16", mix=8),
        # short chunks on caches of very different lengths (drafts to verify, ends of prompts)
        dict(name="chunk_short_ragged", op="chunk", B=16, lo=0, hi=8192, qlo=1, qhi=48, H=32,
             Hkv=8, D=128, bs=32, dtype="bf16", mix=9),
        # a single user's token: latency counts
        dict(name="decode_single", op="decode", B=1, lo=1000, hi=1000, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", mix=10),
        # the 38-sequence decode batch with grouped heads
        dict(name="decode_batch", op="decode", B=38, lo=128, hi=2048, H=40, Hkv=8, D=128, bs=16,
             dtype="fp16", mix=1),
        # few sequences with long contexts
        dict(name="decode_long", op="decode", B=4, lo=60000, hi=131072, H=64, Hkv=8, D=128, bs=32,
             dtype="bf16", mix=11),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "prompt", "chunk", "decode"])
    H, Hkv = rng.choice([(8, 8), (16, 4), (28, 4), (32, 8), (40, 8), (64, 8), (12, 4), (16, 1)])
    D = rng.choice([64, 128, 128])
    dtype = rng.choice(["fp16", "bf16"])
    bs = rng.choice([8, 16, 16, 32])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        B = _log(rng, 1, 1000)
        qhi = _log(rng, 1, max(1, 16000 // B))
        return dict(op=op, B=B, lo=0, hi=_log(rng, 1, 4000), qlo=rng.choice([0, 1]), qhi=qhi,
                    fresh=rng.choice([0.0, 0.3, 1.0]), bs=bs, mix=mix)
    if op == "rope":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, T=_log(rng, 1, 12000), H=H, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2]),
                    axes=axes, interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                    k_out=rng.random() < 0.5, far=_log(rng, 100, 1000000), dtype=dtype, bs=bs,
                    mix=mix)
    if op == "prompt":
        hi = _log(rng, 1, 6000)
        B = _log(rng, 1, max(1, min(64, 12000 // hi)))
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, H=H, Hkv=Hkv, D=D,
                    fused=rng.random() < 0.5, dtype=dtype, mix=mix)
    if op == "chunk":
        qhi = _log(rng, 1, 500)
        hi = _log(rng, 1, 8000)
        B = _log(rng, 1, max(1, min(32, 40000 // (hi + qhi), 4000 // qhi)))
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, qlo=rng.randint(0, qhi), qhi=qhi,
                    H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype, mix=mix)
    hi = _log(rng, 1, 100000)
    B = _log(rng, 1, max(1, min(128, 200000 // hi)))
    return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype,
                mix=mix)


# ---------------------------------------------------------------- inputs
def _sections(case):
    """The axis of each rotary pair: contiguous sections, the first axis's the shortest."""
    n = case["R"] // 2
    if case["axes"] == 1:
        return np.zeros(n, np.int64)
    first = n // 4 if case["axes"] == 3 else n // 2
    rest = np.arange(n - first) * (case["axes"] - 1) // (n - first) + 1
    return np.concatenate([np.zeros(first, np.int64), rest])


def _pool(case, cached, new, g, gen, dev):
    """Block tables of a shuffled pool for cached + new tokens, and the blocks left over."""
    bs = case["bs"]
    need = -(-(cached + new) // bs)
    M = int(need.max()) + 2
    NB = max(2, int(math.ceil(1.2 * need.sum())) + 4)
    ids = g.permutation(NB).astype(np.int32)
    return need, M, NB, ids


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    g = np.random.default_rng([int(seed), 77])
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(
            DTYPES[case["dtype"]])

    def whole(x, t):
        return torch.from_numpy(np.ascontiguousarray(x)).to(dev, t)

    st = {"case": dict(case)}
    if op == "plan":
        cached, new = _lens(case)
        bs = case["bs"]
        need, M, NB, ids = _pool(case, cached, new, g, gen, dev)
        have = -(-cached // bs)
        bt = np.full((len(need), M), -1, np.int32)
        at = 0
        for b in range(len(need)):
            bt[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        left = ids[at:]
        head = int(g.integers(0, 10 * NB))  # the ring has been around before
        ring = np.full(NB, -1, np.int32)
        ring[(head + np.arange(len(left))) % NB] = left
        Tmax = int(-(-max(1, new.sum()) // 64) * 64)  # a captured step's fixed size
        st.update(cached=whole(cached, torch.int32), new=whole(new, torch.int32),
                  tables=whole(bt, torch.int32), ring=whole(ring, torch.int32),
                  free=whole(np.array([head, head + len(left)]), torch.int64), Tmax=Tmax)
        if own:
            import paged_kv_cache_172_gb300 as pk
            st["out"] = pk.StepPlan.empty(len(need), Tmax, dev)
        return st
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if op == "rope":
        T, bs = case["T"], case["bs"]
        if case["fused"]:  # views of one projection's output
            qkv = normal(T, H + 2 * Hkv, D)
            q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            q, k, v = normal(T, H, D), normal(T, Hkv, D), normal(T, Hkv, D)
        pos = g.integers(0, case["far"], (case["axes"], T))
        NB = -(-T // bs) + 3
        slots = g.permutation(NB * bs)[:T].astype(np.int64)
        slots[g.random(T) < 0.02] = -1  # padding rows of a captured step
        inv = 10000.0 ** (-np.arange(case["R"] // 2) * 2.0 / case["R"])
        st.update(q=q, k=k, v=v, positions=whole(pos, torch.int32),
                  slots=whole(slots, torch.int64), inv=whole(inv, torch.float64),
                  axis=whole(_sections(case), torch.int64),
                  k_cache=torch.zeros(NB, bs, Hkv, D, dtype=DTYPES[case["dtype"]], device=dev))
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        st["q_out"] = torch.empty(T, H, D, dtype=q.dtype, device=dev)
        st["k_out"] = torch.empty(T, Hkv, D, dtype=q.dtype, device=dev) if case["k_out"] else None
        if own:
            import paged_kv_cache_172_gb300 as pk
            st["table"] = pk.pa_rope_table(inv, _sections(case), device=dev)
        return st
    cached, new = _lens(case)
    total = int(new.sum())
    offs = np.concatenate([[0], np.cumsum(new)])
    st.update(offsets=whole(offs, torch.int32), scale=1.0 / math.sqrt(D),
              Lmax=int(new.max()), Nmax=int((cached + new).max()))
    if op == "prompt":
        if case["fused"]:
            qkv = normal(total, H + 2 * Hkv, D)
            st.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
        else:
            st.update(q=normal(total, H, D), k=normal(total, Hkv, D), v=normal(total, Hkv, D))
    else:
        bs = case["bs"]
        need, M, NB, ids = _pool(case, cached, new, g, gen, dev)
        bt = np.full((len(need), M), -1, np.int32)
        at = 0
        for b in range(len(need)):
            bt[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        st.update(q=normal(total, H, D), k_cache=normal(NB, bs, Hkv, D),
                  v_cache=normal(NB, bs, Hkv, D), tables=whole(bt, torch.int32),
                  context=whole(cached + new, torch.int32))
    st["out"] = torch.empty(total, H, D, dtype=DTYPES[case["dtype"]], device=dev)
    if own and op in ("chunk", "decode"):  # workspaces, as a serving loop keeps them
        import paged_kv_cache_172_gb300 as pk
        B, M = st["tables"].shape
        if op == "chunk":
            n = pk.pa_chunk_attention_workspace_size(B, total, H, Hkv, D, M * case["bs"])
        else:
            n = pk.pa_decode_grouped_workspace_size(B, H, Hkv, D, case["bs"], st["Nmax"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    return st


# ---------------------------------------------------------------- plain forms
def _plain_plan(st):
    bs, ring, bt = st["case"]["bs"], st["ring"], st["tables"]
    c, n = st["cached"].long(), st["new"].long()
    NB, M = ring.numel(), bt.shape[1]
    have, want = (c + bs - 1) // bs, (c + n + bs - 1) // bs
    need = want - have
    free = st["free"]
    fits = (need.sum() <= free[1] - free[0]) & (n.sum() <= st["Tmax"])
    n, need, want = n * fits, need * fits, torch.where(fits, want, have)
    ends, before = torch.cumsum(n, 0), torch.cumsum(need, 0) - need
    i = torch.arange(M, device=bt.device)
    taken = (free[0] + before[:, None] + i - have[:, None]) % NB
    fresh = (i >= have[:, None]) & (i < want[:, None])
    bt.copy_(torch.where(fresh, ring[taken], bt))
    t = torch.arange(st["Tmax"], device=bt.device)
    seq = (t[:, None] >= ends).sum(1)
    real = seq < c.numel()
    seq = torch.where(real, seq, 0)
    pos = torch.where(real, c[seq] + t - (ends - n)[seq], 0)
    slot = torch.where(real, bt[seq, pos // bs].long() * bs + pos % bs, -1)
    zero = torch.zeros(1, dtype=ends.dtype, device=bt.device)
    return {"tables": bt, "context_lens": (c + n).int(), "q_offsets": torch.cat([zero, ends]).int(),
            "slot_mapping": slot, "positions": pos.int(),
            "free_state": torch.stack([free[0] + need.sum(), free[1]])}


def _turn(x, cos, sin, R, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([r, x[..., R:]], -1)


def _plain_rope(st):
    case = st["case"]
    pos = st["positions"].double()[st["axis"]].T  # [T, R / 2]
    angle = pos * st["inv"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _turn(st["q"], cos, sin, case["R"], case["interleaved"]).to(st["q"].dtype)
    k = _turn(st["k"], cos, sin, case["R"], case["interleaved"]).to(st["q"].dtype)
    keep = st["slots"] >= 0
    rows = st["k_cache"].flatten(0, 1)
    rows[st["slots"][keep]] = k[keep]
    rows = st["v_cache"].flatten(0, 1)
    rows[st["slots"][keep]] = st["v"][keep]
    return {"q": q, "k": k if case["k_out"] else None, "k_cache": st["k_cache"],
            "v_cache": st["v_cache"]}


def _plain_attention(q, k, v, new, ctx, scale):
    """q [B, L, H, D], k, v [B, N, Hkv, D], new and ctx [B]: query i of a sequence is at
    position ctx - new + i and sees the keys up to itself.  Softmax in 32 bits."""
    B, L, H, D = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    i, j = torch.arange(L, device=q.device), torch.arange(N, device=q.device)
    seen = j <= (ctx - new)[:, None, None] + i[:, None]
    seen &= (j < ctx[:, None, None]) & (i[:, None] < new[:, None, None])
    there = (j < ctx[:, None])[:, :, None, None]
    k, v = torch.where(there, k.float(), 0.0), torch.where(there, v.float(), 0.0)
    q = q.float().reshape(B, L, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, Hkv, -1, D) * scale
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).reshape(B, Hkv, -1, L, N)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(B, Hkv, -1, N), v.permute(0, 2, 1, 3)).reshape(B, Hkv, -1, L, D)
    o = torch.where(total > 0, o / total.clamp_min(1e-30), 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, L, H, D)


def _padded(x, offsets, L):
    """Packed rows as [B, L, ...]; the rows past a sequence's end hold others' values."""
    at = offsets[:-1, None].long() + torch.arange(L, device=x.device)
    return x[at.clamp_max(x.shape[0] - 1)]


def _plain_packed(st):
    offs = st["offsets"].long()
    new = offs[1:] - offs[:-1]
    L = st["Lmax"]
    if st["case"]["op"] == "prompt":
        ctx = new
        k, v = _padded(st["k"], offs, L), _padded(st["v"], offs, L)
    else:
        ctx = st["context"].long()
        bs = st["case"]["bs"]
        bt = st["tables"][:, :-(-st["Nmax"] // bs)].clamp_min(0).long()
        k, v = st["k_cache"][bt].flatten(1, 2), st["v_cache"][bt].flatten(1, 2)
    o = _plain_attention(_padded(st["q"], offs, L), k, v, new, ctx, st["scale"])
    i = torch.arange(L, device=o.device)
    return o[i < new[:, None]].to(st["q"].dtype)


def run(st):
    op, case = st["case"]["op"], st["case"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope}.get(op, _plain_packed)(st)
    import paged_kv_cache_172_gb300 as pk
    if op == "plan":
        p = pk.pa_step_plan(st["cached"], st["new"], st["tables"], st["ring"], st["free"],
                            case["bs"], st["Tmax"], out=st["out"])
        return {"tables": st["tables"], "context_lens": p.context_lens, "q_offsets": p.q_offsets,
                "slot_mapping": p.slot_mapping, "positions": p.positions,
                "free_state": p.free_state}
    if op == "rope":
        q, k = pk.pa_rope_cache_write(st["q"], st["k"], st["v"], st["positions"], st["table"],
                                      st["slots"], st["k_cache"], st["v_cache"],
                                      interleaved=case["interleaved"], q_out=st["q_out"],
                                      k_out=st["k_out"])
        return {"q": q, "k": k, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if op == "prompt":
        return pk.pa_prompt_attention(st["q"], st["k"], st["v"], st["offsets"], st["scale"],
                                      out=st["out"])
    if op == "chunk":
        return pk.pa_chunk_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                     st["context"], st["offsets"], st["scale"], out=st["out"],
                                     workspace=st["ws"])
    return pk.pa_decode_grouped(st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                st["context"], st["scale"], st["Nmax"], out=st["out"],
                                workspace=st["ws"])


# ---------------------------------------------------------------- what cannot be done without
def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lens(case)
        have, want = -(-cached // case["bs"]), -(-(cached + new) // case["bs"])
        fresh = int((want - have).sum())
        T = int(-(-max(1, new.sum()) // 64) * 64)
        # both lengths, the ring's ids into the tables, the cached blocks that new tokens
        # continue, then context, offsets, slots, positions and the ring's state
        return {"bytes": 16 * len(new) + 4 + 8 * fresh + 4 * int((cached % case["bs"] > 0).sum())
                + 12 * T + 32, "flops": 0}
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if op == "rope":
        T, row = case["T"], 2 * D
        rows = 2 * H + (5 if case["k_out"] else 4) * Hkv
        return {"bytes": T * (rows * row + 8 + 4 * case["axes"]) + 8 * (case["R"] // 2),
                "flops": T * (H + Hkv) * case["R"] * 3}
    cached, new = _lens(case)
    total, ctx = int(new.sum()), cached + new
    pairs = int((new * cached + new * (new + 1) // 2).sum())
    bytes_ = 2 * total * H * D * 2 + 4 * (len(new) + 1)
    if op == "prompt":
        bytes_ += 2 * total * Hkv * D * 2
    else:
        live = np.where(new > 0, ctx, 0)
        bytes_ += 2 * int(live.sum()) * Hkv * D * 2 + 4 * int((-(-live // case["bs"])).sum())
        bytes_ += 4 * len(new)
    return {"bytes": bytes_, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None  # whole numbers: compared with the plain form's, bit for bit
    if op == "rope":
        R = case["R"]
        axis, inv = st["axis"].cpu().numpy(), st["inv"].cpu().numpy()
        pos = st["positions"].cpu().numpy().astype(np.float64)
        z = np.exp(1j * (pos[axis] * inv[:, None]).T)  # a rotation is a complex product
        z = torch.from_numpy(z).to(st["q"].device)[:, None]
        lo = torch.arange(0, R, 2) if case["interleaved"] else torch.arange(R // 2)
        hi = lo + 1 if case["interleaved"] else lo + R // 2
        got = {}
        for name in ("q", "k"):
            x = st[name].double().clone()
            w = torch.complex(x[..., lo], x[..., hi]) * z
            x[..., lo], x[..., hi] = w.real, w.imag
            got[name] = x
        keep = st["slots"] >= 0
        for name, rows in (("k_cache", got["k"]), ("v_cache", st["v"].double())):
            c = st[name].double().flatten(0, 1)
            c[st["slots"][keep]] = rows[keep]
            got[name] = c.reshape(st[name].shape)
        if not case["k_out"]:
            got["k"] = None
        return got
    cached, new = _lens(case)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if 4 * D * H * float((new * (cached + new)).sum()) > 1.2e13:
        return None
    out = torch.zeros(int(new.sum()), H, D, dtype=torch.float64, device=st["q"].device)
    at = 0
    for b in range(len(new)):
        n, N = int(new[b]), int(cached[b] + new[b])
        if n == 0:
            continue
        if op == "prompt":
            k, v = st["k"][at:at + n].double(), st["v"][at:at + n].double()
        else:
            t = torch.arange(N, device=out.device)
            blk = st["tables"][b].long()[t // case["bs"]]
            k = st["k_cache"][blk, t % case["bs"]].double()
            v = st["v_cache"][blk, t % case["bs"]].double()
        for g in range(Hkv):
            heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                last = N - n + i1  # no query here sees a key past this one
                q = st["q"][at + i0:at + i1, heads].double().transpose(0, 1)
                w = torch.einsum("hid,jd->hij", q, k[:last, g]) / math.sqrt(D)
                j = torch.arange(last, device=out.device)
                i = torch.arange(i0, i1, device=out.device)
                w = w.masked_fill(j[None, :] > i[:, None] + (N - n), -math.inf)
                p = torch.softmax(w, -1)
                out[at + i0:at + i1, heads] = torch.einsum("hij,jd->ihd", p, v[:last, g])
        at += n
    return out
