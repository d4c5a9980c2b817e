"""Cases of generation with an encoder's states and beams: cross attention, beam selection,
the reordering of a paged cache's block tables, and the way back through the beams, with
their plain forms in torch.

A beam-searching decoder runs them in this order each step: its queries attend to the
encoder's states; the best continuations over beams and vocabulary are chosen; the block
tables follow the chosen beams; and at the end the hypotheses' tokens are gathered along
their parents.  ``run`` computes one of them, in its plain form or (``own``) through this
package.  The lengths of a case come from the case itself (``mix`` seeds them), the data
from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's token with four beams over the states of a 30-second recording: latency
        dict(name="cross_beams_single", op="cross", B=1, qlo=4, qhi=4, lo=1500, hi=1500, H=16,
             Hkv=16, D=64, dtype="fp16", states="pool", mix=21),
        # a step of a translating batch: four beams each, sources of very different lengths
        dict(name="cross_beams_batch", op="cross", B=32, qlo=4, qhi=4, lo=200, hi=1500, H=16,
             Hkv=16, D=64, dtype="fp16", states="pool", mix=22),
        # few requests over whole documents, grouped heads: the states' bandwidth
        dict(name="cross_beams_long", op="cross", B=4, qlo=4, qhi=4, lo=30000, hi=65536, H=32,
             Hkv=8, D=128, dtype="bf16", states="fused", mix=23),
        # decoder prompts and drafts of many lengths, one without states
        dict(name="cross_prompts", op="cross", B=16, qlo=1, qhi=400, lo=0, hi=4096, H=40, Hkv=8,
             D=128, dtype="fp16", states="fused", mix=24),
        # the encoder's own attention over a ragged batch: every token sees every other
        dict(name="encoder_batch", op="cross", B=8, qlo=500, qhi=4096, lo=0, hi=0, H=16, Hkv=16,
             D=64, dtype="bf16", states="self", mix=25),
        # one user's beams: latency
        dict(name="select_single", op="select", B=1, W=4, V=32000, dtype="fp32", padded=False,
             mix=26),
        # a batch, an odd vocabulary, logits as the model wrote them
        dict(name="select_batch", op="select", B=64, W=4, V=50001, dtype="bf16", padded=False,
             mix=27),
        # wide beams and a large vocabulary, rows padded to whole tiles
        dict(name="select_wide", op="select", B=32, W=16, V=255999, dtype="fp32", padded=True,
             mix=28),
        # a batch in the middle of its answers
        dict(name="reorder_batch", op="reorder", B=32, W=4, lo=64, hi=512, bs=16, mix=29),
        # many requests with long contexts
        dict(name="reorder_long", op="reorder", B=256, W=8, lo=500, hi=8000, bs=16, mix=30),
        # the best hypothesis of each of a batch of short answers
        dict(name="backtrack_best", op="backtrack", B=32, W=4, K=1, S=100, mix=31),
        # every hypothesis of long ones
        dict(name="backtrack_all", op="backtrack", B=64, W=8, K=8, S=2048, mix=32),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["cross"] * 4 + ["select"] * 3 + ["reorder"] * 2 + ["backtrack"])
    mix = rng.randrange(1 << 30)
    if op == "cross":
        H, Hkv = rng.choice([(8, 8), (16, 16), (12, 12), (16, 4), (32, 8), (40, 8), (12, 4),
                             (16, 1)])
        case = dict(op=op, H=H, Hkv=Hkv, D=rng.choice([64, 64, 128]),
                    dtype=rng.choice(["fp16", "bf16"]), mix=mix)
        kind = rng.choice(["beams", "beams", "prompts", "self"])
        row = 4 * case["D"] * H  # operations of a query and a key
        if kind == "self":
            hi = min(_log(rng, 1, 4000), int(math.sqrt(1.7e11 / row)))
            B = _log(rng, 1, max(1, min(64, 12000 // hi, int(1.7e11 / row) // (hi * hi))))
            return dict(case, B=B, qlo=rng.randint(0, hi), qhi=hi, lo=0, hi=0, states="self")
        qhi = _log(rng, 1, 16) if kind == "beams" else _log(rng, 1, 1000)
        hi = _log(rng, 1, 50000 if kind == "beams" else 8000)
        B = _log(rng, 1, max(1, min(96, 4000 // qhi, int(1.7e11 / row) // (qhi * hi),
                                    int(8e8) // (4 * case["D"] * Hkv * hi))))
        return dict(case, B=B, qlo=qhi if kind == "beams" else rng.randint(0, qhi), qhi=qhi,
                    lo=rng.randint(0, hi), hi=hi, states=rng.choice(["pool", "fused", "padded"]))
    if op == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
        V = _log(rng, 40, 260000)
        B = _log(rng, 1, max(1, min(256, 100_000_000 // (W * V))))
        return dict(op=op, B=B, W=W, V=V, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    padded=rng.random() < 0.5, mix=mix)
    if op == "reorder":
        W = rng.choice([2, 3, 4, 5, 8, 16])
        hi = _log(rng, 1, 8000)
        B = _log(rng, 1, max(1, min(256, 40_000_000 // (W * W * hi) + 1)))
        return dict(op=op, B=B, W=W, lo=rng.randint(0, hi), hi=hi, bs=rng.choice([8, 16, 16, 32]),
                    mix=mix)
    W = rng.choice([2, 3, 4, 5, 8, 16])
    S = _log(rng, 1, 2048)
    return dict(op=op, B=_log(rng, 1, max(1, min(256, 1_000_000 // (W * S)))), W=W,
                K=rng.choice([1, W]), S=S, mix=mix)


# ---------------------------------------------------------------- lengths of a case
def _spread(rng, B, lo, hi):
    """B lengths in [lo, hi], the first one hi, so that the case's size is what it says."""
    x = rng.integers(lo, hi + 1, B)
    x[0] = hi
    return x.astype(np.int64)


def _lens(case):
    """Query and state lengths of a cross attention's requests, two int64 arrays."""
    rng = np.random.default_rng(case["mix"])
    q = _spread(rng, case["B"], case["qlo"], case["qhi"])
    return q, q if case["states"] == "self" else _spread(rng, case["B"], case["lo"], case["hi"])


def _live(case):
    """Beams that are alive, [B, W] truth values: some requests take their first step, with one
    beam, some are done."""
    rng = np.random.default_rng(case["mix"])
    live = np.ones((case["B"], case["W"]), bool)
    kind = rng.random(case["B"])
    kind[0] = 1.0
    live[kind < 0.15, 1:] = False
    live[kind < 0.05] = False
    return live


def _contexts(case):
    return _spread(np.random.default_rng(case["mix"]), case["B"], case["lo"], case["hi"])


# ---------------------------------------------------------------- inputs
def _beam_tables(case, g):
    """Block tables of beams that have parted on their way, their lengths, the ids left, and
    the pool's blocks."""
    B, W, bs = case["B"], case["W"], case["bs"]
    lens = _contexts(case)
    need = -(-lens // bs)
    M = int(need.max()) + 2
    rows = np.full((B, W, M), -1, np.int64)
    prompt = (need * g.uniform(0.0, 0.9, B)).astype(np.int64)
    at = 0
    for i in range(int(need.max())):
        one = (i < prompt)[:, None] & np.ones(W, bool)
        ids = np.where(one, at + np.arange(B)[:, None], at + B + np.arange(B * W).reshape(B, W))
        at += B + B * W
        if i % 3 == 2:  # beams have followed others since the last column
            p = np.sort(g.integers(0, W, (B, W)), 1)
            rows = np.take_along_axis(rows, p[:, :, None], 1)
        rows[:, :, i] = np.where((i < need)[:, None], ids, -1)
    used, where = np.unique(rows, return_inverse=True)
    n = len(used) - (used[0] < 0)  # ids in use
    NB = W * int(need.sum()) + max(8, B * W)  # (as if nothing were shared)
    ids = g.permutation(NB)
    table = np.concatenate([[-1], ids[:n]]) if used[0] < 0 else ids[:n]
    return table[where.reshape(rows.shape)], np.repeat(lens, W), ids[n:], NB


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    g = np.random.default_rng([int(seed), 78])
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(
            DTYPES[case["dtype"]])

    def whole(x, t=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(x)).to(dev, t)

    st = {"case": dict(case)}
    if op == "cross":
        H, Hkv, D = case["H"], case["Hkv"], case["D"]
        ql, n = _lens(case)
        T, B = int(ql.sum()), case["B"]
        if case["states"] == "self":  # views of one projection's output
            qkv = normal(T, H + 2 * Hkv, D)
            q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
            starts = np.cumsum(ql) - ql
        else:
            q = normal(T, H, D)
            if case["states"] == "padded":
                starts, rows = np.arange(B) * case["hi"], B * case["hi"]
            else:  # requests in the order they came in, with what others left between them
                order = g.permutation(B)
                room = n + g.integers(0, 9, B)
                starts = np.empty(B, np.int64)
                starts[order] = np.cumsum(room[order]) - room[order]
                rows = int(room.sum())
            if case["states"] == "pool":
                k, v = normal(max(1, rows), Hkv, D), normal(max(1, rows), Hkv, D)
            else:
                kv = normal(max(1, rows), 2 * Hkv, D)
                k, v = kv[:, :Hkv], kv[:, Hkv:]
        st.update(q=q, k=k, v=v, starts=whole(starts), lens=whole(n), scale=1.0 / math.sqrt(D),
                  offsets=whole(np.concatenate([[0], np.cumsum(ql)])), Lmax=int(ql.max()),
                  Nmax=int(n.max()), out=torch.empty(T, H, D, dtype=q.dtype, device=dev))
        if own:
            import paged_kv_cache_172_gb300 as pk
            size = pk.pa_cross_attention_workspace_size(B, T, H, Hkv, D, st["Lmax"], st["Nmax"])
            st["ws"] = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        return st
    if op == "select":
        B, W, V = case["B"], case["W"], case["V"]
        live = _live(case)
        cols = -(-V // 64) * 64 if case["padded"] else V
        logits = normal(B * W, cols)
        logits *= 2.5
        # what a model is sure of, and what a request does not allow
        sure = torch.randint(0, V, (B * W,), generator=gen, device=dev)
        rows = torch.arange(B * W, device=dev)
        logits[rows, sure] += whole(g.uniform(0, 12, B * W), logits.dtype)
        logits[:, torch.randint(0, V, (V // 100,), generator=gen, device=dev)] = -math.inf
        scores = -np.sort(g.uniform(0, 6, (B, W)), 1) - g.uniform(0, 30, (B, 1))
        scores = np.where(live, scores, -np.inf)
        st.update(logits=logits[:, :V], scores=whole(scores, torch.float32),
                  eos=int(g.integers(0, V)), pad=0)
        # an end that is as likely as other continuations
        logits[:, st["eos"]] = logits[:, :V].amax(1) - 1.0
        if own:
            import paged_kv_cache_172_gb300 as pk
            st["out"] = pk.BeamStep.empty(B, W, dev)
            size = pk.pa_beam_select_workspace_size(B, W, V)
            st["ws"] = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        return st
    if op == "reorder":
        B, W, bs = case["B"], case["W"], case["bs"]
        rows, lens, left, NB = _beam_tables(case, g)
        parents = np.sort(g.integers(0, W, (B, W)), 1)
        kind = g.random(B)
        parents[kind < 0.2] = np.arange(W)  # nothing moves
        parents[kind < 0.05] = -1  # done: its blocks come back
        head = int(g.integers(0, 10 * NB))
        ring = np.full(NB, -1, np.int64)
        ring[(head + np.arange(len(left))) % NB] = left
        M = rows.shape[2]
        shared = np.minimum(g.integers(0, 2, B) * bs * g.integers(0, 4, B), lens[::W])
        st.update(parents=whole(parents), tables=whole(rows.reshape(B * W, M)),
                  context=whole(lens), ring=whole(ring),
                  free=whole(np.array([head, head + len(left)]), torch.int64),
                  shared=whole(shared))
        if own:
            import paged_kv_cache_172_gb300 as pk
            st["out"] = pk.BeamTables.empty(B * W, M, dev)
        return st
    B, W, K, S = case["B"], case["W"], case["K"], case["S"]
    lengths = g.integers(max(0, S // 2), S + 1, (B, K))
    lengths[0, 0] = S
    st.update(tokens=whole(g.integers(0, 50000, (S, B, W))),
              parents=whole(np.sort(g.integers(0, W, (S, B, W)), 2)), lengths=whole(lengths),
              beams=whole(g.integers(0, W, (B, K))), pad=-1,
              out=torch.empty(B, K, S, dtype=torch.int32, device=dev))
    return st


# ---------------------------------------------------------------- plain forms
def _plain_cross(st):
    """Every request's queries and states padded to the longest; softmax in 32 bits."""
    offs, n, L, N = st["offsets"].long(), st["lens"].long(), st["Lmax"], st["Nmax"]
    ql = offs[1:] - offs[:-1]
    i = torch.arange(L, device=offs.device)
    j = torch.arange(N, device=offs.device)
    q = st["q"][(offs[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)].float()  # [B, L, H, D]
    at = (st["starts"].long()[:, None] + j).clamp_max(st["k"].shape[0] - 1)
    there = (j < n[:, None])[:, :, None, None]
    k = torch.where(there, st["k"][at].float(), 0.0)
    v = torch.where(there, st["v"][at].float(), 0.0)
    B, _, H, D = q.shape
    Hkv = k.shape[2]
    q = q.reshape(B, L, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q * st["scale"], k.permute(0, 2, 3, 1))
    s.masked_fill_(j >= n[:, None, None, None], float("-inf"))
    if N:
        s.sub_(s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v.permute(0, 2, 1, 3))
    o = torch.where(total > 0, o / total.clamp_min(1e-30), 0.0)
    o = o.reshape(B, Hkv, -1, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, H, D)
    return o[i < ql[:, None]].to(st["q"].dtype)


def _plain_select(st):
    """Scores in 64 bits: the next candidate may be a rounding of 32 away."""
    B, W = st["scores"].shape
    x = st["logits"].double().reshape(B, W, -1)
    V = x.shape[2]
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    score = st["scores"].double()[..., None]
    c = torch.where(torch.isfinite(score) & torch.isfinite(lse), score + (x - lse), -math.inf)
    end = c[..., st["eos"]].clone()
    c[..., st["eos"]] = -math.inf
    # (a stable sort of all candidates would do; the W best of a row come first)
    best, token = _top(c, W)
    best, at = _top(best.reshape(B, -1), W)
    token = token.reshape(B, -1).gather(1, at)
    parent = at // min(W, V)
    if best.shape[1] < W:
        more = W - best.shape[1]
        best, token, parent = (torch.cat([t, t.new_full((B, more), f)], 1) for t, f in
                               ((best, -math.inf), (token, 0), (parent, 0)))
    none = best == -math.inf
    own_index = torch.arange(W, device=x.device).expand(B, W)
    last = best[:, -1:]
    w = own_index
    ahead = (end > last) | ((end == last) & _before(w, st["eos"], parent[:, -1:], token[:, -1:]))
    return {"tokens": torch.where(none, st["pad"], token).int(),
            "parents": torch.where(none, own_index, parent).int(), "scores": best.float(),
            "ended": torch.where(ahead & (end > -math.inf), end, -math.inf).float()}


def _before(w, v, w2, v2):
    return (w < w2) | ((w == w2) & (v < v2))


def _top(x, k):
    """The k largest of the last axis and where they are, ties to the lowest index."""
    k = min(k, x.shape[-1])
    kth = torch.topk(x, k, -1).values[..., -1:]
    above = x > kth
    rank = torch.cumsum(x == kth, -1)
    keep = above | ((x == kth) & (rank <= k - above.sum(-1, keepdim=True)))
    at = keep.nonzero()[:, -1].reshape(*x.shape[:-1], k)  # k of every row, in order
    got, order = torch.sort(x.gather(-1, at), dim=-1, descending=True, stable=True)
    return got, at.gather(-1, order)


def _plain_reorder(st):
    case, bt, ring, free = st["case"], st["tables"].long(), st["ring"].long(), st["free"]
    B, W, bs = case["B"], case["W"], case["bs"]
    M, NB, dev = bt.shape[1], ring.numel(), bt.device
    old, lens, p = bt.reshape(B, W, M), st["context"].long().reshape(B, W), st["parents"].long()
    col, beam = torch.arange(M, device=dev), torch.arange(W, device=dev)
    here = p >= 0
    src = p.clamp_min(0)
    new_lens = torch.where(here, lens.gather(1, src), 0)
    had, has = (lens + bs - 1) // bs, (new_lens + bs - 1) // bs
    held, holds = col < had[..., None], col < has[..., None]
    new = torch.where(holds, old.gather(1, src[..., None].expand(B, W, M)), -1)
    # the last block, half full, of a beam that is not the first to hold it: a copy
    tail = (has - 1).clamp_min(0)
    tail_id = new.gather(2, tail[..., None])[..., 0]
    part = (new_lens % bs != 0) & (tail_id >= 0) & (tail_id < NB)
    same = (tail_id[:, :, None] == tail_id[:, None]) & (tail[:, :, None] == tail[:, None])
    need = part & (same & part[:, None] & (beam < beam[:, None])).any(2)
    taken = need.sum()
    fits = taken <= free[1] - free[0]
    rank = torch.cumsum(need.flatten(), 0).reshape(B, W) - 1
    fresh = ring[(free[0] + rank) % NB]
    moved = new
    new = torch.where(need[..., None] & (col == tail[..., None]), fresh[..., None], new)
    pairs = torch.where(need[..., None], torch.stack([tail_id, fresh], -1), 0)
    # blocks that no beam of the request holds any more, by column and beam
    kept = ((old[:, :, None] == moved[:, None]) & holds[:, None]).any(2)
    again = ((old[:, :, None] == old[:, None]) & held[:, None]
             & (beam < beam[:, None])[None, :, :, None]).any(2)
    own_col = col >= (st["shared"].long() // bs)[:, None]
    drop = held & ~kept & ~again & own_col[:, None] & (old >= 0) & (old < NB)
    drop = drop.transpose(1, 2).flatten() & fits
    put = torch.where(drop, (free[1] + torch.cumsum(drop, 0) - 1) % NB, NB)
    ring = torch.cat([ring, ring[:1]])
    ring[put] = old.transpose(1, 2).flatten()
    state = torch.stack([free[0] + taken * fits, free[1] + drop.sum()])
    return {"tables": torch.where(fits, new, old).reshape(B * W, M).int(),
            "context": torch.where(fits, new_lens, lens).flatten().int(),
            "ring": ring[:NB].int(), "free": state,
            "pairs": torch.where(fits, pairs, 0).reshape(B * W, 2)}


def _plain_backtrack(st):
    """By doubling: which beam of step s - 2^k a beam of step s comes from, for each k."""
    tokens, jump = st["tokens"].long(), st["parents"].long()
    n, beam = st["lengths"].long(), st["beams"].long()
    S, B, W = tokens.shape
    K = n.shape[1]
    step = torch.arange(S, device=n.device)
    left = (n[..., None] - 1 - step).clamp_min(0)  # [B, K, S] steps to go back
    at = (n[..., None] - 1).expand(B, K, S).clamp_min(0)
    beam = beam[..., None].expand(B, K, S)
    b = torch.arange(B, device=n.device)[:, None, None]
    for k in range(max(1, (S - 1).bit_length())):
        go = (left >> k) & 1 == 1
        beam = torch.where(go, jump[at, b, beam], beam)
        at = torch.where(go, at - (1 << k), at)
        jump = jump[(step - (1 << k)).clamp_min(0)].gather(2, jump)
    seen = step < n[..., None]
    return torch.where(seen, tokens[step, b, beam], st["pad"]).int()


def run(st):
    op, case = st["case"]["op"], st["case"]
    if not own:
        return {"cross": _plain_cross, "select": _plain_select, "reorder": _plain_reorder,
                "backtrack": _plain_backtrack}[op](st)
    import paged_kv_cache_172_gb300 as pk
    if op == "cross":
        return pk.pa_cross_attention(st["q"], st["k"], st["v"], st["offsets"], st["starts"],
                                     st["lens"], st["scale"], st["Lmax"], st["Nmax"],
                                     out=st["out"], workspace=st["ws"])
    if op == "select":
        s = pk.pa_beam_select(st["logits"], st["scores"], eos_token=st["eos"],
                              pad_token=st["pad"], out=st["out"], workspace=st["ws"])
        return {"tokens": s.tokens, "parents": s.parents, "scores": s.scores,
                "ended": s.ended_scores}
    if op == "reorder":
        t = pk.pa_beam_reorder(st["parents"], st["tables"], st["context"], st["ring"], st["free"],
                               case["bs"], shared_lens=st["shared"], out=st["out"])
        return {"tables": t.block_tables, "context": t.context_lens, "ring": st["ring"],
                "free": t.free_state, "pairs": t.copy_pairs}
    return pk.pa_beam_backtrack(st["tokens"], st["parents"], st["lengths"], st["beams"],
                                pad_token=st["pad"], out=st["out"])


# ---------------------------------------------------------------- what cannot be done without
def work(case):
    op = case["op"]
    if op == "cross":
        H, Hkv, D = case["H"], case["Hkv"], case["D"]
        ql, n = _lens(case)
        keys = int(np.where(ql > 0, n, 0).sum())
        return {"bytes": 4 * int(ql.sum()) * H * D + 4 * keys * Hkv * D + 12 * len(ql) + 4,
                "flops": 4 * D * H * int((ql * n).sum())}
    if op == "select":
        B, W, V = case["B"], case["W"], case["V"]
        rows = int(_live(case).sum())
        return {"bytes": rows * V * (4 if case["dtype"] == "fp32" else 2) + 20 * B * W,
                "flops": 4 * rows * V}
    if op == "reorder":
        B, W, bs = case["B"], case["W"], case["bs"]
        need = -(-_contexts(case) // bs)
        # tables to their lengths, parents and lengths; all of the new tables, lengths, pairs
        return {"bytes": 4 * W * int(need.sum()) + 8 * B * W
                + 4 * B * W * (int(need.max()) + 2) + 20 * B * W, "flops": 0}
    B, W, K, S = (case[x] for x in ("B", "W", "K", "S"))
    return {"bytes": 4 * B * S * W + 8 * B * K * S + 8 * B * K, "flops": 0}


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("reorder", "backtrack"):
        return None  # whole numbers: compared with the plain form's, bit for bit
    st = prepare(case, seed)
    dev = st["scores"].device if op == "select" else st["q"].device
    if op == "select":
        B, W = st["scores"].shape
        scores, ended = [], []
        for b in range(B):
            row = torch.log_softmax(st["logits"][b * W:(b + 1) * W].double(), -1)
            row = row + st["scores"][b].double()[:, None]
            row = torch.where(row.isnan(), -math.inf, row)
            # all candidates in order, those that end among them
            row, order = torch.sort(row.flatten(), descending=True, stable=True)
            ends = order % case["V"] == st["eos"]
            live = torch.cumsum(~ends, 0)
            got = row[~ends & (live <= W)]
            scores.append(torch.cat([got, got.new_full((W - got.numel(),), -math.inf)]))
            end = torch.full((W,), -math.inf, dtype=torch.float64, device=dev)
            on_time = ends & (live < W)
            end[order[on_time] // case["V"]] = row[on_time]
            ended.append(end)
        return {"tokens": None, "parents": None, "scores": torch.stack(scores),
                "ended": torch.stack(ended)}
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    ql, n = _lens(case)
    if 4 * D * H * float((ql * n).sum()) > 6e12:
        return None
    out = torch.zeros(int(ql.sum()), H, D, dtype=torch.float64, device=dev)
    starts = st["starts"].tolist()
    at = 0
    for b in range(case["B"]):
        rows = slice(at, at + int(ql[b]))
        at += int(ql[b])
        keys = slice(starts[b], starts[b] + int(n[b]))
        if ql[b] == 0 or n[b] == 0:
            continue
        for h in range(H):
            w = st["q"][rows, h].double() @ st["k"][keys, h * Hkv // H].double().T
            p = torch.softmax(w / math.sqrt(D), -1)
            out[rows, h] = p @ st["v"][keys, h * Hkv // H].double()
    return out
