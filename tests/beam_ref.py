"""Plain implementations of the beam calls, one element after the other, in 64 bits.

pa_beam_select against them.  Which candidates are chosen is exact within a beam; between
beams the kernel's log-sum-exp is off by at most lse_error(V).  Relative to the sum:
  24 * 2^-23       a weight's argument: the difference from the maximum and its product with
                   log2 e, 2^-24 each, of at most 24 nats that still count, whether taken at
                   once or in the steps of its rescalings
  2^-22 + 2^-24    each exponential, with its product: a weight's own, one to each rise of its
                   lane's maximum (one a chunk of 512 at most; 24 are not seen in a lane of
                   values in random order), one where lanes are joined and one where pieces are
  2^-24            each addition: 8 within a chunk, V / 512 chunks and 1, 5 where lanes are
                   joined and 6 where pieces are
and 2^-25 of the logarithm.  So a chosen list that differs from the reference is right when
every place's score is within that of the reference's; scores are compared with it and half
a step of fp32."""
import math

import numpy as np


def lse_error(V, rises=24):
    chunks = V // 512 + 1
    return (24 * 2.0 ** -23 + (3 + min(rises, chunks)) * (2.0 ** -22 + 2.0 ** -24)
            + (chunks + 20) * 2.0 ** -24 + 2.0 ** -25)


def select(logits, scores, eos=-1, pad=0):
    """logits [B*W, V], scores [B, W] (numpy, any float type).  Dict of [B, W] arrays with
    scores in 64 bits, and `bad`: whether a live beam's logits were none."""
    B, W = scores.shape
    x = logits.astype(np.float64).reshape(B, W, -1)
    V = x.shape[2]
    tokens, parents = np.full((B, W), pad, np.int64), np.tile(np.arange(W), (B, 1))
    best, ended = np.full((B, W), -np.inf), np.full((B, W), -np.inf)
    bad = False
    for b in range(B):
        cand, ends = [], []
        for w in range(W):
            s = float(scores[b, w])
            if not math.isfinite(s):
                continue
            row = x[b, w]
            top = row.max()
            if np.isnan(top) or top == np.inf:
                bad = True
                continue
            if top == -np.inf:
                continue
            lse = top + math.log(np.exp(row - top).sum())
            live = np.argsort(-row, kind="stable")[:W + 1]
            live = [i for i in live if i != eos and row[i] > -np.inf][:W]
            cand += [(-(s + (row[i] - lse)), w, -row[i], int(i)) for i in live]
            if 0 <= eos < V and row[eos] > -np.inf:
                ends.append((-(s + (row[eos] - lse)), w, -row[eos], eos))
        cand = sorted(cand)[:W]
        for j, (c, w, _, i) in enumerate(cand):
            tokens[b, j], parents[b, j], best[b, j] = i, w, -c
        for e in ends:
            if len(cand) < W or e < cand[-1]:
                ended[b, e[1]] = -e[0]
    return dict(tokens=tokens, parents=parents, scores=best, ended=ended, bad=bad)


def compare(out, logits, scores, eos, pad, rises=24):
    """What pa_beam_select gave (tensors) against select()."""
    x, s = logits.double().cpu().numpy(), scores.cpu().numpy()
    ref = select(x, s, eos, pad)
    V = logits.shape[1]
    tol = lse_error(V, rises)
    got = [t.cpu().numpy() for t in out]
    fine = np.isfinite(ref["scores"])
    assert (np.isfinite(got[2]) == fine).all()
    top = np.abs(ref["scores"], where=fine, out=np.zeros_like(ref["scores"])).max()
    half = 2.0 ** -24 * top + tol
    assert (np.abs(got[2][fine] - ref["scores"][fine]) <= half).all()
    # a different choice only where two beams' candidates are as near as the sums' error
    B, W = s.shape
    for b, j in zip(*np.nonzero((got[0] != ref["tokens"]) | (got[1] != ref["parents"]))):
        w, v = int(got[1][b, j]), int(got[0][b, j])
        assert fine[b, j] and 0 <= v < V and v != eos, (b, j, w, v)
        row = x[b * W + w]
        m = row.max()
        c = s[b, w] + (row[v] - (m + math.log(np.exp(row - m).sum())))
        assert abs(c - ref["scores"][b, j]) <= 2 * tol, (b, j, w, v)
        assert len({(int(p), int(t)) for p, t in zip(got[1][b], got[0][b])}) == W
    ends = np.isfinite(ref["ended"])
    off = ends != np.isfinite(got[3])
    if off.any():
        b, w = (i[0] for i in np.nonzero(off))
        assert False, (b, w, got[3][b], ref["ended"][b], ref["scores"][b])
    top = np.abs(ref["ended"], where=ends, out=np.zeros_like(ref["ended"])).max()
    assert (np.abs(got[3][ends] - ref["ended"][ends]) <= 2.0 ** -24 * top + tol).all()


def reorder(parents, tables, lens, ring, state, bs, shared=None):
    """numpy arrays; returns (tables, lens, ring, state, pairs, flags) as lists of lists, flags
    a set of names."""
    B, W = parents.shape
    M, NB = tables.shape[1], len(ring)
    rows = tables.reshape(B, W, M).tolist()
    L = lens.reshape(B, W).tolist()
    P = parents.tolist()
    sh = [0] * B if shared is None else list(map(int, shared))
    ring0, ring = list(map(int, ring)), list(map(int, ring))
    head, tail = int(state[0]), int(state[1])
    flags = set()
    same = (tables.tolist(), lens.tolist(), ring0, [head, tail], [[0, 0]] * (B * W))

    def blocks(n):
        return -(-n // bs)

    bad = []
    for b in range(B):
        off = False
        for w in range(W):
            if not -1 <= P[b][w] < W:
                flags.add("beam")
                off = True
            if L[b][w] < 0 or blocks(L[b][w]) > M:
                flags.add("context")
                off = True
        if sh[b] < 0:
            flags.add("context")
            off = True
        bad.append(off)
    new_rows, new_lens, pairs, wants = [], [], [], []
    for b in range(B):
        if bad[b]:
            new_rows.append([list(r) for r in rows[b]])
            new_lens.append(list(L[b]))
            pairs.append([[0, 0] for _ in range(W)])
            continue
        seen, out, ol, op = set(), [], [], []
        for w in range(W):
            p = P[b][w]
            n = L[b][p] if p >= 0 else 0
            k = blocks(n)
            r = (rows[b][p][:k] if p >= 0 else []) + [-1] * (M - k)
            op.append([0, 0])
            if n % bs:
                t = r[k - 1]
                if not 0 <= t < NB:
                    flags.add("id")
                elif (k - 1, t) in seen:
                    wants.append((b, w, k - 1, t))
                else:
                    seen.add((k - 1, t))
            out.append(r)
            ol.append(n)
        new_rows.append(out)
        new_lens.append(ol)
        pairs.append(op)
    if not (head >= 0 and head <= tail <= head + NB) or len(wants) > tail - head:
        return same + (flags | {"blocks"},)
    moved = [[list(r) for r in q] for q in new_rows]
    for i, (b, w, col, t) in enumerate(wants):
        new = ring0[(head + i) % NB]
        if 0 <= new < NB:
            new_rows[b][w][col], pairs[b][w] = new, [t, new]
        else:
            flags.add("id")
            new_rows[b][w][col] = -1
    put = 0
    for b in range(B):
        if bad[b]:
            continue
        for col in range(sh[b] // bs, M):
            keep = {moved[b][w][col] for w in range(W) if col < blocks(new_lens[b][w])}
            for w in range(W):
                if col >= blocks(L[b][w]) or rows[b][w][col] in keep:
                    continue
                x = rows[b][w][col]
                keep.add(x)
                if not 0 <= x < NB:
                    flags.add("id")
                    continue
                if tail - head + put < NB:
                    ring[(tail + put) % NB] = x
                    put += 1
                else:
                    flags.add("id")
    return ([r for q in new_rows for r in q], [n for q in new_lens for n in q], ring,
            [head + len(wants), tail + put], [p for q in pairs for p in q], flags)


def backtrack(tokens, parents, lengths, beams, pad=0):
    S, B, W = tokens.shape
    K = lengths.shape[1]
    out = np.full((B, K, S), pad, np.int64)
    bad = False
    for b in range(B):
        for k in range(K):
            n, w = int(lengths[b, k]), int(beams[b, k])
            if not 0 <= n <= S or (n > 0 and not 0 <= w < W):
                bad = True
                continue
            for s in range(n - 1, -1, -1):
                out[b, k, s] = tokens[s, b, w]
                w = int(parents[s, b, w])
                if s > 0 and not 0 <= w < W:
                    bad = True
                    break
    return out, bad
