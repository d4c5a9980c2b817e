"""Reference and error bound of the grouped attention tests, in 64 bits.

Per element, with A = sum_j p_j |v_j| / sum_j p_j and u = eps / 2 of the 16-bit
type (2^-8 bf16, 2^-11 fp16):
  u A     the weights p_j, each rounded once to that type;
  u |o|   the result's rounding;
  2 d A   the scores: fp32 sums of D products, each partial sum off by at most
          2^-23 of the magnitudes it holds, so d <= D 2^-23 S in nats with S =
          max_j scale sum |q k_j|; a weight's relative error is d, and the
          quotient doubles it;
  n 2^-22 A + 2^-19 A   fp32 sums over n weights and values in whatever order
          (2^-23 a step each), and the exponentials and rescalings (2^-21 each
          where they do not cancel, few dozens of them);
  2^-24 sum |v_j|   fp16 only: weights below 2^-14 of the row's maximum are
          subnormal, off by 2^-25 of at most its double, and the sum of
          weights is at least one;
  2^-24   fp16 only: subnormal results.
"""
import numpy as np
import torch


def attend(q, k, v, scale, first):
    """q [L, H, D], k and v [N, Hkv, D] on any device, query i sees keys 0 ..
    first + i.  (result, bound) in 64 bits, bound for q's type."""
    L, H, D = q.shape
    N, Hkv = k.shape[0], k.shape[1]
    if L == 0 or N == 0:
        z = torch.zeros(L, H, D, dtype=torch.float64, device=q.device)
        return z, z
    u = torch.finfo(q.dtype).eps / 2
    fp16 = q.dtype == torch.float16
    qd = q.double().reshape(L, Hkv, H // Hkv, D)
    kd, vd = k.double(), v.double()
    s = torch.einsum("lgid,ngd->giln", qd, kd) * scale
    mag = torch.einsum("lgid,ngd->giln", qd.abs(), kd.abs()) * abs(scale)
    i = torch.arange(L, device=q.device)[:, None]
    seen = torch.arange(N, device=q.device)[None] <= i + first
    s = s.masked_fill(~seen, -float("inf"))
    mag = mag.masked_fill(~seen, 0.0)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.einsum("giln,ngd->lgid", p, vd)
    A = torch.einsum("giln,ngd->lgid", p, vd.abs())
    d = D * 2.0 ** -23 * mag.amax(-1).permute(2, 0, 1)[..., None]
    n = seen.sum(-1).double()[:, None, None, None]
    tol = u * (A + out.abs()) + (2 * d + n * 2.0 ** -22 + 2.0 ** -19) * A
    if fp16:
        tol = tol + 2.0 ** -24 * torch.einsum("ln,ngd->lgd", seen.double(), vd.abs())[:, :, None]
        tol = tol + 2.0 ** -24
    return out.reshape(L, H, D), tol.reshape(L, H, D)


def check(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    over = (err - tol).max().item() if err.numel() else 0.0
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert over <= 0, f"{what}: {over:.3e} past the bound, max error {err.max().item():.3e}"


class Packed:
    """Random packed prompts; fused: q, k, v are views of one array."""

    def __init__(self, lens, H, Hkv, D, dtype, seed=0, fused=False, before=0, behind=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.lens = list(lens)
        T = before + sum(lens) + behind
        qkv = torch.randn(T, H + 2 * Hkv, D, generator=g, device=device).to(dtype)
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.start = before + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.offsets = torch.tensor(self.start, dtype=torch.int32, device=device)
        self.scale = D ** -0.5

    def rows(self, b):
        return slice(int(self.start[b]), int(self.start[b + 1]))


class Paged:
    """Random caches with shuffled blocks; NaN in every slot no sequence holds."""

    def __init__(self, ctx, qlens, H, Hkv, D, bs, dtype, seed=0, device="cuda:0", before=0,
                 behind=0, spare=2):
        g = torch.Generator(device=device).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.qlens = list(ctx), list(qlens)
        need = [-(-c // bs) for c in ctx]
        NB, M = sum(need) + spare, max(need) + 1
        ids = rng.permutation(NB)
        self.tables_h = np.full((len(ctx), M), -1, np.int32)
        shape = (NB, bs, Hkv, D)
        self.k_cache = torch.full(shape, float("nan"), dtype=dtype, device=device)
        self.v_cache = torch.full(shape, float("nan"), dtype=dtype, device=device)
        self.keys, self.values = [], []
        at = 0
        for b, c in enumerate(ctx):
            blocks = ids[at:at + need[b]]
            at += need[b]
            self.tables_h[b, :need[b]] = blocks
            kv = torch.randn(2, c, Hkv, D, generator=g, device=device).to(dtype)
            self.keys.append(kv[0])
            self.values.append(kv[1])
            self.store(b)
        self.tables = torch.tensor(self.tables_h, device=device)
        self.context = torch.tensor(self.ctx, dtype=torch.int32, device=device)
        T = before + sum(qlens) + behind
        self.q = torch.randn(T, H, D, generator=g, device=device).to(dtype)
        self.start = before + np.concatenate([[0], np.cumsum(qlens)]).astype(np.int64)
        self.offsets = torch.tensor(self.start, dtype=torch.int32, device=device)
        self.scale = D ** -0.5
        self.bs = bs

    def store(self, b):
        """(Re)writes sequence b's keys and values to the cache."""
        bs = self.k_cache.shape[1]
        j = np.arange(self.ctx[b])
        slot = torch.as_tensor(self.tables_h[b, j // bs].astype(np.int64) * bs + j % bs,
                               device=self.k_cache.device)
        self.k_cache.flatten(0, 1)[slot] = self.keys[b]
        self.v_cache.flatten(0, 1)[slot] = self.values[b]

    def rows(self, b):
        return slice(int(self.start[b]), int(self.start[b + 1]))

    def ref(self, b):
        return attend(self.q[self.rows(b)], self.keys[b], self.values[b], self.scale,
                      self.ctx[b] - self.qlens[b])
