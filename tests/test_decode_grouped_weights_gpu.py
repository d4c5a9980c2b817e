"""Precision of pa_decode_grouped's softmax weights.

Queries in {-1, 0, 1} and keys that are multiples of 1/4 make every score exact in
fp32, and at most 128 keys keep the sums short, so that little but the weights and the
result's rounding is left.  Per element, with A = sum_j p_j |v_j| / sum_j p_j:
  u |o|            the result's rounding, u = 2^-8 bf16, 2^-11 fp16;
  2^-15 A, 2^-21 A (bf16, fp16)  a weight enters its product as two 16-bit values,
                   the first cut off (below 2^-7, 2^-10 of it) and the rest rounded
                   (2^-8, 2^-11 of that);
  n 2^-22 A        fp32 sums over n weights and values (2^-23 a step each);
  2^-21 s A        exponents: products, scale and differences of magnitude s =
                   max |score log2 e|, each rounded once to fp32;
  2^-19 A          exponentials and rescalings (2^-21 each, most cancel);
  2^-24            fp16 only: subnormal results.
Weights of one 16-bit value are off by u A: far outside where |o| is below A.
"""
import math

import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import Paged, check
from pk_testutil import zero_status

DEV = torch.device("cuda:0")
CTX = [2, 5, 16, 17, 33, 64, 65, 100, 128]


def exact_scores(q, keys, seed):
    """Fills q and the list of keys with values whose products sum without rounding."""
    g = torch.Generator(device=q.device).manual_seed(seed)
    q.copy_(torch.randint(-1, 2, q.shape, generator=g, device=q.device))
    for k in keys:
        k.copy_(torch.randint(-4, 5, k.shape, generator=g, device=q.device) / 4)


def attend_exactly(q, k, v, scale, dtype):
    """Single query q [H, D] over k, v [n, Hkv, D]: (result, bound), in 64 bits."""
    H, D = q.shape
    n, Hkv = k.shape[:2]
    s = torch.einsum("gid,ngd->gin", q.double().view(Hkv, H // Hkv, D), k.double()) * scale
    p = torch.softmax(s, -1)
    o = torch.einsum("gin,ngd->gid", p, v.double()).reshape(H, D)
    A = torch.einsum("gin,ngd->gid", p, v.double().abs()).reshape(H, D)
    fp16 = dtype == torch.float16
    s2 = s.abs().max().item() * math.log2(math.e)
    w = 2.0 ** -21 if fp16 else 2.0 ** -15
    tol = torch.finfo(dtype).eps / 2 * o.abs() + (w + n * 2.0 ** -22 + s2 * 2.0 ** -21
                                                  + 2.0 ** -19) * A
    return o, tol + (2.0 ** -24 if fp16 else 0.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_bound_tells_rounded_weights(dtype):
    # one rounding of the weights alone, everything else exact, is past the bound
    g = torch.Generator().manual_seed(1)
    H, Hkv, D, n = 8, 2, 64, 33
    q, k = torch.empty(H, D), torch.empty(n, Hkv, D)
    exact_scores(q, [k], 2)
    v = torch.randn(n, Hkv, D, generator=g).to(dtype)
    o, tol = attend_exactly(q, k, v, D ** -0.5, dtype)
    s = torch.einsum("gid,ngd->gin", q.double().view(Hkv, H // Hkv, D), k.double()) * D ** -0.5
    p = torch.exp(s - s.amax(-1, keepdim=True))
    for weights, fits in ((p, True), (p.to(dtype).double(), False)):
        got = torch.einsum("gin,ngd->gid", weights, v.double()) / p.sum(-1, keepdim=True)
        err = (got.reshape(H, D).to(dtype).double() - o).abs()
        assert bool((err <= tol).all()) == fits


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (3, 3), (24, 2), (40, 1)])
def test_weights_keep_more_than_the_caches_type(dtype, D, H, Hkv):
    import __graft_entry__
    __graft_entry__.build()
    p = Paged(CTX, [1] * len(CTX), H, Hkv, D, 16, dtype, seed=H + D)
    exact_scores(p.q, p.keys, D)
    for b in range(len(CTX)):
        p.store(b)
    for pt in (0, 64, 128):
        status = zero_status(DEV)
        out = torch.full_like(p.q, float("nan"))
        pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale, max(CTX),
                             out=out, partition_tokens=pt, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for b in range(len(CTX)):
            o, tol = attend_exactly(p.q[b], p.keys[b], p.values[b], p.scale, dtype)
            check(out[b], o, tol, f"partition {pt} context {CTX[b]}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_infinite_value_shows_in_its_dim_alone(dtype):
    p = Paged([100, 100], [1, 1], 8, 2, 64, 16, dtype, seed=3)
    exact_scores(p.q, p.keys, 4)
    p.values[0][37, :, 9] = float("inf")
    p.values[0][80, :, 11] = -float("inf")
    for b in range(2):
        p.store(b)
    for pt in (0, 64):
        out = pk.pa_decode_grouped(p.q, p.k_cache, p.v_cache, p.tables, p.context, p.scale, 100,
                                   partition_tokens=pt)
        assert (out[0, :, 9] == float("inf")).all() and (out[0, :, 11] == -float("inf")).all()
        for b in range(2):
            v = p.values[b].clone()
            v[torch.isinf(v)] = 0
            o, tol = attend_exactly(p.q[b], p.keys[b], v, p.scale, dtype)
            got = torch.where(torch.isinf(out[b]), o.to(dtype), out[b])
            check(got, o, tol, f"partition {pt} sequence {b}")
