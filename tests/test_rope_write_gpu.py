"""pa_rope_cache_write against rotations computed in 64 bits on the host.

Error bound of an element with pair (x, y): half a unit of the output type,
eps / 2 relative to the result (2^-8 for bf16, 2^-11 for fp16), and from the
arithmetic before that rounding: the angle is off by 2^-26 of a turn (9.4e-8),
sine and cosine by 2 units of fp32 (2.4e-7), two products and a sum by 2^-24
each of at most |x| + |y| (1.8e-7); together below 6e-7 (|x| + |y|).  fp16 results
below its smallest normal add 2^-25.
"""
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


def rotated(x, pos, inv, axis, R, interleaved):
    """(result, |x| + |y| of each element's pair), x [T, heads, D], in 64 bits."""
    x = x.double().cpu().numpy()
    angle = pos.astype(np.float64).reshape(-1, x.shape[0])[axis].T * inv  # [T, R / 2]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    out, mag = x.copy(), np.zeros_like(x)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2),
                                                                  slice(R // 2, R))
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, mag


def close(got, want):
    ref, mag = want
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(ref) + 6e-7 * mag + tiny
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())


def make(T, H, Hkv, D, R, n_axes, dtype, bs=16, fused=False, far=4096, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = torch.randn(T, H + 2 * Hkv, D, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    NB = T // bs + 2
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    if T > 2:
        slots[1] = -1
    inv = 10000.0 ** (-np.arange(R // 2) * 2.0 / R)
    axis = rng.integers(0, n_axes, R // 2)
    pos = rng.integers(-far, far, (n_axes, T))
    cache = torch.full((NB, bs, Hkv, D), 3.0, dtype=dtype, device=DEV)
    return dict(q=q, k=k, v=v, pos=pos, inv=inv, axis=axis, slots=slots, k_cache=cache,
                v_cache=cache.clone(), R=R)


def call(m, interleaved=False, **kw):
    status = zero_status(DEV)
    q, k = pk.pa_rope_cache_write(
        m["q"], m["k"], m["v"], torch.from_numpy(m["pos"].astype(np.int32)).to(DEV),
        pk.pa_rope_table(m["inv"], m["axis"], device=DEV),
        torch.from_numpy(m["slots"]).to(DEV), m["k_cache"], m["v_cache"],
        interleaved=interleaved, status=status, **kw)
    torch.cuda.synchronize()
    return q, k, int(status.item())


def check_cache(m, k_want, v):
    """Written slots hold the rotated keys and the values' bits; the others are untouched."""
    keep = m["slots"] >= 0
    at = torch.from_numpy(m["slots"][keep]).to(DEV)
    kc, vc = m["k_cache"].flatten(0, 1), m["v_cache"].flatten(0, 1)
    close(kc[at], (k_want[0][keep], k_want[1][keep]))
    assert torch.equal(vc[at], v[torch.from_numpy(keep).to(DEV)])
    rest = torch.ones(kc.shape[0], dtype=torch.bool, device=DEV)
    rest[at] = False
    assert (kc[rest] == 3).all() and (vc[rest] == 3).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hkv,D,R,n_axes,bs,fused", [
    (1, 8, 8, 64, 64, 1, 4, False), (3, 5, 1, 128, 128, 3, 16, True),
    (38, 40, 8, 128, 64, 2, 16, True), (17, 12, 4, 64, 16, 4, 8, False),
    (700, 28, 4, 128, 112, 3, 32, True), (401, 2, 2, 64, 48, 1, 16, False),
])
def test_rotation_and_write(dtype, interleaved, T, H, Hkv, D, R, n_axes, bs, fused):
    m = make(T, H, Hkv, D, R, n_axes, dtype, bs=bs, fused=fused, seed=T)
    want_q = rotated(m["q"], m["pos"], m["inv"], m["axis"], R, interleaved)
    want_k = rotated(m["k"], m["pos"], m["inv"], m["axis"], R, interleaved)
    v = m["v"].clone()
    k_out = torch.empty(T, Hkv, D, dtype=dtype, device=DEV)
    q, k, st = call(m, interleaved, k_out=k_out)
    assert st == 0 and k is k_out
    close(q, want_q)
    close(k, want_k)
    check_cache(m, want_k, v)


@pytest.mark.parametrize("fused", [False, True])
def test_in_place(fused):
    m = make(90, 6, 2, 128, 128, 3, torch.bfloat16, fused=fused, seed=4)
    want_q = rotated(m["q"], m["pos"], m["inv"], m["axis"], 128, False)
    want_k = rotated(m["k"], m["pos"], m["inv"], m["axis"], 128, False)
    v = m["v"].clone()
    q, k, st = call(m, q_out=m["q"], k_out=m["k"])
    assert st == 0
    close(q, want_q)
    close(k, want_k)
    assert torch.equal(m["v"], v)
    check_cache(m, want_k, v)


def test_rotation_without_a_cache():
    m = make(50, 4, 4, 64, 64, 2, torch.float16, seed=6)
    q, k = pk.pa_rope_cache_write(m["q"], m["k"], None,
                                  torch.from_numpy(m["pos"].astype(np.int32)).to(DEV),
                                  pk.pa_rope_table(m["inv"], m["axis"], device=DEV), None)
    close(q, rotated(m["q"], m["pos"], m["inv"], m["axis"], 64, False))
    close(k, rotated(m["k"], m["pos"], m["inv"], m["axis"], 64, False))


def test_far_positions_are_exact():
    # angles of positions up to 2^31 - 1: the reference reduces them with whole
    # numbers, frac(position * F / 2^120) for F = round(inv / 2 pi * 2^120)
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230782")
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6 + 1, 123456789, -987654321])
    m = make(len(pos), 2, 1, 128, 128, 1, torch.float16, seed=8)
    m["pos"] = pos[None]
    frac = np.zeros((len(pos), 64))
    for i, f in enumerate(m["inv"]):
        F = int((Decimal(float(f)) / two_pi * 2 ** 120).to_integral_value())
        for t, p in enumerate(pos):
            frac[t, i] = float(Decimal((int(p) * F) % 2 ** 120) / 2 ** 120)
    angle = frac * 2 * np.pi
    x = m["q"].double().cpu().numpy()
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = x[..., :64], x[..., 64:]
    ref = np.concatenate([a * c - b * s, b * c + a * s], -1)
    mag = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    q, _, st = call(m)
    assert st == 0
    close(q, (ref, mag))


def test_bad_slots_are_flagged_and_skipped():
    m = make(5, 2, 1, 64, 64, 1, torch.float16, seed=10)
    n = m["k_cache"].shape[0] * 16
    m["slots"] = np.array([0, n, n + 5, 2 ** 40, n - 1])
    want_k = rotated(m["k"], m["pos"], m["inv"], m["axis"], 64, False)
    q, _, st = call(m)
    assert st == pk.PA_DEV_BAD_SLOT
    close(q, rotated(m["q"], m["pos"], m["inv"], m["axis"], 64, False))  # still rotated
    m["slots"] = np.array([0, -1, -1, -1, n - 1])
    check_cache(m, want_k, m["v"])


def test_empty_and_refusals():
    m = make(0, 4, 2, 64, 64, 1, torch.float16)
    q, k, st = call(m)
    assert st == 0 and q.shape == (0, 4, 64)
    m = make(4, 4, 2, 64, 64, 1, torch.float16)
    with pytest.raises(TypeError):
        call(dict(m, k=m["k"].bfloat16()))
    with pytest.raises(TypeError):
        call(dict(m, q=m["q"].float()))
    with pytest.raises(ValueError):
        call(dict(m, q=m["q"].transpose(0, 1)))
    with pytest.raises(ValueError):
        call(dict(m, v=m["v"][:, :1]))
    with pytest.raises(pk.PagedKVError):  # a token stride that is not 16-byte aligned
        wide = torch.zeros(4, 4 * 64 + 4, dtype=torch.float16, device=DEV)
        call(dict(m, q=wide[:, :256].unflatten(1, (4, 64))))
    with pytest.raises(pk.PagedKVError):  # rotary_dim past the head
        call(dict(m, inv=np.ones(40), axis=np.zeros(40, np.int64)))
    with pytest.raises(pk.PagedKVError):  # 3 query heads on 2 K/V heads
        call(dict(m, q=m["q"][:, :3].contiguous()))
