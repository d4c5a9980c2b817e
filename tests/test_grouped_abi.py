"""Argument validation of the grouped-head calls, without a GPU: every refusal
returns before anything is launched, and a call with nothing to do launches
nothing."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from paged_kv_cache_172_gb300 import build_lib

P = 0x1000  # any 32-byte aligned address: these calls return before touching memory


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pk.lib()


def plan(lib, **kw):
    a = dict(c=P, n=P, B=4, bs=16, nb=64, mb=8, T=32, ring=P, state=P, bt=P, ctx=P, off=P, slot=P,
             pos=P, out=P)
    a.update(kw)
    return lib.pa_step_plan(a["c"], a["n"], a["B"], a["bs"], a["nb"], a["mb"], a["T"], a["ring"],
                            a["state"], a["bt"], a["ctx"], a["off"], a["slot"], a["pos"],
                            a["out"], None, None)


def test_step_plan_refusals(lib):
    for kw in (dict(B=-1), dict(T=-1), dict(nb=0), dict(mb=0), dict(mb=2 ** 27), dict(c=None),
               dict(n=None), dict(ring=None), dict(state=None), dict(bt=None), dict(ctx=None),
               dict(off=None), dict(slot=None), dict(pos=None), dict(out=None)):
        assert plan(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(bs=12), dict(bs=64), dict(B=16385)):
        assert plan(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw


def rope(lib, **kw):
    a = dict(q=P, k=P, v=P, pos=P, table=P, slot=P, T=4, H=8, Hkv=2, D=128, R=128, axes=1, il=0,
             dt=0, qs=1024, ks=256, vs=256, bs=16, nb=8, qo=P + 64, qos=1024, ko=P + 32, kos=256,
             kc=P, vc=P)
    a.update(kw)
    return lib.pa_rope_cache_write(
        a["q"], a["k"], a["v"], a["pos"], a["table"], a["slot"], a["T"], a["H"], a["Hkv"], a["D"],
        a["R"], a["axes"], a["il"], a["dt"], a["qs"], a["ks"], a["vs"], a["bs"], a["nb"], a["qo"],
        a["qos"], a["ko"], a["kos"], a["kc"], a["vc"], None, None)


def test_rope_refusals(lib):
    for kw in (dict(T=-1), dict(H=0), dict(Hkv=0), dict(H=9), dict(H=65536, Hkv=65536),
               dict(axes=0), dict(axes=5), dict(dt=2), dict(dt=-1), dict(q=None), dict(q=P + 8),
               dict(qs=1020), dict(qs=1016), dict(ks=248), dict(vs=8), dict(pos=None),
               dict(table=None), dict(qo=None), dict(qo=P + 8), dict(qos=1000),
               dict(kc=None), dict(vc=None), dict(slot=None), dict(v=None), dict(nb=0),
               dict(nb=2 ** 27), dict(ko=None, kc=None, vc=None), dict(kos=8),
               dict(qo=P, qos=2048), dict(ko=P, kos=512)):
        assert rope(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(D=96), dict(D=256), dict(R=8), dict(R=136), dict(R=0), dict(R=100),
               dict(bs=12)):
        assert rope(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    assert rope(lib, T=0) == pk.PA_OK


def test_rope_table(lib):
    inv = np.array([1.0, 0.25, 3e-5, 2 * math.pi, -0.5, 1e9 + 0.5, 0.0])
    axes = [0, 1, 2, 3, 0, 1, 2]
    t = pk.pa_rope_table(inv, axes).numpy().view(np.uint64)
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    for f, a, x in zip(inv, axes, t):
        assert int(x) & 3 == a
        turns = Decimal(float(f)) / two_pi
        turns -= turns.to_integral_value(rounding="ROUND_FLOOR")
        off = abs(int(x) - int(x) % 4 - int(turns * 2 ** 64)) % 2 ** 64
        # 2^-62 for the two low bits, and the second double's rounding, 2^-105 of the turns
        assert min(off, 2 ** 64 - off) <= 8 + 2 ** 64 * 2.0 ** -100 * max(1.0, abs(f)), (f, off)
    for bad in ([math.inf], [math.nan], [2.0 ** 50]):
        with pytest.raises(pk.PagedKVError):
            pk.pa_rope_table(bad)
    for bad in ([4], [-1]):
        with pytest.raises(pk.PagedKVError):
            pk.pa_rope_table([1.0], bad)
    with pytest.raises(ValueError):
        pk.pa_rope_table([1.0, 2.0], [0])
    assert lib.pa_rope_table(None, None, 0, None) == pk.PA_OK
    assert lib.pa_rope_table(None, None, 1, None) == pk.PA_ERR_INVALID


def prompt(lib, **kw):
    a = dict(q=P, k=P, v=P, off=P, B=2, T=8, H=8, Hkv=2, D=128, dt=1, qs=1024, ks=256, vs=256,
             scale=0.1, out=P)
    a.update(kw)
    return lib.pa_prompt_attention(a["q"], a["k"], a["v"], a["off"], a["B"], a["T"], a["H"],
                                   a["Hkv"], a["D"], a["dt"], a["qs"], a["ks"], a["vs"],
                                   a["scale"], a["out"], None, None)


def chunk(lib, **kw):
    a = dict(q=P, k=P, v=P, bt=P, ctx=P, off=P, B=2, T=8, H=8, Hkv=2, D=128, dt=1, qs=1024,
             bs=16, nb=8, mb=4, cap=64, scale=0.1, out=P, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_chunk_attention(a["q"], a["k"], a["v"], a["bt"], a["ctx"], a["off"], a["B"],
                                  a["T"], a["H"], a["Hkv"], a["D"], a["dt"], a["qs"], a["bs"],
                                  a["nb"], a["mb"], a["cap"], a["scale"], a["out"], a["ws"],
                                  a["wsb"], None, None)


def decode(lib, **kw):
    a = dict(q=P, k=P, v=P, bt=P, ctx=P, B=2, H=8, Hkv=2, D=128, dt=1, bs=16, nb=8, mb=4, cap=64,
             pt=0, scale=0.1, out=P, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_decode_grouped(a["q"], a["k"], a["v"], a["bt"], a["ctx"], a["B"], a["H"],
                                 a["Hkv"], a["D"], a["dt"], a["bs"], a["nb"], a["mb"], a["cap"],
                                 a["pt"], a["scale"], a["out"], a["ws"], a["wsb"], None, None)


COMMON = (dict(B=-1), dict(H=7), dict(Hkv=0), dict(H=0), dict(dt=7), dict(q=None), dict(k=None),
          dict(v=None), dict(out=None), dict(q=P + 8), dict(out=P + 8), dict(k=P + 4),
          dict(scale=math.nan), dict(scale=math.inf))
PACKED = (dict(T=-1), dict(off=None), dict(qs=1000), dict(qs=1020), dict(scale=0.0),
          dict(scale=-1.0))
CACHED = (dict(bt=None), dict(ctx=None), dict(nb=0), dict(nb=2 ** 27), dict(mb=0), dict(cap=65),
          dict(cap=-1))


def test_prompt_refusals(lib):
    for kw in COMMON + PACKED + (dict(ks=100), dict(vs=64)):
        assert prompt(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(D=80), dict(H=129, Hkv=1, qs=129 * 128)):
        assert prompt(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    assert prompt(lib, B=0) == pk.PA_OK and prompt(lib, T=0) == pk.PA_OK


def test_chunk_refusals(lib):
    for kw in COMMON + PACKED + CACHED + (dict(ws=P + 8, wsb=2 ** 30),):
        assert chunk(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(D=80), dict(bs=4), dict(bs=64, cap=8), dict(H=258, qs=258 * 128)):
        assert chunk(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    assert chunk(lib, B=0) == pk.PA_OK and chunk(lib, T=0) == pk.PA_OK


def test_decode_refusals(lib):
    for kw in COMMON + CACHED + (dict(B=65536), dict(pt=-64), dict(pt=100), dict(pt=2112)):
        assert decode(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(D=80), dict(bs=4), dict(bs=64, cap=8)):
        assert decode(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    big = dict(mb=1000, cap=16000, pt=64)
    assert decode(lib, **big) == pk.PA_ERR_WORKSPACE
    assert decode(lib, ws=P, wsb=64, **big) == pk.PA_ERR_WORKSPACE
    need = pk.pa_decode_grouped_workspace_size(2, 8, 2, 128, 16, 16000, 64)
    assert need == 2 * 8 * 250 * 130 * 4
    assert decode(lib, ws=P + 8, wsb=need, **big) == pk.PA_ERR_INVALID
    assert decode(lib, B=0) == pk.PA_OK


def test_sizes_of_nothing_are_zero(lib):
    assert pk.pa_decode_grouped_workspace_size(0, 8, 2, 128, 16, 100) == 0
    assert pk.pa_decode_grouped_workspace_size(2, 8, 3, 128, 16, 100) == 0
    assert pk.pa_decode_grouped_workspace_size(2, 8, 2, 128, 16, 64) == 0  # one partition
    assert pk.pa_chunk_attention_workspace_size(0, 8, 8, 2, 128, 100) == 0
    assert pk.pa_chunk_attention_workspace_size(2, 0, 8, 2, 128, 100) == 0


def test_bindings_reject_cpu_tensors_and_wrong_types():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    i32 = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(2, 16, 4, 64, dtype=torch.float16)
    for call in (lambda: pk.pa_prompt_attention(q, q, q, i32, 0.1),
                 lambda: pk.pa_decode_grouped(q, cache, cache, i32.view(1, 4).repeat(3, 1),
                                              i32[:3], 0.1, 16),
                 lambda: pk.pa_chunk_attention(q, cache, cache, i32.view(1, 4).repeat(3, 1),
                                               i32[:3], i32, 0.1),
                 lambda: pk.pa_rope_cache_write(q, q, q, i32[:3], torch.zeros(32).long(),
                                                i32[:3].long()),
                 lambda: pk.pa_step_plan(i32, i32, i32.view(4, 1), i32, i32[:2].long(), 16, 8)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        pk.pa_prompt_attention(q.float(), q, q, i32, 0.1)
    with pytest.raises(TypeError):
        pk.pa_prompt_attention(None, q, q, i32, 0.1)
    with pytest.raises(ValueError):
        pk.pa_prompt_attention(q[0], q, q, i32, 0.1)


def test_counts_that_32_bits_cannot_step_past_are_refused(lib):
    for T in (2 ** 31 - 32768, 2 ** 31 - 1):
        assert plan(lib, T=T) == pk.PA_ERR_INVALID
        assert chunk(lib, mb=2 ** 27, cap=T) == pk.PA_ERR_INVALID
        assert decode(lib, mb=2 ** 27, cap=T) == pk.PA_ERR_INVALID
