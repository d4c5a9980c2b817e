"""Argument validation of the beam and cross-attention calls, without a GPU: every refusal
returns before anything is launched, and a call with nothing to do launches nothing."""
import pytest

import paged_kv_cache_172_gb300 as pk
from paged_kv_cache_172_gb300 import build_lib

P = 0x1000  # any 32-byte aligned address: these calls return before touching memory


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pk.lib()


def cross(lib, **kw):
    a = dict(q=P, k=P, v=P, off=P, st=P, ln=P, B=2, T=64, Tk=99, H=8, Hkv=2, D=128, dt=1, qs=1024,
             ks=256, vs=256, mq=32, mk=50, scale=0.1, out=P, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_cross_attention(a["q"], a["k"], a["v"], a["off"], a["st"], a["ln"], a["B"],
                                  a["T"], a["Tk"], a["H"], a["Hkv"], a["D"], a["dt"], a["qs"],
                                  a["ks"], a["vs"], a["mq"], a["mk"], a["scale"], a["out"],
                                  a["ws"], a["wsb"], None, None)


def test_cross_refusals(lib):
    for kw in (dict(B=-1), dict(T=-1), dict(T=2 ** 31 - 32767), dict(Tk=-1), dict(Tk=2 ** 31 - 1),
               dict(H=0), dict(Hkv=3), dict(dt=2), dict(dt=-1), dict(mq=-1), dict(mk=-1),
               dict(mk=2 ** 31 - 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(q=None), dict(q=P + 8), dict(qs=1016), dict(k=None), dict(v=None),
               dict(ks=248), dict(vs=257), dict(off=None), dict(st=None), dict(ln=None),
               dict(out=None), dict(out=P + 2), dict(ws=P + 8, wsb=2 ** 40)):
        assert cross(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(D=96), dict(D=256), dict(H=258, Hkv=2, qs=258 * 128)):
        assert cross(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    for kw in (dict(B=0), dict(T=0)):
        assert cross(lib, **kw) == pk.PA_OK, kw
    long = dict(T=2, H=8, Hkv=8, qs=1024, ks=1024, vs=1024, mq=1, mk=10 ** 6, Tk=10 ** 6)
    need = lib.pa_cross_attention_workspace_size(2, 2, 8, 8, 128, 1, 10 ** 6)
    assert need > 0
    assert cross(lib, ws=P, wsb=need - 1, **long) == pk.PA_ERR_WORKSPACE


def test_cross_workspace_size(lib):
    size = lib.pa_cross_attention_workspace_size
    for a in ((0, 2, 8, 8, 128, 1, 100), (2, 0, 8, 8, 128, 1, 100), (2, 2, 8, 3, 128, 1, 100),
              (2, 2, 8, 8, 96, 1, 100), (2, 2, 8, 8, 128, 0, 100), (2, 2, 8, 8, 128, 1, 0),
              (2, 2, 8, 8, 128, 1, 2 ** 31 - 1), (2, 2, 1024, 1, 128, 2, 10 ** 6)):
        assert size(*a) == 0, a
    # more queries than there are count as those there are
    assert size(1, 2, 8, 8, 128, 2, 10 ** 6) == size(1, 2, 8, 8, 128, 99, 10 ** 6) > 0


def select(lib, **kw):
    a = dict(x=P, dt=2, stride=100, s=P, B=2, W=4, V=100, eos=5, pad=0, t=P, p=P, n=P, e=P, ws=P,
             wsb=2 ** 40)
    a.update(kw)
    return lib.pa_beam_select(a["x"], a["dt"], a["stride"], a["s"], a["B"], a["W"], a["V"],
                              a["eos"], a["pad"], a["t"], a["p"], a["n"], a["e"], a["ws"],
                              a["wsb"], None, None)


def test_select_refusals(lib):
    for kw in (dict(x=None), dict(x=P + 2), dict(dt=1, x=P + 1), dict(dt=3), dict(dt=-1),
               dict(stride=99), dict(stride=2 ** 40), dict(s=None), dict(B=-1), dict(W=0),
               dict(B=2 ** 19, W=4), dict(V=0), dict(V=2 ** 28 + 1, stride=2 ** 31),
               dict(eos=100), dict(eos=-2), dict(t=None), dict(p=None), dict(n=None),
               dict(e=None)):
        assert select(lib, **kw) == pk.PA_ERR_INVALID, kw
    assert select(lib, W=33) == pk.PA_ERR_UNSUPPORTED
    assert lib.pa_beam_select_workspace_size(2, 4, 100) == 0
    need = lib.pa_beam_select_workspace_size(1, 16, 200000)
    wide = dict(B=1, W=16, V=200000, stride=200000)
    if need > 0:  # (on a GPU of many SMs, as without one)
        assert select(lib, ws=None, **wide) == pk.PA_ERR_WORKSPACE
        assert select(lib, wsb=need - 1, **wide) == pk.PA_ERR_WORKSPACE
        assert select(lib, ws=P + 8, **wide) == pk.PA_ERR_INVALID
    assert select(lib, B=0, x=None) == pk.PA_OK
    for a in ((0, 4, 100), (2, 33, 100), (2, 4, 0), (-1, 4, 100), (2 ** 20, 2, 100)):
        assert lib.pa_beam_select_workspace_size(*a) == 0, a


def reorder(lib, **kw):
    a = dict(p=P, bt=P, ctx=P, sh=None, B=2, W=4, bs=16, nb=64, mb=8, ring=P, st=P, to=P, co=P,
             so=P, pairs=P, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_beam_reorder(a["p"], a["bt"], a["ctx"], a["sh"], a["B"], a["W"], a["bs"],
                               a["nb"], a["mb"], a["ring"], a["st"], a["to"], a["co"], a["so"],
                               a["pairs"], a["ws"], a["wsb"], None, None)


def test_reorder_refusals(lib):
    for kw in (dict(p=None), dict(bt=None), dict(ctx=None), dict(B=-1), dict(W=0), dict(nb=0),
               dict(mb=0), dict(mb=2 ** 27), dict(mb=2 ** 31 - 1), dict(ring=None), dict(st=None),
               dict(to=None), dict(co=None), dict(so=None), dict(pairs=None),
               dict(B=2 ** 19, W=4)):
        assert reorder(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(bs=12), dict(bs=64), dict(W=33)):
        assert reorder(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    need = lib.pa_beam_reorder_workspace_size(2000, 4, 8)
    assert need > 0 and lib.pa_beam_reorder_workspace_size(2, 4, 8) == 0
    assert reorder(lib, B=2000) == pk.PA_ERR_WORKSPACE
    assert reorder(lib, B=2000, ws=P, wsb=need - 1) == pk.PA_ERR_WORKSPACE
    assert reorder(lib, B=2000, ws=P + 8, wsb=need) == pk.PA_ERR_INVALID


def back(lib, **kw):
    a = dict(t=P, p=P, n=P, w=P, S=10, B=2, W=4, K=4, pad=0, out=P)
    a.update(kw)
    return lib.pa_beam_backtrack(a["t"], a["p"], a["n"], a["w"], a["S"], a["B"], a["W"], a["K"],
                                 a["pad"], a["out"], None, None)


def test_backtrack_refusals(lib):
    for kw in (dict(t=None), dict(p=None), dict(n=None), dict(w=None), dict(out=None), dict(S=-1),
               dict(B=-1), dict(W=0), dict(K=-1), dict(S=2 ** 26)):
        assert back(lib, **kw) == pk.PA_ERR_INVALID, kw
    for kw in (dict(W=33), dict(K=33)):
        assert back(lib, **kw) == pk.PA_ERR_UNSUPPORTED, kw
    for kw in (dict(S=0), dict(B=0), dict(K=0)):
        assert back(lib, t=None, **kw) == pk.PA_OK, kw
