"""Cross attention against 64 bits: packed queries over rows of another array, both
kernels (few queries a request, and many), with a bound per element (grouped_ref)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import attend, check

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


class Cross:
    """Random queries and states; NaN in every row of the states that no request holds.
    layout: 'pool' (any order, gaps), 'fused' (views of one [Tk, 2 Hkv, D] array),
    'padded'."""

    def __init__(self, qlens, lens, H, Hkv, D, dtype, layout="pool", seed=0, before=0, behind=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.qlens, self.lens, self.G = list(qlens), list(lens), H // Hkv
        B = len(lens)
        if layout == "padded":
            top = max(lens)
            starts, rows = np.arange(B) * top, B * top
        else:
            room = np.array(lens) + rng.integers(0, 5, B)
            order = rng.permutation(B)
            starts = np.zeros(B, np.int64)
            starts[order] = np.cumsum(room[order]) - room[order]
            rows = int(room.sum()) + 3
        kv = torch.full((rows, 2 * Hkv, D), float("nan"), device=device).to(dtype)
        for s, n in zip(starts, lens):
            kv[s:s + n] = torch.randn(n, 2 * Hkv, D, generator=g, device=device).to(dtype)
        self.k, self.v = kv[:, :Hkv], kv[:, Hkv:]
        if layout != "fused":
            self.k, self.v = self.k.contiguous(), self.v.contiguous()
        T = before + sum(qlens) + behind
        self.q = torch.randn(T, H, D, generator=g, device=device).to(dtype)
        self.at = before + np.concatenate([[0], np.cumsum(qlens)]).astype(np.int64)
        self.starts_h = starts
        self.offsets = torch.tensor(self.at, dtype=torch.int32, device=device)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=device)
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.scale = D ** -0.5
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def run(self, max_q=True, max_kv=True, **kw):
        return pk.pa_cross_attention(
            self.q, self.k, self.v, self.offsets, self.starts, self.kv_lens, self.scale,
            max(self.qlens) if max_q is True else max_q,
            max(self.lens) if max_kv is True else max_kv, status=self.status, **kw)

    def check(self, out, what="", skip=()):
        for b, n in enumerate(self.lens):
            if b in skip:
                continue
            rows = slice(int(self.at[b]), int(self.at[b + 1]))
            s = int(self.starts_h[b])
            ref, tol = attend(self.q[rows], self.k[s:s + n], self.v[s:s + n], self.scale, n)
            check(out[rows], ref, tol, f"{what} request {b}: {self.qlens[b]} on {n}")
        if not skip:
            assert self.status.item() == 0


HEADS = [(4, 4, 64), (16, 16, 64), (8, 2, 128), (12, 3, 64), (40, 8, 128), (14, 2, 64),
         (16, 1, 128), (5, 5, 128)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_few_queries(H, Hkv, D, dtype):
    """Beams and single tokens, one request without states, states of 1 to 1,000 rows."""
    lens = [1, 15, 16, 17, 0, 63, 64, 65, 129, 1000, 300]
    for beams in (1, 4):
        for layout in ("pool", "fused", "padded"):
            c = Cross([beams] * len(lens), lens, H, Hkv, D, dtype, layout, seed=beams)
            c.check(c.run(), f"{beams} beams, {layout}")
            c.check(c.run(split=False), f"{beams} beams, {layout}, whole")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_many_queries(H, Hkv, D, dtype):
    qlens = [1, 130, 0, 64, 33, 257, 7, 128]
    lens = [300, 127, 50, 0, 1, 129, 640, 128]
    for layout in ("pool", "fused"):
        c = Cross(qlens, lens, H, Hkv, D, dtype, layout, seed=3)
        c.check(c.run(), layout)
        c.check(c.run(max_q=None, max_kv=None, split=False), f"{layout}, loose bounds, whole")


@pytest.mark.parametrize("qlens", [[3, 0, 1, 2, 4], [16, 5, 0, 9, 1], [17, 1, 2, 0, 0]])
def test_ragged_few(qlens):
    lens = [700, 40, 1, 2000, 90]
    for H, Hkv in ((4, 4), (8, 2), (8, 1)):
        c = Cross(qlens, lens, H, Hkv, 64, BF16, seed=sum(qlens))
        c.check(c.run(), f"{qlens} {H} on {Hkv}")


@pytest.mark.parametrize("B,qlen,n,H,Hkv,D", [(1, 1, 20000, 8, 8, 64), (2, 4, 30011, 8, 2, 128),
                                             (3, 16, 9000, 4, 4, 64), (40, 4, 3000, 16, 16, 64),
                                             (1, 40, 25000, 8, 8, 64), (2, 100, 17000, 8, 2, 128)])
def test_long_states(B, qlen, n, H, Hkv, D):
    """Keys split over CTAs and joined, in the launch (clusters) and by a second one."""
    c = Cross([qlen] * B, [n - 13 * b for b in range(B)], H, Hkv, D, BF16, seed=n)
    c.check(c.run())
    c.check(c.run(max_kv=None), "loose bound")


def test_encoder_self_attention():
    """An encoder's own rows: q, k, v views of one projection's output."""
    lens, H, Hkv, D = [200, 1, 513, 64], 8, 4, 64
    g = torch.Generator(device="cuda").manual_seed(7)
    T = sum(lens)
    qkv = torch.randn(T, H + 2 * Hkv, D, generator=g, device="cuda").to(FP16)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    at = np.concatenate([[0], np.cumsum(lens)])
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = pk.pa_cross_attention(q, k, v, off, off[:-1], n, 0.125, max(lens), max(lens))
    for b, m in enumerate(lens):
        r = slice(at[b], at[b + 1])
        check(out[r], *attend(q[r], k[r], v[r], 0.125, m), f"sequence {b}")


@pytest.mark.parametrize("qlen", [2, 70])
def test_shared_states(qlen):
    """Three requests over the same rows, another over a part of them."""
    c = Cross([qlen] * 4, [500, 500, 500, 500], 8, 8, 64, BF16, seed=5)
    c.starts_h = np.array([int(c.starts_h[0])] * 3 + [int(c.starts_h[0]) + 37])
    c.lens = [500, 500, 500, 463]
    c.starts = torch.tensor(c.starts_h, dtype=torch.int32, device="cuda")
    c.kv_lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    c.check(c.run())


@pytest.mark.parametrize("qlen", [3, 200])
def test_rows_outside_stay(qlen):
    c = Cross([qlen, 0, qlen + 1], [100, 200, 300], 4, 2, 128, FP16, before=3, behind=5, seed=9)
    out = torch.full_like(c.q, 7.0)
    assert c.run(out=out) is out
    c.check(out)
    assert (out[:3] == 7).all() and (out[-5:] == 7).all()


@pytest.mark.parametrize("qlen", [4, 150])
def test_bad_requests(qlen):
    """Lengths and starts that do not fit: flagged, zero rows, the others as ever."""
    base = dict(H=8, Hkv=4, D=64, dtype=BF16, seed=11)
    for what, val in (("len", -1), ("len", 401), ("len", 2 ** 31 - 1), ("start", -1),
                      ("start", 2 ** 31 - 1), ("start", "end")):
        c = Cross([qlen] * 4, [300, 400, 200, 100], **base)
        t = c.kv_lens if what == "len" else c.starts
        t[1] = c.k.shape[0] - 399 if val == "end" else val
        out = torch.full_like(c.q, 7.0)
        c.run(out=out)
        c.check(out, f"{what} {val}", skip=(1,))
        assert (out[qlen:2 * qlen] == 0).all()
        assert c.status.item() == pk.PA_DEV_BAD_CONTEXT
    # more queries than the bound
    for bound in (1, qlen - 1):
        c = Cross([bound, qlen, bound], [300, 400, 200], **base)
        out = torch.full_like(c.q, 7.0)
        c.run(max_q=bound, out=out)
        c.check(out, f"bound {bound}", skip=(1,))
        assert (out[bound:bound + qlen] == 0).all()
        assert c.status.item() == pk.PA_DEV_BAD_CONTEXT


@pytest.mark.parametrize("qlen", [4, 150])
def test_bad_offsets(qlen):
    """Offsets that fall or leave the array lose their own requests only."""
    for bad in (-5, 10 ** 6):
        c = Cross([qlen] * 4, [300, 400, 200, 100], 8, 4, 64, BF16, seed=12)
        c.offsets[4] = bad
        out = torch.full_like(c.q, 7.0)
        c.run(out=out)
        c.check(out, f"offset {bad}", skip=(3,))
        assert (out[3 * qlen:] == 7).all()
        assert c.status.item() == pk.PA_DEV_BAD_CONTEXT


@pytest.mark.parametrize("H,Hkv", [(4, 4), (160, 1)])
def test_no_states_at_all(H, Hkv):
    q = torch.randn(6, H, 64, device="cuda").to(BF16)
    k = torch.empty(0, Hkv, 64, device="cuda").to(BF16)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    if H // Hkv * 4 > 16 and H // Hkv > 128:
        with pytest.raises(pk.PagedKVError) as e:
            pk.pa_cross_attention(q, k, k, off, zero, zero, 0.1, 4, 0, out=out)
        assert e.value.code == pk.PA_ERR_UNSUPPORTED
        return
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.pa_cross_attention(q, k, k, off, zero, zero, 0.1, 4, 0, out=out, status=status)
    assert (out == 0).all() and status.item() == 0
    pk.pa_cross_attention(q, k, k, off, zero, zero, 0.1, out=out.fill_(7), status=status)
    assert (out == 0).all() and status.item() == 0
    zero[1] = 1  # a state that is not there
    pk.pa_cross_attention(q, k, k, off, zero, zero, 0.1, 4, 8, out=out.fill_(7), status=status)
    assert (out == 0).all() and status.item() == pk.PA_DEV_BAD_CONTEXT


@pytest.mark.parametrize("H,Hkv", [(4, 4), (40, 2)])
def test_no_queries(H, Hkv):
    """Requests without queries under a bound of none: nothing is written.  (One query counts
    as within it.)"""
    c = Cross([0, 0, 0], [300, 5000, 1], H, Hkv, 64, BF16, behind=4, seed=18)
    out = torch.full_like(c.q, 7.0)
    c.run(max_q=0, out=out)
    assert (out == 7).all() and c.status.item() == 0
    c = Cross([1, 0, 2], [300, 5000, 1], H, Hkv, 64, BF16, seed=19)
    c.run(max_q=0, out=out[:3])
    c.check(out[:3], skip=(2,))
    assert (out[1:3] == 0).all() and (out[3] == 7).all()
    assert c.status.item() == pk.PA_DEV_BAD_CONTEXT


@pytest.mark.parametrize("qlen", [4, 150])
def test_strided_queries(qlen):
    c = Cross([qlen, qlen], [777, 130], 8, 8, 64, FP16, seed=13)
    wide = torch.zeros(c.q.shape[0], 11, 64, dtype=FP16, device="cuda")
    wide[:, 2:10] = c.q
    c.q = wide[:, 2:10]
    c.check(c.run())


@pytest.mark.parametrize("qlen", [4, 150])
def test_far_rows(qlen):
    """Rows whose offset passes 2^32 elements."""
    H, D, n = 8, 64, 200
    row = 2 ** 16  # elements between rows
    rows = (2 ** 32 + 2 ** 27) // row
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.empty(rows * row, dtype=FP16, device="cuda").view(rows, row)
    k = buf[:, :H * D].unflatten(1, (H, D))
    v = buf[:, 4096:4096 + H * D].unflatten(1, (H, D))
    start = rows - n
    k[start:] = torch.randn(n, H, D, generator=g, device="cuda").to(FP16)
    v[start:] = torch.randn(n, H, D, generator=g, device="cuda").to(FP16)
    q = torch.randn(qlen, H, D, generator=g, device="cuda").to(FP16)
    t = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, qlen], [start], [n])]
    out = pk.pa_cross_attention(q, k, v, *t, 0.125, qlen, n)
    check(out, *attend(q, k[start:], v[start:], 0.125, n))


@pytest.mark.parametrize("qlen", [4, 150])
def test_captured_and_replayed(qlen):
    """A graph over buffers whose lengths and data change between replays."""
    c = Cross([qlen] * 3, [3000, 900, 1], 8, 4, 128, BF16, seed=15)
    out = torch.empty_like(c.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(out=out)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.run(out=out)
    for lens in ([3000, 900, 1], [0, 17, 1], [2999, 640, 0]):
        c.lens = lens
        c.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.q.normal_()
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, f"{lens}")


def test_other_stream():
    c = Cross([4] * 3, [5000, 900, 1], 8, 4, 128, BF16, seed=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(stream=s)
    s.synchronize()
    c.check(out)


def test_small_weights_beside_a_large_one():
    """One key far above 4,000 others, whose weights are small but not nothing."""
    for qlen, dtype in ((2, FP16), (40, FP16), (2, BF16)):
        c = Cross([qlen], [4000], 4, 4, 64, dtype, seed=17)
        s = int(c.starts_h[0])
        c.k[s + 1000] = 3.0 * c.q[0]
        c.check(c.run(), f"{qlen} {dtype}")


def test_refusals():
    c = Cross([2, 2], [10, 20], 8, 4, 64, BF16)
    a = [c.q, c.k, c.v, c.offsets, c.starts, c.kv_lens]

    def call(i=None, x=None, **kw):
        args = list(a)
        if i is not None:
            args[i] = x
        return pk.pa_cross_attention(*args, kw.pop("scale", 0.1), **kw)

    for i, x, err in ((0, c.q.float(), TypeError), (1, c.k.half(), TypeError),
                      (2, c.v[:-1], ValueError), (1, c.k[:, :3], ValueError),
                      (3, c.offsets.long(), TypeError), (3, c.offsets[:2], ValueError),
                      (4, c.starts[:1], ValueError), (5, c.kv_lens.cpu(), ValueError),
                      (0, c.q.cpu(), ValueError), (0, None, TypeError),
                      (1, c.k.transpose(1, 2).contiguous().transpose(1, 2), ValueError)):
        with pytest.raises(err):
            call(i, x)
    for kw, err in ((dict(out=c.q[:3]), ValueError), (dict(out=c.q.float()), TypeError),
                    (dict(workspace=3), TypeError), (dict(status=c.q), TypeError),
                    (dict(scale=0.0), pk.PagedKVError), (dict(scale=float("nan")), pk.PagedKVError),
                    (dict(max_q_len=-1), pk.PagedKVError), (dict(max_kv_len=-1), pk.PagedKVError)):
        with pytest.raises(err):
            call(**kw)
    c = Cross([2], [50000], 8, 4, 64, BF16)
    a = [c.q, c.k, c.v, c.offsets, c.starts, c.kv_lens]
    assert pk.pa_cross_attention_workspace_size(1, 2, 8, 4, 64, 2, 50000) > 64
    with pytest.raises(pk.PagedKVError) as e:
        call(max_q_len=2, max_kv_len=50000,
             workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pk.PA_ERR_WORKSPACE
