"""Many keys of small weight beside a large one, in fp16: a weight of 2^-25.6 of the
row's largest is below half the smallest step of fp16, but 32,768 of them are 6e-4 of
the result, which fp16 holds to 2^-11.

The first key scores 17.75 (142 / 8) and has v = 0, all others score 0 and have v = 1:
    o = (n - 1) w / (1 + (n - 1) w),  w = e^-17.75.
Bound, relative to o: 2^-5 for the weights (held from 2^6 of the largest down to steps
of 2^-24: 2^-31 of the largest at most, 2^-5.4 of w), the rest (2^-11 for the result,
fp32 sums, exponents of magnitude 26) far below it, taken as 2^-9.
"""
import math

import pytest
import torch

import paged_kv_cache_172_gb300 as pk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
N, H, HKV = 32768, 4, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def tensors(D, rows):
    q = torch.zeros(rows, H, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 1
    k = torch.zeros(N, HKV, D, dtype=torch.float16, device=DEV)
    k[0, :, 0] = 142
    v = torch.ones_like(k)
    v[0] = 0
    return q, k, v


def check(out, seen):
    """out [rows, H, D], seen: keys each row sees."""
    w = math.exp(-17.75)
    small = (torch.as_tensor(seen, dtype=torch.float64, device=DEV) - 1) * w
    o = (small / (1 + small))[:, None, None]
    assert ((out.double() - o).abs() <= (2.0 ** -5 + 2.0 ** -9) * o + 2.0 ** -25).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt(D):
    q, k, v = tensors(D, N)
    off = torch.tensor([0, N], dtype=torch.int32, device=DEV)
    out = pk.pa_prompt_attention(q, k, v, off, 0.125)
    check(out, range(1, N + 1))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("split", [False, True])
def test_chunk(D, split):
    q, k, v = tensors(D, 5)
    tables = torch.arange(N // 16, dtype=torch.int32, device=DEV).view(1, -1)
    ctx = torch.tensor([N], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    out = pk.pa_chunk_attention(q, k.view(-1, 16, HKV, D), v.view(-1, 16, HKV, D), tables, ctx, off,
                                0.125, split=split)
    check(out, range(N - 4, N + 1))


@pytest.mark.parametrize("D", [64, 128])
def test_decode(D):
    q, k, v = tensors(D, 1)
    tables = torch.arange(N // 16, dtype=torch.int32, device=DEV).view(1, -1)
    ctx = torch.tensor([N], dtype=torch.int32, device=DEV)
    for pt in (0, 2048):
        out = pk.pa_decode_grouped(q, k.view(-1, 16, HKV, D), v.view(-1, 16, HKV, D), tables, ctx,
                                   0.125, N, partition_tokens=pt)
        check(out, [N])
