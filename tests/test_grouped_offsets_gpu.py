"""The grouped-head calls where offsets pass 32 bits: caches of 4.9 billion
elements and packed rows that lie 33 million elements apart."""
import pytest
import torch

import paged_kv_cache_172_gb300 as pk
from grouped_ref import attend, check
from pk_testutil import zero_status

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


def randn(*shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def test_blocks_behind_4_billion_elements():
    NB, bs, H, Hkv, D, dtype = 300_000, 16, 16, 8, 128, torch.bfloat16
    k_cache = torch.empty(NB, bs, Hkv, D, dtype=dtype, device=DEV)
    v_cache = torch.empty_like(k_cache)
    assert k_cache.numel() > 2 ** 32
    ctx = [300, 77]
    # blocks on both sides of 2^31 and 2^32 elements, the last one among them
    ids = [NB - 1, 3, NB - 2, 131_071, 131_072, 262_143, 262_144] + list(range(NB - 40, NB - 20))
    tables = torch.full((2, 19), -1, dtype=torch.int32)
    tables[0, :19] = torch.tensor(ids[:19])
    tables[1, :5] = torch.tensor(ids[19:24])
    tables = tables.to(DEV)
    slots = torch.cat([tables[b, torch.arange(n, device=DEV) // bs].long() * bs
                       + torch.arange(n, device=DEV) % bs for b, n in enumerate(ctx)])
    T = sum(ctx)
    q = randn(T, H, D, dtype=dtype, seed=1)
    k, v = randn(T, Hkv, D, dtype=dtype, seed=2), randn(T, Hkv, D, dtype=dtype, seed=3)
    still = pk.pa_rope_table(torch.zeros(D // 2), device=DEV)  # turns by nothing
    status = zero_status(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    q_out, _ = pk.pa_rope_cache_write(q, k, v, pos, still, slots, k_cache, v_cache, status=status)
    assert torch.equal(q_out, q)
    assert torch.equal(k_cache.flatten(0, 1)[slots], k)
    assert torch.equal(v_cache.flatten(0, 1)[slots], v)

    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, *ctx], dtype=torch.int32, device=DEV).cumsum(0).int()
    scale = D ** -0.5
    last = q[[ctx[0] - 1, T - 1]].contiguous()
    for pt in (0, 64, 2048):
        got = pk.pa_decode_grouped(last, k_cache, v_cache, tables, lens, scale, max(ctx),
                                   partition_tokens=pt, status=status)
        for b in range(2):
            rows = slice(sum(ctx[:b]), sum(ctx[:b + 1]))
            ref, tol = attend(last[b:b + 1], k[rows], v[rows], scale, ctx[b] - 1)
            check(got[b:b + 1], ref, tol, f"decode {b}, partition {pt}")
    got = pk.pa_chunk_attention(q, k_cache, v_cache, tables, lens, offsets, scale, status=status)
    for b in range(2):
        rows = slice(sum(ctx[:b]), sum(ctx[:b + 1]))
        ref, tol = attend(q[rows], k[rows], v[rows], scale, 0)
        check(got[rows], ref, tol, f"chunk {b}")
    assert int(status.item()) == 0


def test_rows_33_million_elements_apart():
    T, H, Hkv, D, dtype = 70, 8, 2, 64, torch.float16
    step = 2 ** 25  # T * step > 2^31 elements, 2^32 bytes
    room = torch.empty((T - 1) * step + 4096, dtype=dtype, device=DEV)
    q = room.as_strided((T, H, D), (step, D, 1), 0)
    k = room.as_strided((T, Hkv, D), (step, D, 1), 1024)
    v = room.as_strided((T, Hkv, D), (step, D, 1), 2048)
    q0, k0 = randn(T, H, D, dtype=dtype, seed=4), randn(T, Hkv, D, dtype=dtype, seed=5)
    v0 = randn(T, Hkv, D, dtype=dtype, seed=6)
    q.copy_(q0)
    k.copy_(k0)
    v.copy_(v0)
    status = zero_status(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    still = pk.pa_rope_table(torch.zeros(D // 2), device=DEV)
    q_out, k_out = pk.pa_rope_cache_write(q, k, None, pos, still, None, q_out=q, k_out=k,
                                          status=status)
    assert torch.equal(q_out, q0) and torch.equal(k_out, k0)
    offsets = torch.tensor([0, 40, T], dtype=torch.int32, device=DEV)
    got = pk.pa_prompt_attention(q, k, v, offsets, 0.125, status=status)
    for rows in (slice(0, 40), slice(40, T)):
        ref, tol = attend(q0[rows], k0[rows], v0[rows], 0.125, 0)
        check(got[rows], ref, tol, f"rows {rows}")
    # the same rows as one chunk over a cache
    k_cache, v_cache = torch.zeros(2, 5, 16, Hkv, D, dtype=dtype, device=DEV)
    k_cache.view(80, Hkv, D)[:T] = k0
    v_cache.view(80, Hkv, D)[:T] = v0
    got = pk.pa_chunk_attention(q, k_cache, v_cache,
                                torch.arange(5, dtype=torch.int32, device=DEV)[None],
                                torch.tensor([T], dtype=torch.int32, device=DEV),
                                torch.tensor([0, T], dtype=torch.int32, device=DEV), 0.125,
                                status=status)
    ref, tol = attend(q0, k0, v0, 0.125, 0)
    check(got, ref, tol, "chunk")
    assert int(status.item()) == 0
