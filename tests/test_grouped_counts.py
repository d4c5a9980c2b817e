"""Counts that the packed calls' 32-bit arithmetic cannot step past are refused before
anything is launched."""
import pytest

import paged_kv_cache_172_gb300 as pk
from paged_kv_cache_172_gb300 import build_lib

P = 0x1000  # any 32-byte aligned address: these calls return before touching memory
PAST = (2 ** 31 - 32768, 2 ** 31 - 4, 2 ** 31 - 1)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pk.lib()


@pytest.mark.parametrize("T", PAST)
def test_tokens_of_prompts(lib, T):
    assert lib.pa_prompt_attention(P, P, P, P, 1, T, 1, 1, 64, 0, 64, 64, 64, 0.1, P, None,
                                   None) == pk.PA_ERR_INVALID


@pytest.mark.parametrize("T", PAST)
def test_tokens_of_chunks(lib, T):
    assert lib.pa_chunk_attention(P, P, P, P, P, P, 1, T, 1, 1, 64, 0, 64, 16, 8, 4, 64, 0.1, P,
                                  None, 0, None, None) == pk.PA_ERR_INVALID


@pytest.mark.parametrize("T", PAST)
def test_tokens_of_the_rotation(lib, T):
    assert lib.pa_rope_cache_write(P, P, None, P, P, None, T, 1, 1, 64, 64, 1, 0, 0, 64, 64, 0, 16,
                                   8, P, 64, P, 64, None, None, None, None) == pk.PA_ERR_INVALID


@pytest.mark.parametrize("cap", PAST)
def test_a_refused_context_needs_no_workspace(lib, cap):
    # as other refused arguments; the partitions of such contexts cannot be counted in 32 bits
    for pt in (0, 64):
        assert pk.pa_decode_grouped_workspace_size(2, 8, 2, 128, 16, cap, pt) == 0
    assert pk.pa_chunk_attention_workspace_size(2, 8, 8, 2, 128, cap) == 0
    assert pk.pa_chunk_attention_workspace_size(2, cap, 8, 2, 128, 100) == 0
