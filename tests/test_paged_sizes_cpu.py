"""Query rows of a KV head (new tokens times heads a group) are counted in 32 bits on the device: calls with more are refused."""
import ctypes

import pytest

from tests.test_paged_cpu import L, attention  # noqa: F401


@pytest.mark.parametrize("page_dtype", [1, 2])
@pytest.mark.parametrize("tokens,starts,max_q,ok", [(1 << 25, 4096, 1 << 25, False), (1 << 26, 4096, 1 << 25, False), (1 << 26, 0, 0, False),
                                                    ((1 << 25) - 1, 4096, 1 << 30, True), (1 << 26, 4096, (1 << 25) - 1, True),
                                                    (1 << 29, 4096, 1 << 29, False), (1 << 29, 4096, 7, True)])
def test_rows_beyond_32_bits(L, page_dtype, tokens, starts, max_q, ok):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = attention(page_dtype=page_dtype, hq=64, h=1, tokens=tokens, q_starts=starts, max_q=max_q)
    assert L.kvevict_paged_attention_workspace_bytes(a, n) == (0 if ok else -1)
    if not ok:
        assert L.kvevict_paged_attention(a, None) == -1
