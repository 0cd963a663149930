"""A packed batch that is said to have no new tokens (max_q = 0) is launched as one of single tokens, so that the lengths on
the device are looked at."""
import struct

import pytest
import torch

from tests.test_paged_cpu import L, as_if_on_gpu, make  # noqa: F401


def test_max_q_of_zero_counts_as_one(as_if_on_gpu, monkeypatch):  # noqa: F811
    import kv_cache_eviction_decode_gb300 as kv
    from kv_cache_eviction_decode_gb300 import ops, paged
    seen = []
    for m in (ops, paged):
        monkeypatch.setattr(m, "_call", lambda name, dev, args: seen.append((name, args)))
    c = make()
    q, starts = torch.zeros(6, 8, 64).bfloat16(), torch.zeros(4, dtype=torch.int32)
    for max_q in (0, 1, 5):
        kv.paged_attention(q, *c, q_starts=starts, max_q=max_q)
        kv.window_attention(q, q, q, q_starts=starts, k_starts=starts, max_q=max_q, max_k=9)
        (paged_name, a), (window_name, w) = seen[-2:]
        assert (paged_name, window_name) == ("kvevict_paged_attention", "kvevict_window_attention")
        assert paged._ATTENTION_HEAD.unpack_from(a, struct.calcsize("@" + paged._CACHE))[3] == max(1, max_q)
        assert ops._HEAD.unpack_from(w)[7] == max(1, max_q)
    for call in (lambda: kv.paged_attention(q, *c, q_starts=starts, max_q=-1),
                 lambda: kv.window_attention(q, q, q, q_starts=starts, k_starts=starts, max_q=-1, max_k=9)):
        with pytest.raises(ValueError, match="^max_q"):
            call()
