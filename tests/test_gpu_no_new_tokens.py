"""Packed batches that are said to have no new tokens (max_q = 0): rows that no sequence owns are left as they were, and
sequences that have some all the same are reported, as with any other max_q that is too small."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests.paged_reference import Pool
from tests.test_gpu_paged_attention import check_sequence, starts_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,four", [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True), (torch.float32, True)])
def test_paged_attention(cuda_device, dtype, four):
    pool = Pool([50, 60, 9], 2, 16, 64, dtype, four)
    q = torch.randn(6, 4, 64, device="cuda", dtype=dtype)
    for new, bits in (([0, 0, 0], 0), ([0, 1, 0], 0), ([2, 0, 1], 0x10)):
        out, lse = torch.full_like(q, 7.0), torch.full((6, 4), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, q_starts=starts_of(new), max_q=0, out=out, lse=lse, error_word=err)
        assert int(err) == bits
        at, done = 0, torch.zeros(6, dtype=torch.bool, device="cuda")
        for b, n in enumerate(new):
            if n:  # the first of its tokens
                row = slice(at, at + 1)
                check_sequence(pool, b, q[row], out[row], lse[row], pool.lens[b], 0, None, 64 ** -0.5, n)
                done[row] = True
            at += n
        assert (out[~done] == 7).all() and (lse[~done] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_window_attention(cuda_device, dtype):
    q, k = torch.randn(6, 4, 64, device="cuda", dtype=dtype), torch.randn(40, 2, 64, device="cuda", dtype=dtype)
    ks = starts_of([20, 20])
    for new, bits in (([0, 0], 0), ([2, 0], 0x10)):
        out, err = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        kv.window_attention(q, k, k, q_starts=starts_of(new), k_starts=ks, max_q=0, max_k=20, out=out, error_word=err)
        assert int(err) == bits and (out[1:] == 7).all() and bool((out[0] == 7).all()) == (bits == 0)
