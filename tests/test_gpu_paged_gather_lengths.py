"""paged_gather, packed: a sequence longer than its rows is reported, also where it has no rows at all."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests.paged_reference import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("starts,lens,bits", [([0, 0, 20], [5, 20], 0x10), ([0, 20, 20], [20, 1], 0x10), ([0, 0, 20], [0, 20], 0), ([0, 20, 20], [20, 0], 0),
                                              ([0, 0, 20], [-1, 20], 0x10), ([3, 3, 3], [0, 9], 0x10), ([0, 4, 20], [5, 16], 0x10),
                                              ([0] * 300 + [20], [0] * 299 + [20], 0), ([0] * 300 + [20], [0] * 270 + [1] + [0] * 28 + [20], 0x10)])
def test_sequences_without_rows(cuda_device, starts, lens, bits, four):
    pool = Pool(lens, 2, 16, 64, torch.bfloat16, four, garbage=False)
    k, v = (torch.full((20, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), k_out=k, v_out=v,
                    error_word=err)
    assert int(err) == bits
    done = torch.zeros(20, dtype=torch.bool, device="cuda")
    for b, m in enumerate(lens):
        n = min(max(m, 0), starts[b + 1] - starts[b])
        if n:
            rows = slice(starts[b], starts[b] + n)
            for which, out in enumerate((k, v)):
                assert torch.equal(out[rows].transpose(0, 1), pool.rows(b, n, which)[0].bfloat16())
            done[rows] = True
    assert (k[~done] == 7).all() and (v[~done] == 7).all()
