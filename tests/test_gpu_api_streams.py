"""Outputs that the calls on a cache make themselves, while work is pending on the caller's stream: the handle's kernels
write no memory that this work still reads."""
import pytest
import torch

from kv_cache_eviction_decode_gb300 import BF16, SINK_WINDOW, KVEvictCache

pytestmark = pytest.mark.gpu


def cache(stream=None):
    return KVEvictCache(policy=SINK_WINDOW, batch=2, n_layers=1, n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=BF16, n_sink=4,
                        n_recent=28, budget=32, device="cuda:0", stream=stream)


@pytest.mark.parametrize("call", ["prefill_attend", "decode_step_shared", "decode_step"])
def test_pending_work_keeps_its_memory(cuda_device, call):
    g = torch.Generator(device="cuda").manual_seed(31)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    Q, K, V, q, k, v, kp, vp = (rnd(*s) for s in ((2, 8, 40, 64), (2, 2, 40, 64), (2, 2, 40, 64), (2, 8, 64), (2, 2, 64), (2, 2, 64),
                                                  (2, 500, 64), (2, 500, 64)))
    run = {"prefill_attend": lambda c: c.prefill_attend(0, Q, K, V), "decode_step": lambda c: c.decode_step(0, q, k, v),
           "decode_step_shared": lambda c: c.decode_step_shared(0, q, k, v, kp, vp)}[call]
    want = run(cache())
    side = torch.cuda.Stream()
    c = cache(side)
    for _ in range(3):  # the caller's blocks of an output's size, one after another
        torch.cuda.synchronize()
        x = torch.full_like(want, 3.0)
        torch.cuda._sleep(100_000_000)
        y = x.clone()   # waits behind the sleep
        del x
    out = run(c)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert (y == 3).all() and torch.equal(out, want)
    assert c.check() == 0
