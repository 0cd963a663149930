"""Tensors that a cache's calls make themselves are used by kernels on the handle's stream: they have to come from the
allocator in that stream's order, and be held for the stream of the caller that reads them. With the allocator and the
streams faked, on the CPU."""
import contextlib
import types

import pytest
import torch

from kv_cache_eviction_decode_gb300 import BF16, RANDOM, KVEvictCache, api, ops


class Stream:
    def __init__(self, number):
        self.cuda_stream, self.device_index, self.device = number, 0, torch.device("cpu")


class Library:
    """Every call succeeds; a size asked for is 64 KiB."""

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                args[-1]._obj.value = 1 << 16
            return 0
        return call


@pytest.fixture
def made(monkeypatch):
    """(cache, list of (tensor, stream it was made on), set of (tensor's address, stream it was held for))."""
    mine, callers = Stream(7), Stream(3)
    now, log, held = [callers], [], set()

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: now[-1])
    monkeypatch.setattr(ops, "_raw_stream", lambda d: now[-1].cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.add((t.data_ptr(), s)))
    for name in ("empty", "empty_like"):
        def make(*a, real=getattr(torch, name), **kw):
            t = real(*a, **kw)
            log.append((t, now[-1]))
            return t
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(api, "lib", Library)
    monkeypatch.setattr(KVEvictCache, "stats", lambda self: {"capacity": 16})
    c = KVEvictCache(policy=RANDOM, budget=16, batch=2, n_layers=1, n_q_heads=4, n_kv_heads=2, head_dim=64, dtype=BF16,
                     device="cpu", stream=mine)
    return types.SimpleNamespace(c=c, log=log, held=held, mine=mine, callers=callers, now=now)


def calls(c):
    def z(*s):
        return torch.zeros(s, dtype=torch.bfloat16)
    Q, K, q, k, pre = z(2, 4, 5, 64), z(2, 2, 5, 64), z(2, 4, 64), z(2, 2, 64), z(2, 9, 64)
    return {"prefill_attend": lambda: c.prefill_attend(0, Q, K, K, return_lse=True),
            "decode_step_shared": lambda: c.decode_step_shared(0, q, k, k, pre, pre),
            "decode_step": lambda: c.decode_step(0, q, k, k),
            "prefill_scored": lambda: c.prefill_scored(0, Q, K, K),
            "prefill_snapkv": lambda: c.prefill_snapkv(0, Q, K, K, 3),
            "select_victims": lambda: c.select_victims(0, torch.zeros(2, 2, 16))}


@pytest.mark.parametrize("name", ["prefill_attend", "decode_step_shared", "decode_step", "prefill_scored", "prefill_snapkv", "select_victims"])
def test_made_on_the_handles_stream_and_held_for_the_callers(made, name):
    made.log.clear()
    got = calls(made.c)[name]()
    assert made.log and all(s is made.mine for _, s in made.log)
    for t in got if isinstance(got, tuple) else (got,):
        assert any(m.untyped_storage().data_ptr() == t.untyped_storage().data_ptr() and (m.data_ptr(), made.callers) in made.held
                   for m, _ in made.log)


def test_the_state_is_made_on_the_handles_stream(made):
    assert [s for t, s in made.log if t is made.c.state] == [made.mine]


def test_nothing_is_held_where_the_streams_are_one(made):
    made.now[:] = [made.mine]
    made.held.clear()
    for call in calls(made.c).values():
        call()
    assert not made.held
