"""The operators without a GPU: the argument structs as the binding packs them,
refusals (made on the host, nothing launched) and the rotary frequencies."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from kv_cache_eviction_decode_gb300 import build
    build.build()
    from kv_cache_eviction_decode_gb300 import _lib
    return _lib.lib()


def test_struct_layouts(tmp_path):
    from kv_cache_eviction_decode_gb300 import ops
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvevict_ops.h"\nint main(void) {'
                   'printf("%zu %zu %zu %zu %zu %zu", sizeof(kvevict_attention_args), sizeof(kvevict_shared_prefix_args), '
                   'sizeof(kvevict_rotary_args), offsetof(kvevict_attention_args, workspace), '
                   'offsetof(kvevict_shared_prefix_args, k_prefix), offsetof(kvevict_rotary_args, inv_freq)); return 0; }')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    assert got == [ops._ATTN.size, ops._SHARED.size, ops._ROT.size, 224, ops._ATTN.size, 208]


def test_pieces_make_the_structs():
    from kv_cache_eviction_decode_gb300 import ops
    attn = ops._HEAD.size + ops._PTRS.size + ops._Q9.size + ops._Q3.size + ops._TAIL.size
    assert attn == ops._ATTN.size and attn + ops._P2.size + 40 == ops._SHARED.size
    assert ops._ROT_HEAD.size + ops._P4.size + ops._Q12.size + ops._ROT_TAIL.size == ops._ROT.size


F = dict(dtype=1, d=128, hq=8, hkv=2, batch=2, n_sink=4, window=64, max_q=0, max_k=0, scale=0.0, q_rows=300, k_rows=300,
         q=4096, k=4096, v=4096, out=4096, lse=0, qs=(8 * 300 * 128, 300 * 128, 128), ks=(2 * 300 * 128, 300 * 128, 128),
         vs=(2 * 300 * 128, 300 * 128, 128), os=(8 * 300 * 128, 300 * 128, 128), q_starts=0, k_starts=0, q_lens=0, kv_lens=0,
         ws=0, wn=0, err=0)


def attn(**kw):
    from kv_cache_eviction_decode_gb300 import ops
    a = {**F, **kw}
    vals = []
    for x in a.values():
        vals += list(x) if isinstance(x, tuple) else [x]
    return ops._ATTN.pack(*vals)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(d=96), dict(hq=7), dict(hkv=0), dict(hq=130, hkv=2), dict(batch=-1), dict(n_sink=-1), dict(window=-1),
    dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(q_rows=-1), dict(k_rows=1 << 30), dict(q_starts=4096),
    dict(q_starts=4096, k_starts=4096, q_lens=4096), dict(q_starts=4096, k_starts=4096, max_q=-1), dict(q_starts=4098, k_starts=4096),
])
def test_window_attention_shapes_refused(L, bad):
    n = ctypes.c_size_t(0)
    assert L.kvevict_window_attention_workspace_bytes(attn(**bad), n) == -1
    assert L.kvevict_window_attention(attn(**bad), None) == -1


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(v=4104), dict(out=4098), dict(qs=(1, 300 * 128, 128)), dict(ks=(2 * 300 * 128, 0, 128)),
    dict(vs=(2 * 300 * 128, 300 * 128, 130)), dict(os=(-8, 300 * 128, 128)), dict(lse=4097), dict(kv_lens=4097), dict(err=4098),
])
def test_window_attention_tensors_refused(L, bad):
    assert L.kvevict_window_attention(attn(**bad), None) == -1


def test_workspace_too_small_or_missing_refused(L):
    n = ctypes.c_size_t(0)
    step = dict(q_rows=1, k_rows=20000, window=0, qs=(1024, 128, 128), os=(1024, 128, 128), ks=(2 * 20000 * 128, 20000 * 128, 128),
                vs=(2 * 20000 * 128, 20000 * 128, 128))
    assert L.kvevict_window_attention_workspace_bytes(attn(**step), n) == 0 and n.value > 0
    assert L.kvevict_window_attention(attn(**step), None) == -1
    assert L.kvevict_window_attention(attn(**step, ws=4096, wn=n.value - 1), None) == -1
    assert L.kvevict_window_attention(attn(**step, ws=4096 + 16, wn=n.value), None) == -1


def test_nothing_to_do_is_ok(L):
    assert L.kvevict_window_attention(attn(q_rows=0), None) == 0
    assert L.kvevict_window_attention(attn(batch=0), None) == 0
    assert L.kvevict_window_attention(attn(q_starts=4096, k_starts=4096, max_q=0), None) == 0
    assert L.kvevict_window_attention(None, None) == -1


def shared(tail=None, **kw):
    from kv_cache_eviction_decode_gb300 import ops
    a = {**F, "n_sink": 0, "window": 0, "q_rows": 1, **kw}
    vals = []
    for x in a.values():
        vals += list(x) if isinstance(x, tuple) else [x]
    t = {"kp": 4096, "vp": 4096, "kps": (500 * 128, 128), "vps": (500 * 128, 128), "P": 500, **(tail or {})}
    return ops._SHARED.pack(*vals, t["kp"], t["vp"], *t["kps"], *t["vps"], t["P"])


@pytest.mark.parametrize("bad", [dict(n_sink=1), dict(window=5), dict(q_rows=2), dict(q_lens=4096), dict(q_starts=4096, k_starts=4096),
                                 dict(tail=dict(P=-1)), dict(tail=dict(P=1 << 30))])
def test_shared_prefix_shapes_refused(L, bad):
    n = ctypes.c_size_t(0)
    assert L.kvevict_shared_prefix_attention_workspace_bytes(shared(**bad), n) == -1
    assert L.kvevict_shared_prefix_attention(shared(**bad), None) == -1


@pytest.mark.parametrize("bad", [dict(q=0), dict(k=0), dict(tail=dict(kp=0)), dict(tail=dict(vp=4100)),
                                 dict(tail=dict(kps=(500 * 128, 0))), dict(tail=dict(vps=(100, 128)))])
def test_shared_prefix_tensors_refused(L, bad):
    n = ctypes.c_size_t(0)
    assert L.kvevict_shared_prefix_attention_workspace_bytes(shared(), n) == 0 and n.value > 0
    assert L.kvevict_shared_prefix_attention(shared(**bad, ws=4096, wn=n.value), None) == -1
    assert L.kvevict_shared_prefix_attention(shared(), None) == -1  # no workspace
    assert L.kvevict_shared_prefix_attention(None, None) == -1


R = dict(dtype=1, d=128, rd=128, il=0, inv=0, p64=1, hq=8, hk=2, batch=1, tokens=10, q=4096, k=4096, qo=4096, ko=4096,
         qs=(10240, 1280, 128), qos=(10240, 1280, 128), ks=(2560, 1280, 128), kos=(2560, 1280, 128), pos=4096, ps=(0, 1), start=0,
         f=4096, scale=1.0)


def rot(**kw):
    from kv_cache_eviction_decode_gb300 import ops
    vals = []
    for x in {**R, **kw}.values():
        vals += list(x) if isinstance(x, tuple) else [x]
    return ops._ROT.pack(*vals)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(d=12), dict(d=2048), dict(rd=0), dict(rd=3), dict(rd=130), dict(il=2), dict(inv=-1), dict(p64=2),
    dict(tokens=-1), dict(batch=1 << 31), dict(batch=1 << 16, tokens=1 << 16), dict(hq=-1), dict(scale=math.inf), dict(f=0), dict(f=4100),
    dict(q=0), dict(qo=4104), dict(ko=0), dict(qs=(10240, 1281, 128)), dict(qos=(10240, 128, 1024)), dict(pos=4100),
])
def test_rotary_refused(L, bad):
    assert L.kvevict_rotary(rot(**bad), None) == -1


def test_rotary_nothing_to_do(L):
    assert L.kvevict_rotary(rot(tokens=0), None) == 0
    assert L.kvevict_rotary(rot(hq=0, k=0), None) == 0
    assert L.kvevict_rotary(None, None) == -1


def test_python_refusals():
    import kv_cache_eviction_decode_gb300 as kv
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kv.window_attention(q, q, q)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        kv.window_attention(q.half(), q.half(), q.half())
    with pytest.raises(ValueError, match="CUDA"):
        kv.rotary(q, None, 0, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        kv.shared_prefix_attention(q[0], q[0], q[0], q, q)


def test_frequencies():
    import kv_cache_eviction_decode_gb300 as kv
    i = torch.arange(64, dtype=torch.float64)
    plain, s = kv.rotary_frequencies(128, device="cpu")
    assert s == 1.0 and torch.allclose(plain, 10000.0 ** (-i / 64), rtol=1e-15)
    lin, s = kv.rotary_frequencies(128, scaling="linear", factor=8.0, device="cpu")
    assert s == 1.0 and torch.equal(lin, plain / 8)
    ntk, s = kv.rotary_frequencies(128, scaling="ntk", factor=8.0, device="cpu")
    assert s == 1.0 and ntk[0] == 1 and math.isclose(ntk[-1], plain[-1] / 8, rel_tol=1e-12)
    yarn, s = kv.rotary_frequencies(128, scaling="yarn", factor=8.0, device="cpu")
    assert math.isclose(s, 0.1 * math.log(8) + 1) and torch.equal(yarn[:10], plain[:10]) and torch.allclose(yarn[-10:], plain[-10:] / 8, rtol=1e-15)
    turns = 4096 * plain / (2 * math.pi)
    assert ((yarn < plain * (1 + 1e-15)) & (yarn > plain / 8 * (1 - 1e-15))).all()
    assert (yarn[turns > 40] == plain[turns > 40]).all()
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, factor=0.5),
                dict(rotary_dim=64, scaling="other"), dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            kv.rotary_frequencies(device="cpu", **bad)


@pytest.mark.parametrize("bad", [
    dict(qos=(10240, 0, 128)), dict(qos=(10240, 1280, 0)), dict(kos=(2560, 1280, 0)), dict(batch=2, qos=(0, 1280, 128)),
    dict(qo=4096, qs=(10240, 0, 128), qos=(10240, 0, 128)),
])
def test_rotary_outputs_that_share_rows_refused(L, bad):
    """An output stride of 0 over an axis of several entries: they would all write the same row."""
    assert L.kvevict_rotary(rot(**{"qo": 1 << 20, "ko": 1 << 21, **bad}), None) == -1


def test_inputs_that_require_gradients_refused():
    """The operators have no backward pass: an output without a graph would lose the gradient without a word."""
    import kv_cache_eviction_decode_gb300 as kv
    q = torch.zeros(1, 2, 3, 64)
    w = torch.zeros(1, 2, 3, 64, requires_grad=True)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda x: kv.window_attention(x, q, q), lambda x: kv.window_attention(q, x, q), lambda x: kv.window_attention(q, q, x),
                 lambda x: kv.window_attention(q, q, q, out=x), lambda x: kv.rotary(x, None, 0, f), lambda x: kv.rotary(q, x, 0, f),
                 lambda x: kv.rotary(q, None, 0, f, q_out=x), lambda x: kv.rotary(q, q, 0, f, k_out=x),
                 lambda x: kv.shared_prefix_attention(x[0], q[0], q[0], q, q), lambda x: kv.shared_prefix_attention(q[0], x[0], q[0], q, q),
                 lambda x: kv.shared_prefix_attention(q[0], q[0], x[0], q, q), lambda x: kv.shared_prefix_attention(q[0], q[0], q[0], x, q),
                 lambda x: kv.shared_prefix_attention(q[0], q[0], q[0], q, x),
                 lambda x: kv.shared_prefix_attention(q[0], q[0], q[0], q, q, out=x[0])):
        with pytest.raises(ValueError, match="no backward"):
            call(w)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # the next check
            call(w)


def test_cache_inputs_that_require_gradients_refused():
    from kv_cache_eviction_decode_gb300 import KVEvictCache
    c = object.__new__(KVEvictCache)
    c.B, c.Hq, c.Hkv, c.D, c.dtype, c.device = 1, 2, 2, 64, torch.float32, torch.device("cpu")
    q = torch.zeros(1, 2, 3, 64)
    w = torch.zeros(1, 2, 3, 64, requires_grad=True)
    for i in range(3):
        with pytest.raises(ValueError, match="no backward"):
            c.prefill_attend(0, *(w if j == i else q for j in range(3)))
    for i in range(5):
        with pytest.raises(ValueError, match="no backward"):
            c.decode_step_shared(0, *((w if j == i else q)[:, :, 0] if j < 3 else (w if j == i else q)[0] for j in range(5)))


@pytest.fixture
def as_if_on_gpu(monkeypatch, L):
    """Lets the binding's checks see CPU tensors as the device's; what passes them all would launch, and stops here."""
    from kv_cache_eviction_decode_gb300 import ops
    monkeypatch.setattr(ops, "_dtype", lambda t, name: ops._DT[t.dtype])

    def launch(*a):
        raise RuntimeError("launched")
    monkeypatch.setattr(ops, "_call", launch)
    monkeypatch.setattr(ops, "_layouts", {})


BAD_STRIDES = {"expanded": lambda t: t[:, :1].expand(t.shape), "unaligned": lambda t: torch.empty(*t.shape[:-1], 67).bfloat16()[..., :64]}


@pytest.mark.parametrize("how", list(BAD_STRIDES))
def test_strides_refused_by_name(as_if_on_gpu, how):
    """Expanded tensors, and rows that start off a 16-byte boundary: refused with the tensor's name."""
    import kv_cache_eviction_decode_gb300 as kv
    bad = BAD_STRIDES[how]
    q, k, p, s = (torch.zeros(x, dtype=torch.bfloat16) for x in ((2, 4, 3, 64), (2, 2, 9, 64), (2, 5, 64), (2, 4, 64)))
    f = torch.zeros(32, dtype=torch.float64)
    starts = torch.zeros(3, dtype=torch.int32)
    packed = dict(q_starts=starts, k_starts=starts, max_q=1, max_k=1)
    for name, call in (("q", lambda: kv.window_attention(bad(q), k, k)), ("k", lambda: kv.window_attention(q, bad(k), k)),
                       ("v", lambda: kv.window_attention(q, k, bad(k))), ("out", lambda: kv.window_attention(q, k, k, out=bad(q))),
                       ("v", lambda: kv.window_attention(s, p, bad(p), **packed)), ("k", lambda: kv.window_attention(s, bad(p), p, **packed)),
                       ("q", lambda: kv.shared_prefix_attention(bad(s), p, p, k, k)),
                       ("k_prefix", lambda: kv.shared_prefix_attention(s, bad(p), p, k, k)),
                       ("v_prefix", lambda: kv.shared_prefix_attention(s, p, bad(p), k, k)),
                       ("k", lambda: kv.shared_prefix_attention(s, p, p, bad(k), k)), ("v", lambda: kv.shared_prefix_attention(s, p, p, k, bad(k))),
                       ("out", lambda: kv.shared_prefix_attention(s, p, p, k, k, out=bad(s))),
                       ("q_out", lambda: kv.rotary(q, None, 0, f, q_out=bad(q))), ("k_out", lambda: kv.rotary(q, q, 0, f, k_out=bad(q)))):
        with pytest.raises(ValueError, match=f"^{name}: .*16 bytes"):
            call()
    if how == "unaligned":
        for name, call in (("q", lambda: kv.rotary(bad(q), None, 0, f)), ("k", lambda: kv.rotary(q, bad(q), 0, f))):
            with pytest.raises(ValueError, match=f"^{name}: .*16 bytes"):
                call()


def test_strides_accepted(as_if_on_gpu):
    """Axes of one entry in any stride, tensors without entries, and (rotary only reads them) expanded inputs."""
    import kv_cache_eviction_decode_gb300 as kv
    q, k, f = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.float64)
    odd = torch.zeros(1000, dtype=torch.bfloat16).as_strided((2, 4, 1, 64), (256, 64, 3, 1))
    none = torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16).expand(2, 2, 9, 64)[:, :, :0]
    for call in (lambda: kv.window_attention(odd, k, k), lambda: kv.window_attention(q, none, none), lambda: kv.window_attention(q, k, k, out=odd),
                 lambda: kv.rotary(odd, odd[:, :1].expand(2, 4, 1, 64), 0, f, q_out=odd)):
        with pytest.raises(RuntimeError, match="launched"):
            call()


def test_operator_errors_refused(L):
    import kv_cache_eviction_decode_gb300 as kv
    assert L.kvevict_operator_errors(None) == -1
    with pytest.raises(ValueError, match="CUDA"):
        kv.operator_errors("cpu")


def test_counts_beyond_32_bits(as_if_on_gpu):
    """More sinks, a longer window or longest sequence than any tensor holds is as much as all of it."""
    import kv_cache_eviction_decode_gb300 as kv
    q, k, s = (torch.zeros(x, dtype=torch.bfloat16) for x in ((2, 4, 3, 64), (2, 2, 9, 64), (7, 4, 64)))
    starts = torch.tensor([0, 7], dtype=torch.int32)
    for call in (lambda: kv.window_attention(q, k, k, n_sink=2**40), lambda: kv.window_attention(q, k, k, window=2**40),
                 lambda: kv.window_attention(s, s, s, q_starts=starts, k_starts=starts, max_q=2**40, max_k=2**40)):
        with pytest.raises(RuntimeError, match="launched"):
            call()
    with pytest.raises(ValueError, match="max_q"):
        kv.window_attention(s, s, s, q_starts=starts, k_starts=starts, max_q=-1, max_k=7)
