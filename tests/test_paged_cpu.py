"""The paged cache and norm_rotary without a GPU: argument structs, refusals (made on the host, nothing launched), and how
the kernels read the rows of new tokens from the device's starts."""
import ctypes
import os
import random
import struct
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
    from kv_cache_eviction_decode_gb300 import ops, paged
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvevict_paged.h"\nint main(void) {'
                   'printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu", sizeof(kvevict_paged_cache), sizeof(kvevict_paged_append_args), '
                   'sizeof(kvevict_paged_gather_args), sizeof(kvevict_paged_attention_args), sizeof(kvevict_norm_rotary_args), '
                   'offsetof(kvevict_paged_cache, block_table), offsetof(kvevict_paged_append_args, inv_freq), '
                   'offsetof(kvevict_paged_attention_args, q), offsetof(kvevict_norm_rotary_args, q_weight)); return 0; }')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    cache = struct.calcsize("@" + paged._CACHE)
    assert got == [cache, paged._APPEND.size, paged._GATHER.size, paged._ATTENTION.size, ops._NORM.size, 96, cache + 64, cache + 32, ops._ROT.size]
    assert paged._SHAPE.size + paged._PAGES.size + paged._TABLE.size == cache
    assert cache + paged._APPEND_TAIL.size == paged._APPEND.size and cache + paged._GATHER_TAIL.size == paged._GATHER.size
    assert cache + paged._ATTENTION_HEAD.size + paged._ATTENTION_TAIL.size == paged._ATTENTION.size
    assert ops._ROT.size + ops._NORM_TAIL.size == ops._NORM.size


C = dict(dtype=1, page_dtype=1, d=128, h=4, S=16, batch=2, width=10, n=20, kp=4096, vp=4096, ks=(4 * 16 * 128, 16 * 128, 128),
         vs=(4 * 16 * 128, 16 * 128, 128), table=4096, ts=10, lens=4096, err=0)
Q4 = dict(page_dtype=2, ks=(4 * 16 * 80, 16 * 80, 0), vs=(4 * 16 * 80, 16 * 80, 0))


def pack(fmt, fields, kw):
    from kv_cache_eviction_decode_gb300 import paged
    a = {**C, **fields, **kw}
    vals = []
    for x in a.values():
        vals += list(x) if isinstance(x, tuple) else [x]
    return getattr(paged, fmt).pack(*vals)


def append(**kw):
    return pack("_APPEND", dict(k=4096, v=4096, xs=(128, 512, 128, 512), tokens=6, starts=0, freq=4096, pos=0, ps=0, p64=0, R=128, il=0, scale=1.0), kw)


def gather(**kw):
    return pack("_GATHER", dict(ko=4096, vo=4096, kos=(4 * 50 * 128, 50 * 128, 128), vos=(4 * 50 * 128, 50 * 128, 128), rows=50, k_starts=0), kw)


def attention(**kw):
    return pack("_ATTENTION", dict(hq=8, n_sink=0, window=0, max_q=0, max_k=0, scale=0.0, tokens=2, q=4096, out=4096, lse=0, qs=(128, 1024),
                                   os=(128, 1024), q_starts=0, ws=4096, wn=1 << 30), kw)


CACHE_SHAPES = [dict(dtype=2), dict(page_dtype=0), dict(page_dtype=3), dict(d=96), dict(h=0), dict(h=40000), dict(S=8), dict(S=24), dict(S=512),
                dict(batch=-1), dict(width=-1), dict(n=-1), dict(width=1 << 26)]
CACHE_TENSORS = [dict(kp=0), dict(vp=4104), dict(ks=(4 * 16 * 128, 16 * 128, 130)), dict(ks=(0, 16 * 128, 128)), dict(vs=(4 * 16 * 128, -8, 128)),
                 dict(table=0), dict(table=4098), dict(ts=-1), dict(lens=0), dict(lens=4097), dict(err=4098),
                 {**Q4, "ks": (4 * 16 * 80 + 8, 16 * 80, 0)}, {**Q4, "vs": (4 * 16 * 80, 0, 0)}]


@pytest.mark.parametrize("bad", CACHE_SHAPES)
def test_cache_shapes_refused(L, bad):
    n = ctypes.c_size_t(0)
    assert L.kvevict_paged_append(append(**bad), None) == -1
    assert L.kvevict_paged_gather(gather(**bad), None) == -1
    assert L.kvevict_paged_attention(attention(**bad), None) == -1
    assert L.kvevict_paged_attention_workspace_bytes(attention(**bad), n) == -1


@pytest.mark.parametrize("bad", CACHE_TENSORS)
def test_cache_tensors_refused(L, bad):
    assert L.kvevict_paged_append(append(**bad), None) == -1
    assert L.kvevict_paged_gather(gather(**bad), None) == -1
    assert L.kvevict_paged_attention(attention(**bad), None) == -1


@pytest.mark.parametrize("bad", [dict(k=0), dict(v=4104), dict(xs=(130, 512, 128, 512)), dict(xs=(128, 512, 128, -8)), dict(tokens=7), dict(tokens=-1),
                                 dict(tokens=1 << 30, starts=4096), dict(starts=4098), dict(R=3), dict(R=130), dict(R=-2), dict(freq=0), dict(freq=4100),
                                 dict(il=2), dict(p64=2), dict(pos=4098), dict(pos=4100, p64=1), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_append_refused(L, bad):
    assert L.kvevict_paged_append(append(**bad), None) == -1


@pytest.mark.parametrize("bad", [dict(ko=0), dict(vo=4100), dict(kos=(4 * 50 * 128, 0, 128)), dict(vos=(4 * 50 * 128, 50 * 128, 4)), dict(rows=-1),
                                 dict(rows=1 << 30), dict(k_starts=4098)])
def test_gather_refused(L, bad):
    assert L.kvevict_paged_gather(gather(**bad), None) == -1


@pytest.mark.parametrize("bad", [dict(hq=6), dict(hq=0), dict(hq=4 * 65), dict(n_sink=-1), dict(window=-1), dict(max_q=-1), dict(max_k=-1),
                                 dict(scale=-1.0), dict(scale=float("nan")), dict(tokens=3), dict(tokens=-2), dict(q_starts=4098)])
def test_attention_shapes_refused(L, bad):
    n = ctypes.c_size_t(0)
    assert L.kvevict_paged_attention(attention(**bad), None) == -1
    assert L.kvevict_paged_attention_workspace_bytes(attention(**bad), n) == -1


@pytest.mark.parametrize("bad", [dict(q=0), dict(out=4104), dict(qs=(0, 1024)), dict(os=(128, 1028)), dict(lse=4097)])
def test_attention_tensors_refused(L, bad):
    assert L.kvevict_paged_attention(attention(**bad), None) == -1


def test_attention_workspace_refused(L):
    n = ctypes.c_size_t(0)
    long = dict(width=2000)
    assert L.kvevict_paged_attention_workspace_bytes(attention(**long), n) == 0 and n.value > 0
    for bad in (dict(ws=0), dict(ws=4096 + 16), dict(wn=n.value - 1)):
        assert L.kvevict_paged_attention(attention(**long, **bad), None) == -1
    assert L.kvevict_paged_attention_workspace_bytes(attention(**long), None) == -1


def test_nothing_to_do_is_ok(L):
    for a in (dict(tokens=0), dict(tokens=0, batch=0)):
        assert L.kvevict_paged_append(append(**a), None) == 0
        assert L.kvevict_paged_attention(attention(**a), None) == 0
    assert L.kvevict_paged_attention(attention(tokens=6, q_starts=4096, max_q=0), None) == 0
    assert L.kvevict_paged_gather(gather(rows=0), None) == 0 and L.kvevict_paged_gather(gather(batch=0), None) == 0
    for f in (L.kvevict_paged_append, L.kvevict_paged_attention, L.kvevict_paged_gather, L.kvevict_norm_rotary):
        assert f(None, None) == -1


N = dict(dtype=1, d=128, rd=128, il=0, inv=0, p64=1, hq=8, hk=2, batch=1, tokens=10, q=4096, k=4096, qo=4096, ko=4096, qs=(0, 128, 1024),
         qos=(0, 128, 1024), ks=(0, 128, 256), kos=(0, 128, 256), pos=0, ps=(0, 0), start=0, freq=4096, scale=1.0, wq=4096, wk=4096, eps=1e-6)


def norm(**kw):
    from kv_cache_eviction_decode_gb300 import ops
    vals = []
    for x in {**N, **kw}.values():
        vals += list(x) if isinstance(x, tuple) else [x]
    return ops._NORM.pack(*vals)


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(d=12), dict(rd=130), dict(rd=3), dict(rd=-2), dict(inv=1), dict(il=2), dict(freq=0), dict(freq=4100),
                                 dict(q=0), dict(qo=4104), dict(kos=(0, 0, 256)), dict(qs=(0, 130, 1024)), dict(wq=0), dict(wk=0), dict(wq=4104),
                                 dict(k=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("inf"))])
def test_norm_rotary_refused(L, bad):
    assert L.kvevict_norm_rotary(norm(**bad), None) == -1


def test_norm_rotary_nothing_to_do(L):
    assert L.kvevict_norm_rotary(norm(tokens=0), None) == 0 and L.kvevict_norm_rotary(norm(batch=0), None) == 0


# ------------------------------------------------------------------------------------------------- the binding
@pytest.fixture
def as_if_on_gpu(monkeypatch, L):
    """Lets the binding's checks see CPU tensors as the device's; what passes them all would launch, and stops here."""
    from kv_cache_eviction_decode_gb300 import ops, paged
    monkeypatch.setattr(ops, "_dtype", lambda t, name: ops._DT[t.dtype])

    def launch(*a):
        raise RuntimeError("launched")
    monkeypatch.setattr(ops, "_call", launch)
    monkeypatch.setattr(paged, "_call", launch)
    monkeypatch.setattr(ops, "_layouts", {})


def make(d=64, H=2, S=16, n=5, B=3, W=4, dtype=torch.bfloat16, four=False):
    import kv_cache_eviction_decode_gb300 as kv
    kp, vp = kv.paged_pool(n, H, S, d, dtype=dtype, four_bit=four, device="cpu")
    return kp, vp, torch.zeros(B, W, dtype=torch.int32), torch.ones(B, dtype=torch.int32)


@pytest.mark.parametrize("four", [False, True])
def test_accepted(as_if_on_gpu, four):
    import kv_cache_eviction_decode_gb300 as kv
    c = make(four=four)
    x, q = torch.zeros(6, 2, 64).bfloat16(), torch.zeros(6, 8, 64).bfloat16()
    starts, f = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    both = torch.zeros(5, 2, *c[0].shape[1:], dtype=c[0].dtype)
    for call in (lambda: kv.paged_append(x, x, *c), lambda: kv.paged_append(x[:5], x[:5], *c, starts=starts, inv_freq=f),
                 lambda: kv.paged_append(x[:1].expand(6, 2, 64), x, *c, inv_freq=f, positions=torch.zeros(6, dtype=torch.int64)),
                 lambda: kv.paged_append(x, x, both[:, 0], both[:, 1], *c[2:]),
                 lambda: kv.paged_gather(*c, max_k=9), lambda: kv.paged_gather(*c, k_starts=starts, rows=9),
                 lambda: kv.paged_attention(q, *c), lambda: kv.paged_attention(q[:5], *c, q_starts=starts, max_q=2**40, max_k=2**40),
                 lambda: kv.paged_attention(q, *c, n_sink=2**40, window=2**40, return_lse=True)):
        with pytest.raises(RuntimeError, match="launched"):
            call()


@pytest.mark.parametrize("four", [False, True])
def test_pages_refused_by_name(as_if_on_gpu, four):
    import kv_cache_eviction_decode_gb300 as kv
    kp, vp, table, lens = make(four=four)
    x, q = torch.zeros(6, 2, 64).bfloat16(), torch.zeros(6, 8, 64).bfloat16()
    ko = torch.zeros(3, 2, 9, 64).bfloat16()
    bad = [("v_pages", (kp, vp[:4], table, lens)), ("v_pages", (kp, vp.float(), table, lens)), ("k_pages", (kp[..., :-1], vp[..., :-1], table, lens)),
           ("k_pages", (kp[:, :, :8], vp[:, :, :8], table, lens)), ("k_pages", (kp[:, 0], vp[:, 0], table, lens)),
           ("k_pages", (kp.transpose(2, 3), vp, table, lens)), ("v_pages", (kp, vp[:, :1].expand(5, 2, 16, vp.shape[3]), table, lens)),
           ("block_table", (kp, vp, table.long(), lens)), ("block_table", (kp, vp, table[0], lens)), ("block_table", (kp, vp, table.t().contiguous().t(), lens)),
           ("block_table", (kp, vp, table[:, :1].expand(3, 2**26), lens)), ("kv_lens", (kp, vp, table, lens[:2])), ("kv_lens", (kp, vp, table, lens.long()))]
    if four:
        bad.append(("k_pages", (kp.transpose(1, 2).contiguous().transpose(1, 2), vp, table, lens)))
    for name, c in bad:
        for call in (lambda: kv.paged_append(x, x, *c), lambda: kv.paged_attention(q, *c), lambda: kv.paged_gather(*c, k_out=ko, v_out=ko)):
            with pytest.raises(ValueError, match=f"^{name}"):
                call()


def test_tokens_refused_by_name(as_if_on_gpu):
    import kv_cache_eviction_decode_gb300 as kv
    c = make()
    x, q, f = torch.zeros(6, 2, 64).bfloat16(), torch.zeros(6, 8, 64).bfloat16(), torch.zeros(32, dtype=torch.float64)
    starts = torch.zeros(4, dtype=torch.int32)
    w = torch.ones(64).bfloat16()
    odd = torch.zeros(6, 2, 67).bfloat16()[..., :64]
    for name, call in (("k", lambda: kv.paged_append(x[:5], x[:5], *c)), ("v", lambda: kv.paged_append(x, x[:5], *c)), ("k", lambda: kv.paged_append(odd, x, *c)),
                       ("k_pages", lambda: kv.paged_append(x[:, :1], x[:, :1], *c)), ("starts", lambda: kv.paged_append(x, x, *c, starts=starts[:3])),
                       ("inv_freq", lambda: kv.paged_append(x, x, *c, inv_freq=f.float())), ("inv_freq", lambda: kv.paged_append(x, x, *c, inv_freq=f.repeat(2))),
                       ("positions", lambda: kv.paged_append(x, x, *c, inv_freq=f, positions=starts)),
                       ("q", lambda: kv.paged_attention(q[:5], *c)), ("q", lambda: kv.paged_attention(q[:, :7], *c)),
                       ("q", lambda: kv.paged_attention(q[:, :1].expand(6, 8, 64), *c)), ("q_starts", lambda: kv.paged_attention(q, *c, q_starts=starts)),
                       ("window", lambda: kv.paged_attention(q, *c, window=0)), ("n_sink", lambda: kv.paged_attention(q, *c, n_sink=-1)),
                       ("max_q", lambda: kv.paged_attention(q, *c, max_k=-1)), ("out", lambda: kv.paged_attention(q, *c, out=q[:5])),
                       ("lse", lambda: kv.paged_attention(q, *c, lse=torch.zeros(6, 7))), ("scale", lambda: kv.paged_attention(q, *c, scale=0.0)),
                       ("k_out", lambda: kv.paged_gather(*c, k_out=torch.zeros(2, 2, 9, 64).bfloat16(), v_out=torch.zeros(2, 2, 9, 64).bfloat16())),
                       ("k_out", lambda: kv.paged_gather(*c, k_out=x)), ("paged_gather", lambda: kv.paged_gather(*c)),
                       ("k_starts", lambda: kv.paged_gather(*c, k_starts=starts[:2], rows=4)),
                       ("q_weight", lambda: kv.norm_rotary(q, None, w[:32], None)), ("k_weight", lambda: kv.norm_rotary(q, x, w, None)),
                       ("q_weight", lambda: kv.norm_rotary(q, None, w.float(), None)), ("eps", lambda: kv.norm_rotary(q, None, w, None, eps=-1.0)),
                       ("q_weight", lambda: kv.norm_rotary(q, None, torch.ones(65).bfloat16()[1:], None))):
        with pytest.raises(ValueError, match=f"^{name}"):
            call()


def test_gradients_refused(as_if_on_gpu):
    import kv_cache_eviction_decode_gb300 as kv
    c = make(dtype=torch.float32)
    x, q, w = torch.zeros(6, 2, 64), torch.zeros(6, 8, 64), torch.ones(64)

    def g(t):
        return t.clone().requires_grad_()
    for call in (lambda: kv.paged_append(g(x), x, *c), lambda: kv.paged_append(x, g(x), *c), lambda: kv.paged_append(x, x, g(c[0]), *c[1:]),
                 lambda: kv.paged_attention(g(q), *c), lambda: kv.paged_attention(q, c[0], g(c[1]), *c[2:]), lambda: kv.paged_gather(g(c[0]), *c[1:], max_k=3),
                 lambda: kv.norm_rotary(g(q), x, w, w), lambda: kv.norm_rotary(q, x, w, g(w))):
        with pytest.raises(ValueError, match="no backward"):
            call()
        with torch.no_grad(), pytest.raises(RuntimeError, match="launched"):
            call()


def test_pool_refused():
    import kv_cache_eviction_decode_gb300 as kv
    for a in ((4, 2, 24, 64), (4, 2, 16, 96), (4, 0, 16, 64), (-1, 2, 16, 64)):
        with pytest.raises(ValueError, match="paged_pool"):
            kv.paged_pool(*a, device="cpu")
    with pytest.raises(ValueError, match="paged_pool"):
        kv.paged_pool(4, 2, 16, 64, dtype=torch.float16, device="cpu")


# --------------------------------------------------------------------------- rows of new tokens, the kernels' own code
SRC = r"""
#include <cstdio>
#include <vector>
#include "paged_common.cuh"
using namespace kvevict;
// a line: batch, rows, then batch + 1 starts
int main()
{
    int batch, rows;
    while (std::scanf("%d %d", &batch, &rows) == 2) {
        std::vector<int> a(batch + 1);
        for (int &x : a) if (std::scanf("%d", &x) != 1) return 1;
        for (int b = 0; b < batch; ++b) {
            const PagedRows r = paged_rows(a.data(), b, 0, rows);
            std::printf("%d %d %d %d ", r.q0, r.n, r.given, r.bad ? 1 : 0);
        }
        std::printf("\n");
    }
}
"""


def test_rows_of_any_starts(tmp_path):
    """Whatever the starts: rows lie in the tensor, and those of ascending starts are disjoint."""
    (tmp_path / "s.cu").write_text(SRC)
    from kv_cache_eviction_decode_gb300 import build
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(tmp_path / "s.cu"), "-o", str(tmp_path / "s")],
                   check=True)
    r = random.Random(3)
    lines, cases = [], []
    for _ in range(500):
        rows, batch = r.choice([1, 7, 100]), r.randint(1, 6)
        a = [r.choice([0, 1, rows, r.randint(0, rows), r.randint(-5, rows + 5), 2**31 - 1, -2**31]) for _ in range(batch + 1)]
        if r.random() < 0.6:
            a.sort()
        cases.append((rows, a))
        lines.append(" ".join(map(str, [batch, rows, *a])))
    out = subprocess.run([str(tmp_path / "s")], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.strip().split("\n")
    for (rows, a), line in zip(cases, out):
        v = [int(x) for x in line.split()]
        end = 0
        for b in range(len(a) - 1):
            q0, n, given, bad = v[4 * b:4 * b + 4]
            assert 0 <= q0 <= rows and 0 <= n <= rows - q0 and given >= n
            good = 0 <= a[b] <= a[b + 1] <= rows
            assert bad == (not good) and (not good or (q0, n, given) == (a[b], a[b + 1] - a[b], n))
            if a == sorted(a):
                assert q0 >= end or n == 0
                end = max(end, q0 + n)
