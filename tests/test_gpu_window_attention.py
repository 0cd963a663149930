"""window_attention against the formula in 64 bits: types, head groups, head
sizes, lengths from nothing to long, masks that leave rows empty, strides,
padding that holds NaN, packed batches, other streams, capture."""
import math

import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(B, Hq, Hkv, n, m, d, dtype, seed=1):
    g = gen(seed)
    return (torch.randn(B, Hq, n, d, generator=g, device="cuda", dtype=dtype),
            torch.randn(B, Hkv, m, d, generator=g, device="cuda", dtype=dtype),
            torch.randn(B, Hkv, m, d, generator=g, device="cuda", dtype=dtype))


def check(q, k, v, out, lse, n_sink, window, q_lens=None, k_lens=None, scale=None):
    """Padded outputs, sequence by sequence."""
    scale = scale or 1 / math.sqrt(q.shape[-1])
    for b in range(q.shape[0]):
        n = q.shape[2] if q_lens is None else int(q_lens[b])
        m = k.shape[2] if k_lens is None else int(k_lens[b])
        r, l, A = ref.sequence(q[b, :, :n], k[b, :, :m], v[b, :, :m], n_sink, window, scale)
        tol, tol_l = ref.bounds(q.dtype, q[b, :, :n], k[b, :, :m], m, scale, r, A, l)
        ref.assert_close(out[b, :, :n], r, tol, f"out {b}")
        ref.assert_close(lse[b, :, :n], l, tol_l, f"lse {b}")


CASES = [
    # B, Hq, Hkv, n, m, d, n_sink, window
    (1, 1, 1, 1, 1, 64, 0, None),
    (2, 4, 4, 130, 130, 128, 4, 33),
    (1, 8, 2, 257, 257, 64, 4, 65),
    (2, 8, 1, 100, 300, 128, 0, None),        # a chunk at the end of a longer prompt
    (1, 3, 1, 300, 300, 64, 1, 128),          # a group of three
    (1, 5, 1, 129, 1000, 128, 130, 200),      # more sinks than a tile
    (1, 2, 2, 513, 513, 128, 0, 1),           # each token sees itself alone
    (1, 2, 2, 640, 640, 64, 600, 7),          # sinks that reach past most windows
    (3, 6, 2, 5, 777, 128, 4, 300),           # a few drafted tokens
    (2, 64, 8, 1, 4097, 128, 4, 2044),        # one token, many keys
    (2, 8, 8, 1, 3000, 64, 0, None),
    (1, 64, 1, 3, 900, 64, 2, 100),           # the widest group
    (1, 2, 1, 40, 17, 128, 4, 8),             # more queries than keys: the first rows see nothing
    (1, 17, 1, 33, 600, 64, 0, 512),          # a group that fits no tile evenly
    (2, 2, 2, 300, 0, 64, 0, None),           # no keys at all
    (1, 4, 4, 1500, 1500, 128, 4, None),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_forms(cuda_device, case, dtype):
    B, Hq, Hkv, n, m, d, n_sink, window = case
    q, k, v = make(B, Hq, Hkv, n, m, d, dtype)
    out, lse = kv.window_attention(q, k, v, n_sink=n_sink, window=window, return_lse=True)
    assert out.dtype == dtype and lse.dtype == torch.float32
    check(q, k, v, out, lse, n_sink, window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 200])
def test_lengths_on_the_device(cuda_device, n, dtype):
    """kv_lens and q_lens; what lies beyond them holds NaN and is neither read into results nor written."""
    B, Hq, Hkv, m, d = 4, 8, 2, 500, 128
    q, k, v = make(B, Hq, Hkv, n, m, d, dtype, 3)
    k_lens = [500, 133, 1, 0]
    q_lens = [n, max(0, n - 3), 1, n]
    for b in range(B):
        k[b, :, k_lens[b]:] = math.nan
        v[b, :, k_lens[b]:] = math.inf
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.window_attention(q, k, v, n_sink=4, window=100, out=out, lse=lse, error_word=err,
                        q_lens=torch.tensor(q_lens, dtype=torch.int32, device="cuda"),
                        kv_lens=torch.tensor(k_lens, dtype=torch.int32, device="cuda"))
    check(q, k, v, out, lse, 4, 100, q_lens, k_lens)
    for b in range(B):
        assert (out[b, :, q_lens[b]:] == 7).all() and (lse[b, :, q_lens[b]:] == 7).all()
    assert int(err) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_keys_nobody_sees_may_hold_anything(cuda_device, dtype):
    """Between the sinks and the window of a chunk's first query."""
    q, k, v = make(2, 4, 2, 3, 1000, 64, dtype, 5)
    k[:, :, 5:1000 - 102] = math.nan
    v[:, :, 5:1000 - 102] = math.nan
    out, lse = kv.window_attention(q, k, v, n_sink=5, window=100, return_lse=True)
    check(q, k, v, out, lse, 5, 100)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_packed(cuda_device, d, dtype):
    """Sequences of uneven lengths, empty ones among them, gaps before, between and behind; the rows outside are left as
    they were, and NaN there reaches nobody."""
    ql, kl = [130, 0, 1, 300, 5, 64], [130, 40, 700, 350, 0, 64]
    q0, k0, gap = 3, 2, 2
    qs, ks = [q0], [k0]
    for a, c in zip(ql, kl):
        qs.append(qs[-1] + a)
        ks.append(ks[-1] + c)
    Hq, Hkv = 6, 2
    g = gen(11)
    q = torch.randn(qs[-1] + gap, Hq, d, generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn(ks[-1] + gap, Hkv, d, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    for t, lo, hi in ((k, k0, ks[-1]), (v, k0, ks[-1])):
        t[:lo] = math.nan
        t[hi:] = math.nan
    k[ks[1]:ks[2]] = math.nan   # the keys of a sequence without queries
    v[ks[1]:ks[2]] = math.nan
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    starts = [torch.tensor(s, dtype=torch.int32, device="cuda") for s in (qs, ks)]
    kv.window_attention(q, k, v, n_sink=4, window=90, q_starts=starts[0], k_starts=starts[1], max_q=max(ql), max_k=max(kl),
                        out=out, lse=lse)
    for b, (n, m) in enumerate(zip(ql, kl)):
        qq, kk, vv = (x[s:s + w].transpose(0, 1) for x, s, w in ((q, qs[b], n), (k, ks[b], m), (v, ks[b], m)))
        if n == 0:
            continue
        r, l, A = ref.sequence(qq, kk, vv, 4, 90, d ** -0.5)
        tol, tol_l = ref.bounds(dtype, qq, kk, m, d ** -0.5, r, A, l)
        ref.assert_close(out[qs[b]:qs[b] + n].transpose(0, 1), r, tol, f"out {b}")
        ref.assert_close(lse[qs[b]:qs[b] + n].transpose(0, 1), l, tol_l, f"lse {b}")
    for t in (out, lse):
        assert (t[:q0] == 7).all() and (t[qs[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(cuda_device, dtype):
    """Token-major storage, heads of one fused tensor, an output inside a larger one."""
    B, H, Hkv, n, d = 2, 4, 2, 150, 64
    fused = torch.randn(B, n, H + 2 * Hkv, d, generator=gen(2), device="cuda", dtype=dtype)
    q, k, v = (fused[:, :, a:b].transpose(1, 2) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    big = torch.full((B, n, 2 * H, d), 7.0, device="cuda", dtype=dtype)
    out = big[:, :, 1:H + 1].transpose(1, 2)
    _, lse = kv.window_attention(q, k, v, n_sink=3, window=50, out=out, return_lse=True)
    check(q, k, v, out, lse, 3, 50)
    assert (big[:, :, 0] == 7).all() and (big[:, :, H + 1:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_equal_logits(cuda_device, dtype):
    """Logits far apart and far from zero (the running maximum moves by hundreds), and all equal."""
    q, k, v = make(1, 2, 2, 300, 700, 64, dtype, 9)
    q, k = (q * 8).contiguous(), k.clone()
    k *= torch.linspace(0.1, 6, 700, device="cuda").to(dtype)[None, None, :, None]
    out, lse = kv.window_attention(q, k, v, return_lse=True)
    check(q, k, v, out, lse, 0, None)
    k = torch.full_like(k, 0.5)
    out, lse = kv.window_attention(q, k, v, return_lse=True, scale=0.25)
    check(q, k, v, out, lse, 0, None, scale=0.25)


def test_masked_infinity_and_visible_nan(cuda_device):
    """An infinite key that a later query sees does not touch the earlier rows' logits; a visible NaN shows."""
    q, k, v = make(1, 1, 1, 64, 64, 64, torch.bfloat16, 4)
    k[0, 0, 40] = math.inf
    out, lse = kv.window_attention(q, k, v, return_lse=True)
    r, l, A = ref.sequence(q[0, :, :40], k[0, :, :40], v[0, :, :40], 0, None, 0.125)
    tol, tol_l = ref.bounds(q.dtype, q[0, :, :40], k[0, :, :40], 40, 0.125, r, A, l)
    ref.assert_close(out[0, :, :40], r, tol, "out")
    ref.assert_close(lse[0, :, :40], l, tol_l, "lse")
    q[0, 0, 50] = math.nan
    out = kv.window_attention(q, k, v)
    assert torch.isnan(out[0, 0, 50]).all() and not torch.isnan(out[0, 0, :40]).any()


@pytest.mark.parametrize("dtype", TYPES)
def test_lengths_out_of_range_are_clamped_and_flagged(cuda_device, dtype):
    q, k, v = make(3, 2, 2, 4, 50, 64, dtype, 6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([70, -5, 20], dtype=torch.int32, device="cuda")
    out, lse = kv.window_attention(q, k, v, kv_lens=lens, error_word=err, return_lse=True)
    check(q, k, v, out, lse, 0, None, None, [50, 0, 20])
    assert int(err) == 0x10


def test_two_streams_and_capture(cuda_device):
    """A split call (workspace and join) on another stream, two in flight at once, and captured ones replayed."""
    q, k, v = make(2, 8, 2, 1, 5000, 128, torch.bfloat16, 8)
    q2, k2, v2 = make(2, 8, 2, 1, 5000, 128, torch.bfloat16, 9)
    want, want2 = kv.window_attention(q, k, v), kv.window_attention(q2, k2, v2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = kv.window_attention(q, k, v)
        with torch.cuda.stream(s2):
            b = kv.window_attention(q2, k2, v2)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want) and torch.equal(b, want2)
    g = torch.cuda.CUDAGraph()
    x = q.clone()
    with torch.cuda.graph(g):
        y = kv.window_attention(x, k, v)
        z = kv.window_attention(y, k2, v2, n_sink=4, window=3000)
    x.copy_(q2)
    g.replay()
    assert torch.equal(y, kv.window_attention(q2, k, v))
    assert torch.equal(z, kv.window_attention(y, k2, v2, n_sink=4, window=3000))


@pytest.mark.parametrize("dtype", TYPES)
def test_same_call_same_bits(cuda_device, dtype):
    q, k, v = make(2, 8, 2, 3, 3000, 128, dtype, 10)
    a = kv.window_attention(q, k, v, n_sink=4, window=2000, return_lse=True)
    for _ in range(4):
        b = kv.window_attention(q, k, v, n_sink=4, window=2000, return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_bad_starts_are_clamped_and_flagged(cuda_device, dtype):
    """Starts that go back, or beyond the tensors, or a sequence above max_q: nothing outside is touched, the rows of the
    sound sequence are right, the error word says so."""
    g = gen(13)
    q = torch.randn(40, 4, 64, generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn(50, 2, 64, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    for qs, ks, max_q, good in (([0, 20, 10, 40], [0, 25, 25, 50], 40, 0), ([0, 20, 30, 99], [0, 20, 30, 99], 40, 1),
                                ([-7, 0, 20, 30], [-3, 0, 20, 30], 40, 1), ([0, 30, 40, 40], [0, 30, 50, 50], 20, 1)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 7.0)
        a, b = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qs, ks))
        kv.window_attention(q, k, v, q_starts=a, k_starts=b, max_q=max_q, max_k=50, out=out, error_word=err)
        assert int(err) == 0x10
        qq, kk, vv = (x[s[good]:s[good + 1]].transpose(0, 1) for x, s in ((q, qs), (k, ks), (v, ks)))
        r, l, A = ref.sequence(qq, kk, vv, 0, None, 0.125)
        tol, _ = ref.bounds(dtype, qq, kk, 50, 0.125, r, A, l)
        ref.assert_close(out[qs[good]:qs[good + 1]].transpose(0, 1), r, tol, "out")


def test_offsets_beyond_32_bits(cuda_device):
    """A cache of more than 2^31 elements: the last sequence's keys and the last head's."""
    B, Hkv, m, d = 70, 8, 30000, 128
    k, v = (torch.empty(B, Hkv, m, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = gen(17)
    assert k.numel() > 2**31
    q = torch.randn(B, 16, 1, d, generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = m
    for t in (k, v):
        t[-1].normal_(generator=g)
    out, lse = kv.window_attention(q, k, v, n_sink=4, window=3000, kv_lens=lens, return_lse=True)
    assert (out[:-1] == 0).all() and (lse[:-1] == -math.inf).all()
    check(q[-1:], k[-1:], v[-1:], out[-1:], lse[-1:], 4, 3000)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_short_sequences_and_one_long(cuda_device, dtype):
    """A packed batch in which nearly all row tiles that max_q allows are empty: tens of thousands for every SM."""
    B, n, H, d = 20000, 1500, 4, 64
    starts = torch.cat([torch.arange(B, dtype=torch.int32), torch.tensor([B - 1 + n], dtype=torch.int32)]).cuda()
    g = gen(37)
    q, k, v = (torch.randn(B - 1 + n, H, d, generator=g, device="cuda", dtype=dtype) for _ in range(3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kv.window_attention(q, k, v, n_sink=2, window=100, q_starts=starts, k_starts=starts, max_q=4096, max_k=n, error_word=err,
                                   return_lse=True)
    assert int(err) == 0
    assert torch.equal(out[:B - 1], v[:B - 1])  # one key: its probability is 1
    qq, kk, vv = (x[B - 1:].transpose(0, 1) for x in (q, k, v))
    r, l, A = ref.sequence(qq, kk, vv, 2, 100, 0.125)
    tol, tol_l = ref.bounds(dtype, qq, kk, n, 0.125, r, A, l)
    ref.assert_close(out[B - 1:].transpose(0, 1), r, tol, "out")
    ref.assert_close(lse[B - 1:].t(), l, tol_l, "lse")
