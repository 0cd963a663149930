"""paged_attention against attention in 64 bits over the values that the pages hold, with the bounds derived in
tests/attn_reference.py and tests/paged_reference.py."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref
from tests.paged_reference import Pool, attention_bounds, parts

pytestmark = pytest.mark.gpu
KINDS = [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True), (torch.float32, True)]


def starts_of(new):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def check_sequence(pool, b, q, out, lse, m, n_sink, window, scale, n_given=None):
    """q, out [n][Hq][d], lse [n][Hq] of the first n of n_given new tokens at the end of m keys of sequence b."""
    n, Hq, d = q.shape
    n_given = n if n_given is None else n_given
    G = Hq // pool.H
    k, ks, kst = pool.rows(b, m, 0)
    v, vs, vst = pool.rows(b, m, 1)
    see = ref.visible(n_given, m, n_sink, window, q.device)[:n]
    some = see.any(0)[None, :, None]

    def clean(x):
        return torch.where(some, x, torch.zeros_like(x)).repeat_interleave(G, 0)
    qq = q.double().transpose(0, 1)
    r, l, _ = ref.rows(qq, clean(k), clean(v), see, scale)
    z = (qq @ clean(k).transpose(1, 2) * scale).masked_fill(~see, -float("inf"))
    p = torch.softmax(z, -1).nan_to_num(0) if m else z
    A = p @ clean(vs)
    A_step = p @ clean(vst) if pool.four else None
    tol, tol_l = attention_bounds(q.dtype, pool.four, qq, clean(k), clean(ks), clean(kst) if pool.four else None, A, A_step, m, scale, r, l)
    ref.assert_close(out.transpose(0, 1), r, tol, "out")
    ref.assert_close(lse.transpose(0, 1), l, tol_l, "lse")


def run(new, lens, Hq, H, S, d, dtype, four, n_sink=0, window=None, scale=None, uniform=False, strides="dense", seed=0, width=None, max_k=None,
        strided=False, spread=1.0):
    pool = Pool(lens, H, S, d, dtype, four, seed=seed, strides=strides, width=width)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = sum(new)
    if strided:
        fused = torch.randn(T + 1, Hq + 3, d, generator=g, device="cuda", dtype=dtype)
        q, out = fused[:T, 1:1 + Hq], torch.full((T, Hq + 2, d), 7.0, device="cuda", dtype=dtype)[:, 1:1 + Hq]
    else:
        q, out = torch.randn(T, Hq, d, generator=g, device="cuda", dtype=dtype) * spread, torch.full((T, Hq, d), 7.0, device="cuda", dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    kw = dict(n_sink=n_sink, window=window, scale=scale, max_k=max_k, error_word=err,
              **({} if uniform else dict(q_starts=starts_of(new), max_q=max(new))))
    kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, out=out, lse=lse, **kw)
    assert int(err) == 0
    at = 0
    for b, (n, m) in enumerate(zip(new, lens)):
        check_sequence(pool, b, q[at:at + n], out[at:at + n], lse[at:at + n], m, n_sink, window, scale or d ** -0.5)
        at += n
    again = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True, **kw)  # the same bits, into outputs of its own
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    return pool, q, out, lse


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (8, 4), (6, 2), (10, 2), (16, 2), (24, 2), (64, 1), (40, 5)])
def test_heads(cuda_device, Hq, H, d, dtype, four):
    run([1] * 4, [1, 16, 17, 300], Hq, H, 16, d, dtype, four, uniform=True)


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2, 15, 31, 33, 63, 64, 65], [0, 129, 257, 1000], [4099]])
def test_lengths_and_pages(cuda_device, lens, S, dtype, four):
    run([1] * len(lens), lens, 8, 2, S, 128, dtype, four, uniform=True)
    run([1 if m else 0 for m in lens], lens, 4, 2, S, 64, dtype, four)


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("n_sink,window", [(0, 1), (0, 16), (4, 17), (20, 100), (5, 1000), (1000, 3), (0, None), (3, None), (33, 2)])
def test_masks(cuda_device, n_sink, window, dtype, four):
    """Several tokens of every sequence: each row has its own end and window."""
    run([3, 0, 7, 1, 5], [3, 40, 130, 1, 777], 8, 2, 16, 64, dtype, four, n_sink, window)
    run([5, 5, 5], [5, 333, 600], 12, 4, 32, 128, dtype, four, n_sink, window, uniform=True, seed=3)


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("new,lens", [([40], [40]), ([1, 70, 2], [500, 70, 9]), ([130], [400]), ([9, 0, 33], [10, 0, 100])])
def test_many_tokens(cuda_device, new, lens, dtype, four):
    run(new, lens, 8, 2, 16, 128, dtype, four)
    run(new, lens, 6, 2, 64, 64, dtype, four, 2, 30)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_more_tokens_than_keys(cuda_device, dtype, four):
    """Rows before the first key see nothing: 0 and -infinity."""
    for H, Hq in ((2, 4), (1, 8)):
        pool, q, out, lse = run([4, 20, 3], [2, 5, 0], Hq, H, 16, 64, dtype, four)
        assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all() and (out[24:] == 0).all()


@pytest.mark.parametrize("dtype,four", KINDS)
def test_long(cuda_device, dtype, four):
    """Keys split over CTAs, of uneven sequences; wide tables of which little is used."""
    run([1, 1, 1], [20000, 7, 9001], 8, 1, 16, 128, dtype, four, uniform=True)
    run([2, 1, 3], [20000, 1, 4], 4, 2, 128, 64, dtype, four, 4, 5000)
    run([1], [300], 8, 8, 16, 64, dtype, four, uniform=True, width=5000)
    run([1], [300], 8, 8, 16, 64, dtype, four, uniform=True, width=5000, max_k=300)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_strides_scale_and_large_logits(cuda_device, dtype, four):
    run([3, 2], [100, 50], 6, 3, 16, 64, dtype, four, strides="joint", strided=True, scale=0.3)
    run([3, 2], [100, 50], 6, 3, 32, 128, dtype, four, strides="tokens", strided=True)
    run([1, 1], [1000, 50], 8, 2, 16, 128, dtype, four, spread=30.0, uniform=True)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_what_nobody_sees_may_hold_anything(cuda_device, dtype, four):
    """Infinities and NaN between the sinks and the window and behind the end (and, 4 bits, in front of one row's window that
    another row still sees)."""
    n_sink, window, lens, new = 3, 20, [200, 90], [1, 1]
    pool = Pool(lens, 2, 16, 64, dtype, four)
    for b, m in enumerate(lens):
        for i in range(n_sink, m - window):
            pool.spoil(b, i)
        table = pool.table[b]
        for j in range(1, (m - window) // 16):  # pages of which no key is seen need not be there
            table[j] = -1
    q = torch.randn(2, 4, 64, device="cuda", dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, n_sink=n_sink, window=window, return_lse=True, error_word=err)
    assert int(err) == 0
    pool.table.clamp_(min=0)
    for b, m in enumerate(lens):
        check_sequence(pool, b, q[b:b + 1], out[b:b + 1], lse[b:b + 1], m, n_sink, window, 64 ** -0.5)


def test_nan_within_one_rows_view_of_four_bits(cuda_device):
    """Two tokens with a window of 1: what the first one's only key holds does not reach the second."""
    pool = Pool([40], 1, 16, 64, torch.bfloat16, True)
    pool.spoil(0, 38)
    q = torch.randn(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    out = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, window=1)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("dtype,four", KINDS)
def test_bad_pages_and_lengths(cuda_device, dtype, four):
    pool = Pool([100, 60, 200], 2, 16, 64, dtype, four, garbage=False, width=13)
    q = torch.randn(3, 4, 64, device="cuda", dtype=dtype)
    good = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True)
    for what, bits in (("page", 0x20), ("long", 0x10), ("negative", 0x10)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        table, lens = pool.table.clone(), pool.kv_lens.clone()
        if what == "page":
            table[1, 2] = pool.k.shape[0]
        else:
            lens[1] = -3 if what == "negative" else 2**31 - 1
            table[1, 4:] = table[1, 0]
        out, lse = kv.paged_attention(q, pool.k, pool.v, table, lens, return_lse=True, error_word=err)
        assert int(err) == bits
        for b in (0, 2):
            assert torch.equal(out[b], good[0][b]) and torch.equal(lse[b], good[1][b])
        if what == "negative":
            assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
        else:
            assert torch.isfinite(out[1]).all()
    # without the page: the softmax over the other keys
    table = pool.table.clone()
    table[1, 2] = -1
    out, lse = kv.paged_attention(q, pool.k, pool.v, table, pool.kv_lens, return_lse=True)
    assert kv.operator_errors() == 0x20
    rest = torch.tensor([i for i in range(60) if not 32 <= i < 48], device="cuda")
    k, v = (pool.rows(1, 60, w)[0][:, rest].repeat_interleave(2, 0) for w in (0, 1))
    see = torch.ones(1, len(rest), dtype=torch.bool, device="cuda")
    r, l, A = ref.rows(q[1].double()[:, None], k, v, see, 64 ** -0.5)
    assert ((out[1].double()[:, None] - r).abs() <= 0.02 * A + 0.01).all() and ((lse[1].double()[:, None] - l).abs() < 1e-2).all()


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("starts,whole", [([0, 4, 2, 3, 8], 1), ([0, 2, 5, 1, 9], 2), ([3, 1, 2, 4, 8], 0), ([0, 2, 4, 6, 20], 4)])
def test_starts_out_of_order(cuda_device, starts, whole, dtype, four):
    lens, T = [2000, 30, 25, 40], 9
    pool = Pool(lens, 2, 16, 64, dtype, four)
    q = torch.randn(T, 4, 64, device="cuda", dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((T, 4), 7.0, device="cuda")
    kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_q=T, out=out,
                       lse=lse, error_word=err)
    assert int(err) == 0x10
    done = torch.zeros(T, dtype=torch.bool, device="cuda")
    for b in range(whole):
        n = min(starts[b + 1], T) - starts[b]
        rows = slice(starts[b], starts[b] + n)
        check_sequence(pool, b, q[rows], out[rows], lse[rows], lens[b], 0, None, 64 ** -0.5, starts[b + 1] - starts[b])
        done[rows] = True
    assert (out[~done] == 7).all() and (lse[~done] == 7).all()


def test_more_tokens_than_max_q(cuda_device):
    pool = Pool([50, 60], 2, 16, 64, torch.bfloat16, True)
    q = torch.randn(7, 4, 64, device="cuda", dtype=torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((7, 4), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, q_starts=starts_of([5, 2]), max_q=3, out=out, lse=lse, error_word=err)
    assert int(err) == 0x10 and (out[3:5] == 7).all()
    check_sequence(pool, 0, q[:3], out[:3], lse[:3], 50, 0, None, 64 ** -0.5, 5)
    check_sequence(pool, 1, q[5:], out[5:], lse[5:], 60, 0, None, 64 ** -0.5)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_capture_streams_and_workspaces(cuda_device, dtype, four):
    """Captured with a workspace of its own, replayed while an eager call runs on another stream; lengths read anew."""
    pool = Pool([3000, 900], 1, 16, 128, dtype, four, garbage=False, width=200)
    q = torch.randn(2, 8, 128, device="cuda", dtype=dtype)
    kw = dict(return_lse=True)
    want = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, **kw)
    torch.cuda.synchronize()
    for _ in range(5):
        g.replay()
        with torch.cuda.stream(side):
            other = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, **kw)
        torch.cuda.synchronize()
        for a, b in ((out, want[0]), (lse, want[1]), (other[0], want[0]), (other[1], want[1])):
            assert torch.equal(a, b)
        out.zero_()
    pool.kv_lens.copy_(torch.tensor([2990, 2], device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    for b, m in enumerate((2990, 2)):
        check_sequence(pool, b, q[b:b + 1], out[b:b + 1], lse[b:b + 1], m, 0, None, 128 ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size_in_four_bits(cuda_device, d):
    """V's groups far from one: small, large, and growing or falling by 2^40 from tile to tile of one sequence."""
    for scale in ([2.0 ** -40], [2.0 ** 50], [2.0 ** -20, 2.0 ** 20], [2.0 ** 30, 2.0 ** -10], [2.0 ** -15, 1.0, 2.0 ** 15, 0.0]):
        pool = Pool([400, 60], 2, 16, d, torch.bfloat16, True, seed=5)
        _, params = parts(pool.v, d)
        for b in range(2):
            for j in range(-(-pool.lens[b] // 16)):
                params[int(pool.table[b, j])] *= scale[j % len(scale)]
        q = torch.randn(2, 8, d, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(6))
        out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True)
        for b, m in enumerate(pool.lens):
            check_sequence(pool, b, q[b:b + 1], out[b:b + 1], lse[b:b + 1], m, 0, None, d ** -0.5)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_no_pages_at_all(cuda_device, dtype, four):
    """A cache without pages: every key is in none, and nothing is read."""
    k, v = kv.paged_pool(0, 2, 16, 64, dtype=dtype, four_bit=four)
    table, lens = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kv.paged_attention(torch.ones(1, 4, 64, device="cuda", dtype=dtype), k, v, table, lens, return_lse=True, error_word=err)
    assert (out == 0).all() and (lse == -float("inf")).all() and int(err) == 0x20


def test_nothing_to_do(cuda_device):
    pool = Pool([50], 2, 16, 64, torch.bfloat16, True)
    q = torch.randn(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    assert kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens).shape == (0, 4, 64)
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    assert kv.paged_attention(q, pool.k, pool.v, none, none[:, 0]).shape == (0, 4, 64)
    # a table without places: nothing is seen
    out, lse = kv.paged_attention(q.new_zeros(1, 4, 64), pool.k, pool.v, pool.table[:, :0], torch.zeros_like(pool.kv_lens), return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_offsets_beyond_32_bits(cuda_device):
    S, d = 16, 64
    big = torch.empty(5 * 2**29 + 4096, device="cuda", dtype=torch.bfloat16)
    kp, vp = (big[o:].as_strided((3, 2, S, d), (5 * 2**28 - 64, S * d, d, 1)) for o in (0, 2048))
    kp.normal_(), vp.normal_()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([45], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    near = kv.paged_attention(q, kp[[2, 0, 1]].contiguous(), vp[[2, 0, 1]].contiguous(), torch.arange(3, device="cuda", dtype=torch.int32)[None], lens)
    assert torch.equal(kv.paged_attention(q, kp, vp, table, lens), near)
