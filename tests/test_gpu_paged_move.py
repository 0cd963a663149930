"""paged_append and paged_gather. Keys that turn: the bounds of the tests of rotary; 4 bits: tests/paged_reference.py; all
else is a copy and has to be equal, the rows that no token goes to included."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests.paged_reference import Pool, check_groups, parts, unpack

pytestmark = pytest.mark.gpu
KINDS = [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True), (torch.float32, True)]


def turned(x, pos, f, interleaved, scale):
    """x [T][H][d] fp64, pos [T]: the result and |a| + |b| per element."""
    y, w = x.clone(), torch.zeros_like(x)
    if f is None:
        return y, w
    R = 2 * f.shape[0]
    t = pos.double()[:, None, None] * f
    c, s = torch.cos(t) * scale, torch.sin(t) * scale
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    w[..., a] = w[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(scale)
    return y, w


def run_append(new, lens, H, S, d, dtype, four, R=None, interleaved=False, scale=1.0, starts=True, positions=None, strides="dense", seed=0,
               strided_input=False):
    pool = Pool(lens, H, S, d, dtype, four, seed=seed, strides=strides)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = sum(new)
    if strided_input:
        fused = torch.randn(T, 2 * H + 3, d, generator=g, device="cuda", dtype=dtype)
        k, v = fused[:, 1:1 + H], fused[:, 2 + H:2 + 2 * H]
    else:
        k, v = (torch.randn(T, H, d, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    f = kv.rotary_frequencies(R)[0] if R else None
    before = pool.k.clone(), pool.v.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.paged_append(k, v, pool.k, pool.v, pool.table, pool.kv_lens, starts=torch.tensor(at, dtype=torch.int32, device="cuda") if starts else None,
                    inv_freq=f, positions=positions, interleaved=interleaved, scale=scale, error_word=err)
    assert int(err) == 0
    place = torch.tensor([(b, m - n + i) for b, (n, m) in enumerate(zip(new, lens)) for i in range(n)], device="cuda").reshape(-1, 2)
    page, slot = pool.table[place[:, 0], place[:, 1] // S].long(), place[:, 1] % S
    pos = place[:, 1] if positions is None else positions
    for which, (pages, x) in enumerate(((pool.k, k), (pool.v, v))):
        y, w = turned(x.double(), pos, f if which == 0 else None, interleaved, scale)
        slack = 2.0 ** -20 * w
        if four:
            codes, params = parts(pages, d)
            check_groups(y.flatten(0, 1), slack.flatten(0, 1), unpack(codes[page, :, slot]).flatten(0, 1), params[page, :, slot].flatten(0, 1))
            old_c, old_p = parts(before[which], d)
            old_c[page, :, slot], old_p[page, :, slot] = codes[page, :, slot], params[page, :, slot]
        else:
            got = pages[page, :, slot].double()
            tol = slack + (torch.finfo(dtype).eps / 2 * y.abs() if which == 0 and f is not None else 0)
            assert ((got - y).abs() <= tol * 1.0001).all()
            before[which][page, :, slot] = pages[page, :, slot]
        assert torch.equal(before[which].view(torch.uint8), pages.contiguous().view(torch.uint8))  # nothing else was written
    return pool


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("d,R,interleaved", [(128, 128, False), (64, 64, False), (128, 48, False), (64, 10, False), (128, None, False),
                                             (128, 128, True), (64, 6, True), (64, 24, True)])
def test_append_layouts(cuda_device, d, R, interleaved, dtype, four):
    run_append([5, 0, 1, 33, 7], [5, 40, 1, 70, 129], 3, 16, d, dtype, four, R, interleaved, scale=1.25 if R else 1.0)


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("new,lens,H,S", [([1], [1], 1, 16), ([1] * 64, list(range(1, 65)), 8, 16), ([3] * 5, [3, 16, 17, 31, 500], 5, 32),
                                          ([300, 1], [300, 1000], 2, 256), ([1], [4097], 64, 64), ([1000], [1000], 1, 128)])
def test_append_sizes(cuda_device, new, lens, H, S, dtype, four):
    run_append(new, lens, H, S, 128, dtype, four, 128)
    if len(set(new)) == 1:
        run_append(new, lens, H, S, 64, dtype, four, 64, starts=False)


@pytest.mark.parametrize("dtype,four", KINDS)
def test_append_strides_and_positions(cuda_device, dtype, four):
    pos = torch.randint(-1000, 100000, (46,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    new, lens = [5, 0, 1, 33, 7], [5, 40, 1, 70, 129]
    run_append(new, lens, 3, 16, 128, dtype, four, 128, positions=pos, strides="joint", strided_input=True)
    run_append(new, lens, 3, 32, 64, dtype, four, 64, positions=pos.int(), strides="tokens", strided_input=True)
    run_append(new, lens, 1, 16, 64, dtype, four, 64, positions=pos.repeat(2)[::2])


def test_append_what_four_bits_cannot_hold(cuda_device):
    """Constant groups are exact where bf16 is; a group with an infinity or NaN stands for NaN, its neighbours do not."""
    pool = Pool([16], 2, 16, 64, torch.float32, True, garbage=False)
    k = torch.zeros(16, 2, 64, device="cuda")
    k[0] = 1.5
    k[1, 0, :32], k[2, 1, 40] = 1e30, float("inf")
    k[3, 0, 5], k[4, 1, 63] = float("nan"), float("-inf")
    k[5, 0] = 1 + 2.0 ** -12  # (no bf16)
    k[6, 0, ::2] = -1e-30
    kv.paged_append(k, k, pool.k, pool.v, pool.table, pool.kv_lens)
    for pages in (pool.k, pool.v):
        got = pool.rows(0, 16, 0 if pages is pool.k else 1)[0].transpose(0, 1)
        bad = torch.zeros(16, 2, 64, dtype=torch.bool, device="cuda")
        bad[2, 1, 32:] = bad[3, 0, :32] = bad[4, 1, 32:] = True
        assert torch.equal(torch.isnan(got), bad)
        assert (got[0] == 1.5).all() and ((got[1, 0, :32] / 1e30 - 1).abs() < 2.0 ** -7).all() and (got[1, 0, 32:] == 0).all()
        assert ((got[5, 0] - 1).abs() <= 2.0 ** -12 * (1 + 2.0 ** -7)).all() and ((got[6, 0] - k[6, 0].double()).abs() <= 1e-31).all()


@pytest.mark.parametrize("d", [64, 128])
def test_append_rounds_ties_to_even(cuda_device, d):
    """bf16 channels over steps in bf16 often lie just between two codes, and steps often need no rounding. Every code that
    64 bits put at k + 1/2 is the even one, all others the nearest but within 2^-18 of a border; the step is the least that
    bf16 has, wherever 64 bits are not within 2^-18 of the one below it; and the base is the nearest (8 hi + 7 lo is exact in
    fp32 here, and its fifteenth put right once)."""
    T, H = 512, 4
    pool = Pool([T], H, 16, d, torch.bfloat16, True, garbage=False)
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(T, H, d, device="cuda", generator=g)
    x = torch.stack([x, torch.round(x * 8) / 8])[torch.arange(T, device="cuda") % 2, torch.arange(T, device="cuda")].bfloat16()  # half of them on a grid
    kv.paged_append(x, x, pool.k, pool.v, pool.table, pool.kv_lens)
    ties = 0
    for pages in (pool.k, pool.v):
        codes, params = parts(pages, d)
        page, slot = pool.table[0, torch.arange(T, device="cuda") // 16].long(), torch.arange(T, device="cuda") % 16
        c = unpack(codes[page, :, slot]).double().unflatten(-1, (-1, 32))
        base, step = (params[page, :, slot][..., i].double()[..., None] for i in (0, 1))
        z = x.double().unflatten(-1, (-1, 32))
        q = (z - base) / step
        near = torch.round(q).clamp(-8, 7)
        tie = (q - q.floor() == 0.5) & (q > -8) & (q < 7)
        ties += int(tie.sum())
        assert torch.equal(c[tie] - 8, near[tie])
        assert ((c - 8 == near) | ((q - q.floor() - 0.5).abs() < 2.0 ** -18)).all()
        exact = ((8 * z.amax(-1, keepdim=True) + 7 * z.amin(-1, keepdim=True)) / 15).bfloat16().double()
        assert torch.equal(base, exact)
        need = torch.maximum((z.amax(-1, keepdim=True) - base) / 7, (base - z.amin(-1, keepdim=True)) / 8)
        below = (params[page, :, slot][..., 1].contiguous().view(torch.int16) - 1).view(torch.bfloat16).double()[..., None]
        assert (below < need * (1 + 2.0 ** -18)).all() and (step >= need * (1 - 2.0 ** -18)).all()
    assert ties > 1000


@pytest.mark.parametrize("dtype,four", KINDS)
@pytest.mark.parametrize("d,S,H", [(128, 16, 8), (64, 32, 3), (128, 256, 1)])
@pytest.mark.parametrize("lens", [[1], [0, 17, 64, 200, 1], [129, 0, 0, 65]])
def test_gather(cuda_device, lens, d, S, H, dtype, four):
    for strides in ("dense", "joint", "tokens"):
        pool = Pool(lens, H, S, d, dtype, four, seed=7, strides=strides)
        starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        M = max(lens) + 5
        for packed in (False, True):
            shape = (sum(lens) + 3, H, d) if packed else (len(lens), H, M, d)
            out = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(2)]
            kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_starts=starts if packed else None, k_out=out[0], v_out=out[1], error_word=err)
            for which, got in enumerate(out):
                for b, m in enumerate(lens):
                    mine = got[int(starts[b]):int(starts[b]) + m].transpose(0, 1) if packed else got[b, :, :m]
                    want = pool.rows(b, m, which)[0]
                    if four:  # rounded to fp32, then (bf16) again: half a step, and fp32's in front of it
                        tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -23) * want.abs()
                        assert ((mine.double() - want).abs() <= tol).all()
                    else:
                        assert torch.equal(mine.double(), want)
                    if not packed:
                        assert (got[b, :, m:] == 7).all()
                if packed:
                    assert (got[sum(lens):] == 7).all()
        assert int(err) == 0


def test_gather_makes_its_outputs(cuda_device):
    pool = Pool([30, 9], 2, 16, 64, torch.bfloat16, True)
    k, v = kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, max_k=30)
    assert k.shape == (2, 2, 30, 64) and k.dtype == torch.bfloat16
    k32, _ = kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, max_k=30, dtype=torch.float32)
    assert torch.equal(k32[0].bfloat16(), k[0]) and torch.equal(k32[0].double(), pool.rows(0, 30, 0)[0].float().double())
    starts = torch.tensor([0, 30, 39], dtype=torch.int32, device="cuda")
    kp, vp = kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_starts=starts, rows=39)
    assert torch.equal(kp[30:], k[1, :, :9].transpose(0, 1)) and torch.equal(vp[:30], v[0].transpose(0, 1))
    assert kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, max_k=0)[0].shape == (2, 2, 0, 64)


@pytest.mark.parametrize("four", [False, True])
def test_append_bad_places(cuda_device, four):
    """Lengths that put a token before the first place or behind the table, entries that are no pages: those tokens are
    dropped and the bits set; the others are written."""
    H, S, d = 2, 16, 64
    pool = Pool([40, 20, 33], H, S, d, torch.bfloat16, four, garbage=False)
    k = torch.randn(9, H, d, device="cuda", dtype=torch.bfloat16)
    for lens, bad_entry, bits in (([40, 2, 33], False, 0x10), ([40, 20, pool.width * S + 1], False, 0x10), ([40, -5, 33], False, 0x10),
                                  ([40, 2**31 - 1, 33], False, 0x10), ([40, 20, 33], True, 0x20)):
        table = pool.table.clone()
        if bad_entry:
            table[1, 1] = pool.k.shape[0]
        a, b = pool.k.clone(), pool.v.clone()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv.paged_append(k, k, a, b, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), error_word=err)
        assert int(err) == bits, (lens, int(err))
        # the same calls one sequence at a time, the sound tokens only
        want_k, want_v = pool.k.clone(), pool.v.clone()
        for s in range(3):
            for i in range(3):
                at = lens[s] - 3 + i
                if 0 <= at < pool.width * S and 0 <= int(table[s, at // S]) < pool.k.shape[0]:
                    kv.paged_append(k[3 * s + i:3 * s + i + 1], k[3 * s + i:3 * s + i + 1], want_k, want_v, table[s:s + 1],
                                    torch.tensor([at + 1], dtype=torch.int32, device="cuda"))
        assert torch.equal(a.view(torch.uint8), want_k.view(torch.uint8)) and torch.equal(b.view(torch.uint8), want_v.view(torch.uint8))


@pytest.mark.parametrize("starts,whole", [([0, 4, 2, 3, 8], 1), ([0, 2, 5, 1, 9], 2), ([3, 1, 2, 4, 8], 0), ([-2, 3, 5, 7, 20], 4)])
def test_append_and_gather_starts_out_of_order(cuda_device, starts, whole):
    """From the first sequence that ends before it starts the batch is left out; starts out of range are clamped."""
    T, H, S, d = 9, 2, 16, 64
    lens = [20, 30, 25, 40]
    pool = Pool(lens, H, S, d, torch.float32, False, garbage=False)
    k = torch.randn(T, H, d, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = pool.k.clone()
    for b in range(whole):
        q0 = min(max(starts[b], 0), T)
        given = max(starts[b + 1], q0) - q0
        for i in range(min(given, T - q0)):
            at = lens[b] - given + i
            if at >= 0:
                want[int(pool.table[b, at // S]), :, at % S] = k[q0 + i]
    kv.paged_append(k, k, pool.k, pool.v, pool.table, pool.kv_lens, starts=st, error_word=err)
    assert int(err[0]) == 0x10 and torch.equal(pool.k, want)
    out = [torch.full((T, H, d), 7.0, device="cuda") for _ in range(2)]
    kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_starts=st, k_out=out[0], v_out=out[1], error_word=err[1:])
    want = torch.full((T, H, d), 7.0, device="cuda")
    for b in range(whole):
        q0 = min(max(starts[b], 0), T)
        n = min(max(starts[b + 1], q0) - q0, T - q0, lens[b])
        want[q0:q0 + n] = pool.rows(b, lens[b], 0)[0][:, :n].transpose(0, 1).float()
    assert int(err[1]) == 0x10 and torch.equal(out[0], want)


def test_gather_bad_lengths_and_pages(cuda_device):
    pool = Pool([40, 20], 2, 16, 64, torch.float32, False, garbage=False, width=4)
    for lens, M, bits, n in (([41, 20], 40, 0x10, [40, 20]), ([-3, 20], 40, 0x10, [0, 20]), ([40, 2**31 - 1], 20, 0x10, [20, 20])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((2, 2, M, 64), 7.0, device="cuda"), torch.empty(2, 2, M, 64, device="cuda")
        kv.paged_gather(pool.k, pool.v, pool.table, torch.tensor(lens, dtype=torch.int32, device="cuda"), k_out=out[0], v_out=out[1], error_word=err)
        assert int(err) == bits
        for b in range(2):
            assert torch.equal(out[0][b, :, :n[b]].double(), pool.rows(b, n[b], 0)[0]) and (out[0][b, :, n[b]:] == 7).all()
    table = pool.table.clone()
    table[0, 1] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((2, 2, 40, 64), 7.0, device="cuda"), torch.empty(2, 2, 40, 64, device="cuda")
    kv.paged_gather(pool.k, pool.v, table, pool.kv_lens, k_out=out[0], v_out=out[1], error_word=err)
    assert int(err) == 0x20 and (out[0][0, :, 16:32] == 7).all() and torch.equal(out[0][0, :, 32:].double(), pool.rows(0, 40, 0)[0][:, 32:])
    # without a word of its own the bits are the device's
    kv.operator_errors()
    kv.paged_gather(pool.k, pool.v, table, pool.kv_lens, k_out=out[0], v_out=out[1])
    assert kv.operator_errors() == 0x20 and kv.operator_errors() == 0


def test_capture_reads_lengths_anew(cuda_device):
    """A captured append and gather follow the lengths and tables that a replay finds."""
    pool = Pool([20, 30], 2, 16, 128, torch.bfloat16, True, garbage=False, width=4)
    k = torch.randn(2, 2, 128, device="cuda", dtype=torch.bfloat16)
    f, _ = kv.rotary_frequencies(128)
    out = [torch.zeros(2, 2, 40, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kv.paged_append(k, k, pool.k, pool.v, pool.table, pool.kv_lens, inv_freq=f)
        kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_out=out[0], v_out=out[1])
    for _ in range(3):
        want = pool.k.clone(), pool.v.clone()
        k.normal_()
        kv.paged_append(k, k, *want, pool.table, pool.kv_lens, inv_freq=f)
        g.replay()
        assert torch.equal(pool.k, want[0]) and torch.equal(pool.v, want[1])
        for b in range(2):
            m = int(pool.kv_lens[b])
            w = pool.rows(b, m, 0)[0]
            assert ((out[0][b, :, :m].double() - w).abs() <= (2.0 ** -8 + 2.0 ** -23) * w.abs()).all()
        pool.kv_lens += 1


def test_offsets_beyond_32_bits(cuda_device):
    """Pages more than 2^31 elements apart."""
    S, d = 16, 64
    big = torch.empty(5 * 2**29 + 4096, device="cuda", dtype=torch.bfloat16)
    kp, vp = (big[o:].as_strided((3, 2, S, d), (5 * 2**28 - 64, S * d, d, 1)) for o in (0, 2048))
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 16], dtype=torch.int32, device="cuda")
    kp.zero_(), vp.zero_()
    k, v = (torch.randn(32, 2, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kv.paged_append(k, v, kp, vp, table, lens + 0 * lens, starts=torch.tensor([0, 16, 32], dtype=torch.int32, device="cuda"))
    got = kv.paged_gather(kp, vp, table, lens, max_k=20)
    for x, y in zip((k, v), got):
        assert torch.equal(y[0, :, 4:], x[:16].transpose(0, 1)) and torch.equal(y[1, :, :16], x[16:].transpose(0, 1))
        assert (y[0, :, :4] == 0).all()
