"""rotary against the formula in 64 bits. The kernel's angle is exact to far
below an fp32 step of the result; cosine, sine (a step or two each) and the
three fp32 operations leave |err| <= 2^-20 (|a| + |b|) scale + half a step of
the output."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def formula(x, pos, f, interleaved, scale, inverse, R):
    """x [B][H][N][d] fp64, pos [B][N]: the result and |a| + |b| per element."""
    t = pos.double()[:, None, :, None] * f
    if inverse:
        t = -t
    c, s = torch.cos(t) * scale, torch.sin(t) * scale
    y, w = x.clone(), x.abs() * 0
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    xa, xb = x[..., a], x[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    w[..., a] = w[..., b] = (xa.abs() + xb.abs()) * abs(scale)
    return y, w


def check(got, x, pos, f, interleaved, scale, inverse):
    R = 2 * f.shape[0]
    y, w = formula(x.double(), pos, f, interleaved, scale, inverse, R)
    tol = 2.0 ** -20 * w + torch.finfo(x.dtype).eps / 2 * y.abs()
    err = (got.double() - y).abs()
    assert (err <= tol * 1.0001).all(), float((err / tol.clamp_min(1e-300)).max())
    assert torch.equal(got[..., R:], x[..., R:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R", [(128, 128), (64, 64), (128, 64), (128, 48), (64, 10), (128, 2), (72, 72), (256, 24), (8, 6)])
def test_layouts(cuda_device, d, R, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(d + R)
    B, Hq, Hk, N = 2, 5, 3, 37
    q = torch.randn(B, Hq, N, d, generator=g, device="cuda", dtype=dtype)
    k = torch.randn(B, Hk, N, d, generator=g, device="cuda", dtype=dtype)
    pos = torch.randint(0, 200000, (B, N), generator=g, device="cuda")
    f, scale = kv.rotary_frequencies(R, scaling="yarn", factor=4.0) if R > 2 else kv.rotary_frequencies(R)
    for inverse in (False, True):
        a, b = kv.rotary(q, k, pos, f, interleaved=interleaved, scale=scale, inverse=inverse)
        check(a, q, pos, f, interleaved, scale, inverse)
        check(b, k, pos, f, interleaved, scale, inverse)
    # in place gives the same bits, and so do queries alone
    q2, k2 = q.clone(), k.clone()
    kv.rotary(q2, k2, pos, f, interleaved=interleaved, scale=scale, inverse=True, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)
    assert torch.equal(kv.rotary(q, None, pos, f, interleaved=interleaved, scale=scale, inverse=True), a)


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens_form_and_position_kinds(cuda_device, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    T, Hq, Hk, d = 301, 12, 4, 128
    q = torch.randn(T, Hq, d, generator=g, device="cuda", dtype=dtype)
    k = torch.randn(T, Hk, d, generator=g, device="cuda", dtype=dtype)
    f, _ = kv.rotary_frequencies(128)

    def heads(x):
        return x.transpose(0, 1)[None]
    for pos in (torch.arange(T, device="cuda", dtype=torch.int32), torch.arange(T, device="cuda")[::1] * 7919 - 1000,
                torch.arange(2 * T, device="cuda", dtype=torch.int32)[::2]):
        a, b = kv.rotary(q, k, pos, f)
        check(heads(a), heads(q), pos[None], f, False, 1.0, False)
        check(heads(b), heads(k), pos[None], f, False, 1.0, False)
    # a start given as a number, and positions shared by the sequences
    x = torch.randn(3, 2, T, d, generator=g, device="cuda", dtype=dtype)
    pos = torch.arange(T, device="cuda") + 12345
    assert torch.equal(kv.rotary(x, None, 12345, f), kv.rotary(x, None, pos, f))
    check(kv.rotary(x, None, pos, f), x, pos[None].expand(3, T), f, False, 1.0, False)


def test_far_and_negative_positions(cuda_device):
    """fp64 itself loses 2^-53 of the angle: the bound grows with it alone."""
    f, _ = kv.rotary_frequencies(64)
    x = torch.randn(1, 2, 6, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    pos = torch.tensor([[0, 1, -1, 2**24 + 1, 2**31 + 5, -2**33]], device="cuda")
    got = kv.rotary(x, None, pos, f)
    y, w = formula(x.double(), pos, f, False, 1.0, False, 64)
    angle = 2.0 ** -51 * pos.abs().double()[:, None, :, None]
    err = (got.double() - y).abs()
    assert (err <= (2.0 ** -20 + angle) * w + 2.0 ** -24 * y.abs()).all()


def test_inverse_is_the_gradient_and_undoes(cuda_device):
    """<g, R x> = <R^T g, x>, checked against differences in 64 bits; with scale 1 the inverse brings x back."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g, e = (torch.randn(1, 3, 50, 64, device="cuda", generator=gen) for _ in range(3))
    f, _ = kv.rotary_frequencies(48, base=500.0)
    for il in (False, True):
        grad = kv.rotary(g, None, 100, f, scale=1.3, inverse=True, interleaved=il)
        # the pass-through part's gradient is g itself
        up = kv.rotary(x + e, None, 100, f, scale=1.3, interleaved=il).double()
        down = kv.rotary(x - e, None, 100, f, scale=1.3, interleaved=il).double()
        lhs, rhs = (g.double() * (up - down) / 2).sum(), (grad.double() * e.double()).sum()
        size = (g.double().abs() * (up.abs() + down.abs())).sum()
        assert abs(lhs - rhs) <= 2.0 ** -20 * size
        back = kv.rotary(kv.rotary(x, None, 100, f, interleaved=il), None, 100, f, inverse=True, interleaved=il)
        assert ((back - x).abs() <= 2.0 ** -18 * (1 + x.abs().max())).all()


def test_moves_a_key_between_positions(cuda_device):
    f, _ = kv.rotary_frequencies(128)
    x = torch.randn(1, 4, 9, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    at, to = torch.arange(9, device="cuda") * 1000, torch.arange(9, device="cuda")
    moved = kv.rotary(kv.rotary(x, None, at, f), None, to - at, f)
    assert ((moved - kv.rotary(x, None, to, f)).abs() <= 2.0 ** -18 * (1 + x.abs().max())).all()


def test_strides_and_nothing_to_do(cuda_device):
    f, _ = kv.rotary_frequencies(64)
    fused = torch.randn(2, 40, 9, 64, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(9))
    keep = fused.clone()
    q, k = fused[:, :, :4].transpose(1, 2), fused[:, :, 4:6].transpose(1, 2)
    a, b = kv.rotary(q, k, 3, f)
    check(a, q, torch.arange(40, device="cuda")[None].expand(2, 40) + 3, f, False, 1.0, False)
    kv.rotary(q, k, 3, f, q_out=q, k_out=k)  # in place inside the fused tensor
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(fused[:, :, 6:], keep[:, :, 6:])
    assert kv.rotary(q[:, :, :0], None, 0, f).shape == (2, 4, 0, 64)


def test_capture_and_stream(cuda_device):
    f, _ = kv.rotary_frequencies(128)
    x = torch.randn(64, 32, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(64, device="cuda")
    want = kv.rotary(x, None, pos, f)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = kv.rotary(x, None, pos, f)
    pos += 9
    g.replay()
    assert torch.equal(y, kv.rotary(x, None, pos, f)) and not torch.equal(y, want)


def test_offsets_beyond_32_bits(cuda_device):
    """Rows of a tensor of more than 2^31 elements, in place and out of it."""
    f, _ = kv.rotary_frequencies(64)
    big = torch.empty(3 * 2**30 + 4096, device="cuda", dtype=torch.bfloat16)
    x = big.as_strided((3, 2, 64), (3 * 2**29, 64, 1))
    x.copy_(torch.randn(3, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(19)))
    pos = torch.tensor([5, 6, 70000], device="cuda")
    want = kv.rotary(x.contiguous(), None, pos, f)
    assert torch.equal(kv.rotary(x, None, pos, f), want)
    kv.rotary(x, None, pos, f, q_out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_of_single_entries(cuda_device, dtype):
    """The stride of an axis of one entry says nothing: one token, one head, one sequence, in any strides, also in place
    through two views that differ in them."""
    f, _ = kv.rotary_frequencies(64)
    g = torch.Generator(device="cuda").manual_seed(23)
    for shape, odd in (((2, 4, 1, 64), 2), ((2, 1, 5, 64), 1), ((1, 4, 5, 64), 0), ((1, 1, 1, 64), 2)):
        x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        want = kv.rotary(x, None, 9, f)
        check(want, x, torch.arange(9, 9 + shape[2], device="cuda")[None].expand(shape[0], -1), f, False, 1.0, False)
        strides = list(x.stride())
        strides[odd] = 3
        view = x.as_strided(shape, strides)
        assert torch.equal(kv.rotary(view, None, 9, f), want)
        kv.rotary(view, None, 9, f, q_out=x)
        assert torch.equal(x, want)


def test_angle_error_grows_with_the_frequency(cuda_device):
    """The fraction of a turn per position comes from one fp64 product with a rounded 1 / 2 pi: off by at most 2^-53 for the
    rounding and 0.557 * 2^-53 for the constant, relative, and by 2^-64 for its own last bit; that times the position.
    Frequencies picked where the product rounds badly, against exact fractions."""
    from fractions import Fraction
    inv_2pi = Fraction(10**100, 2 * 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679)
    freqs = [float.fromhex(x) for x in ("0x1.ffe300998c775p-1", "0x1.91d6b0e0f714ap+2", "0x1.3fa61ea9c18cdp+3", "0x1.8f4bc22623ca6p+6")]
    positions = [1, 2**20 + 7, 2**33 + 11, -2**33 - 5]
    f = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    x = torch.randn(1, 3, 4, 8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(29))
    got = kv.rotary(x, None, torch.tensor([positions], device="cuda"), f).double()
    turns = torch.tensor([[float(Fraction(p) * Fraction(w) * inv_2pi % 1) for w in freqs] for p in positions], dtype=torch.float64, device="cuda")
    c, s = torch.cos(2 * torch.pi * turns), torch.sin(2 * torch.pi * turns)
    a, b = x.double().split(4, -1)
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    pos = torch.tensor(positions, dtype=torch.float64, device="cuda").abs()[:, None]
    angle = 2 * torch.pi * pos * (2.0 ** -52 * f / (2 * torch.pi) + 2.0 ** -64)
    size = (a.abs() + b.abs()).repeat(1, 1, 1, 2)
    assert ((got - want).abs() <= (2.0 ** -20 + angle.repeat(1, 2)) * size + 2.0 ** -24 * want.abs()).all()
