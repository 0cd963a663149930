"""norm_rotary against the formula in 64 bits. Per element of the result, with a and b the normed pair: the sum of squares
(d fp32 operations, each off by at most 2^-24 of a sum of positive terms: (d + 2) 2^-24, halved by the root), the root
(2^-22), two products (2^-23), cosine and sine and the turn (2^-20 with the angle, as in the tests of rotary), then half a
step of the output: |err| <= ((d + 2) 2^-25 + 2^-22 + 2^-23 + 2^-20) (|a| + |b|) scale + eps / 2 |y|."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def check(got, x, w, pos, f, interleaved=False, scale=1.0, eps=1e-6):
    """x, got [B][H][N][d], pos [B][N]."""
    x, w = x.double(), w.double()
    d = x.shape[-1]
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    size = y.abs()
    if f is not None:
        R = 2 * f.shape[0]
        t = pos.double()[:, None, :, None] * f
        c, s = torch.cos(t) * scale, torch.sin(t) * scale
        a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = ya * c - yb * s, ya * s + yb * c
        size[..., a] = size[..., b] = (ya.abs() + yb.abs()) * abs(scale)
    tol = ((d + 2) * 2.0 ** -25 + 2.0 ** -22 + 2.0 ** -23 + 2.0 ** -20) * size + torch.finfo(got.dtype).eps / 2 * y.abs() + 1e-38
    err = (got.double() - y).abs()
    assert (err <= tol * 1.0001).all(), float((err / tol).max())


def tensors(B, Hq, Hk, N, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn(B, H, N, d, generator=g, device="cuda", dtype=dtype) * 3 for H in (Hq, Hk))
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2))
    return q, k, wq, wk, torch.randint(0, 200000, (B, N), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R", [(128, 128), (64, 64), (128, 64), (128, 48), (64, 10), (128, 2), (72, 72), (256, 256), (512, 24), (1024, 1024),
                                 (8, 6), (8, 8), (128, 0), (96, 32)])
def test_layouts(cuda_device, d, R, interleaved, dtype):
    q, k, wq, wk, pos = tensors(2, 5, 3, 37, d, dtype, d + R)
    f, scale = kv.rotary_frequencies(R) if R else (None, 1.0)
    scale = 1.25 if R else 1.0
    a, b = kv.norm_rotary(q, k, wq, wk, pos, f, interleaved=interleaved, scale=scale)
    check(a, q, wq, pos, f, interleaved, scale)
    check(b, k, wk, pos, f, interleaved, scale)
    q2, k2 = q.clone(), k.clone()  # in place gives the same bits, and so do queries alone
    kv.norm_rotary(q2, k2, wq, wk, pos, f, interleaved=interleaved, scale=scale, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)
    assert torch.equal(kv.norm_rotary(q, None, wq, None, pos, f, interleaved=interleaved, scale=scale), a)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 64, 8), (64, 32, 8), (301, 12, 4), (3, 5, 1)])
def test_tokens(cuda_device, T, Hq, Hk, dtype):
    q, k, wq, wk, pos = tensors(1, Hq, Hk, T, 128, dtype, T)
    q, k, pos = q[0].transpose(0, 1).contiguous(), k[0].transpose(0, 1).contiguous(), pos[0]
    f, _ = kv.rotary_frequencies(128)
    for p in (pos, pos.int(), pos - 2**33):
        a, b = kv.norm_rotary(q, k, wq, wk, p, f)
        for got, x, w in ((a, q, wq), (b, k, wk)):
            if p is not pos and p.dtype == torch.int64:
                continue  # far positions: the angle's own bound is in the tests of rotary
            check(got.transpose(0, 1)[None], x.transpose(0, 1)[None], w, p[None], f)
    # the norm's rounding apart, it is rotary of the normed heads
    n = kv.norm_rotary(q, None, wq, None)
    check(n.transpose(0, 1)[None], q.transpose(0, 1)[None], wq, None, None)


def test_small_and_large_heads(cuda_device):
    """Heads of zeros give zeros; squares that only eps keeps apart from zero; large values, infinities and NaN."""
    f, _ = kv.rotary_frequencies(64)
    x = torch.zeros(1, 5, 3, 64, device="cuda")
    x[0, 1] = 1e-5 * torch.randn(3, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[0, 2] = 1e15
    x[0, 3, 1, 7], x[0, 4, 1, 7] = float("inf"), float("nan")
    w = torch.ones(64, device="cuda")
    got = kv.norm_rotary(x, None, w, None, 5, f)
    pos = torch.arange(5, 8, device="cuda")[None]
    assert (got[0, 0] == 0).all()
    check(got[:, :3], x[:, :3], w, pos, f)
    assert torch.isnan(got[0, 3:, 1]).any(-1).all() and torch.isfinite(got[0, 3:, 0::2]).all()


def test_strides_capture_and_nothing_to_do(cuda_device):
    f, _ = kv.rotary_frequencies(64)
    fused = torch.randn(2, 40, 9, 64, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(9))
    keep = fused.clone()
    w = torch.linspace(0.5, 1.5, 64, device="cuda").bfloat16()
    q, k = fused[:, :, :4].transpose(1, 2), fused[:, :, 4:6].transpose(1, 2)
    a, b = kv.norm_rotary(q, k, w, w, 3, f)
    check(a, q, w, torch.arange(40, device="cuda")[None].expand(2, 40) + 3, f)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a2, b2 = kv.norm_rotary(q, k, w, w, 3, f)
    a2.zero_()
    g.replay()
    assert torch.equal(a2, a) and torch.equal(b2, b)
    kv.norm_rotary(q, k, w, w, 3, f, q_out=q, k_out=k)  # in place inside the fused tensor
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(fused[:, :, 6:], keep[:, :, 6:])
    assert kv.norm_rotary(q[:, :, :0], None, w, None, 0, f).shape == (2, 4, 0, 64)


def test_offsets_beyond_32_bits(cuda_device):
    f, _ = kv.rotary_frequencies(64)
    big = torch.empty(3 * 2**30 + 4096, device="cuda", dtype=torch.bfloat16)
    x = big.as_strided((3, 2, 64), (3 * 2**29, 64, 1))
    x.copy_(torch.randn(3, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(19)))
    w, pos = torch.ones(64, device="cuda").bfloat16(), torch.tensor([5, 6, 70000], device="cuda")
    want = kv.norm_rotary(x.contiguous(), None, w, None, pos, f)
    assert torch.equal(kv.norm_rotary(x, None, w, None, pos, f), want)
    kv.norm_rotary(x, None, w, None, pos, f, q_out=x)
    assert torch.equal(x, want)
