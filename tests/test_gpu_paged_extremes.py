"""4-bit groups, and queries over them, at the ends of fp32's range. The bounds of check_groups in tests/paged_reference.py
with the absolute term of fp32's own grid instead of one that hides these groups: differences and products below 2^-126 are
off by 2^-150 each, eight of them at most (2^-147), and a base or a step is rounded on bf16's grid, 2^-133 there."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests.paged_reference import Pool, parts, unpack
from tests.test_gpu_paged_attention import check_sequence

pytestmark = pytest.mark.gpu
GRID = 2.0 ** -133


def check(x, codes, params):
    """x [n][d] fp64, codes [n][d], params [n][d / 32][2] as stored."""
    x, c = x.unflatten(-1, (-1, 32)), codes.double().unflatten(-1, (-1, 32))
    base, step = params[..., 0].double(), params[..., 1].double()
    lo, hi = x.amin(-1), x.amax(-1)
    size = lo.abs() + hi.abs()
    assert torch.isfinite(base).all() and torch.isfinite(step).all()
    assert ((base - (8 * hi + 7 * lo) / 15).abs() <= 2.0 ** -8 * base.abs() + 2.0 ** -20 * size + GRID).all()
    need = torch.maximum((hi - base) / 7, (base - lo) / 8)
    fuzz = 2.0 ** -20 * (size + base.abs()) + 2.0 ** -147
    assert (step >= need - fuzz).all() and (step <= need * (1 + 2.0 ** -7) + 2 * fuzz + GRID).all()
    v = base[..., None] + (c - 8) * step[..., None]
    # (half a step, and the quotient's own error: 15 steps times 2^-22)
    off = ((v - x).abs() - fuzz[..., None]) / step[..., None].clamp_min(2.0 ** -149)
    assert (off <= 0.5 + 15 * 2.0 ** -22).all(), float(off.max())
    assert (c[(step == 0)[..., None].expand_as(c)] == 8).all()


def appended(x, R=None):
    """x [T][1][d] as the keys and values of one sequence, and what its pages hold of them."""
    T, H, d = x.shape
    pool = Pool([T], H, 16, d, x.dtype, True, garbage=False)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = None if R is None else kv.rotary_frequencies(R)[0] * 0  # (angles of 0: the keys as they are)
    kv.paged_append(x, x, pool.k, pool.v, pool.table, pool.kv_lens, inv_freq=f, error_word=err)
    assert int(err) == 0
    pages = pool.table[0].long()
    for p in (pool.k, pool.v):
        codes, params = parts(p, d)
        yield unpack(codes[pages].transpose(0, 1).reshape(H, -1, d // 2)[:, :T])[0], params[pages].transpose(0, 1).reshape(H, -1, d // 32, 2)[0, :T]


def values(dtype, d, T=48):
    g = torch.Generator(device="cuda").manual_seed(d)
    return torch.rand(T, 1, d, generator=g, device="cuda", dtype=torch.float64) * 2 - 1


@pytest.mark.parametrize("R", [None, 64, 6])  # (both kernels that write 4 bits)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_far_apart(cuda_device, d, dtype, R):
    """Groups that reach from one end of the type's range to the other."""
    most = torch.finfo(dtype).max
    x = values(dtype, d)
    x[:, :, ::32], x[:, :, 1::32] = -1, 1
    x = (x * torch.linspace(0.8, 1, x.shape[0], device="cuda", dtype=torch.float64)[:, None, None] * most).to(dtype)
    for codes, params in appended(x, R):
        check(x[:, 0].double(), codes, params)


@pytest.mark.parametrize("R", [None, 64, 6])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_close_together(cuda_device, d, dtype, R):
    """Groups whose steps are below the smallest normal value, down to nothing but zeros; a few around it; and values of one
    size with such steps between them and without."""
    x = values(dtype, d, 60)
    x = x * torch.exp2(torch.linspace(-149, -115, 60, device="cuda", dtype=torch.float64).round())[:, None, None]
    for codes, params in appended(x.to(dtype), R):
        check(x.to(dtype)[:, 0].double(), codes, params)
    x = torch.full_like(x, 2.0 ** -110) * (1 + 2.0 ** -7 * (values(dtype, d, 60) > 0))
    x[::3] = torch.tensor([3.0e38, -1.5, 2.0 ** -126, 0.0], device="cuda", dtype=torch.float64).repeat(5)[:, None, None]
    for codes, params in appended(x.to(dtype), R):
        check(x.to(dtype)[:, 0].double(), codes, params)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 2)])
@pytest.mark.parametrize("up", [-100, -30, 30, 90, 114])
def test_queries_of_any_size(cuda_device, up, G, n, d):
    """Queries up to 2^118 and keys as much smaller, and the other way around: the same logits."""
    lens = [300, 40]
    pool = Pool(lens, 2, 16, d, torch.bfloat16, True, seed=3)
    parts(pool.k, d)[1].mul_(2.0 ** -up)
    q = torch.randn(2 * n, 2 * G, d, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(8)) * 2.0 ** up
    assert float(q.abs().max()) < 2.0 ** 118
    out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True)
    for b, m in enumerate(lens):
        rows = slice(b * n, b * n + n)
        check_sequence(pool, b, q[rows], out[rows], lse[rows], m, 0, None, d ** -0.5)
