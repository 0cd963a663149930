"""shared_prefix_attention against the formula in 64 bits over prefix and suffix together."""
import math

import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def make(B, Hq, Hkv, P, M, d, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=dtype)
    return r(B, Hq, d), r(Hkv, P, d), r(Hkv, P, d), r(B, Hkv, M, d), r(B, Hkv, M, d)


def check(q, kp, vp, k, v, lens, out, lse, scale=None):
    B, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = scale or d ** -0.5
    # a sum of two parts, each rounded to fp32, and for bf16 each with probabilities rounded on their own scale
    for b in range(B):
        kk, vv = torch.cat([kp, k[b, :, :lens[b]]], 1), torch.cat([vp, v[b, :, :lens[b]]], 1)
        see = torch.ones(1, kk.shape[1], dtype=torch.bool, device="cuda")
        r, l, A = ref.rows(q[b][:, None].double(), kk.double().repeat_interleave(G, 0), vv.double().repeat_interleave(G, 0), see, scale)
        tol, tol_l = ref.bounds(q.dtype, q[b][:, None], kk, kk.shape[1], scale, r, A, l)
        ref.assert_close(out[b][:, None], r, tol, f"out {b}")
        ref.assert_close(lse[b][:, None], l, tol_l, f"lse {b}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hq,Hkv,P,M,d", [
    (1, 1, 1, 1, 1, 64), (3, 8, 2, 333, 40, 128), (20, 8, 8, 1000, 129, 64), (33, 16, 2, 700, 3, 128),
    (5, 64, 1, 200, 300, 64), (4, 6, 2, 5000, 0, 128), (7, 4, 4, 0, 200, 64), (2, 2, 2, 0, 0, 64), (130, 4, 2, 129, 1, 64),
])
def test_forms(cuda_device, B, Hq, Hkv, P, M, d, dtype):
    q, kp, vp, k, v = make(B, Hq, Hkv, P, M, d, dtype)
    lens = [(b * 37 + 1) % (M + 1) for b in range(B)]
    for b in range(B):
        k[b, :, lens[b]:] = math.nan
        v[b, :, lens[b]:] = math.nan
    out, lse = kv.shared_prefix_attention(q, kp, vp, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    check(q, kp, vp, k, v, lens, out, lse)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_no_lengths(cuda_device, dtype):
    B, Hq, Hkv, P, M, d = 4, 8, 4, 300, 77, 128
    q, kp, vp, k, v = make(B, Hq, Hkv, P, M, d, dtype, 3)
    qq = torch.empty(B, 3 * Hq, d, device="cuda", dtype=dtype)[:, Hq:2 * Hq].copy_(q)
    kpp, vpp = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (kp, vp))   # token-major
    kk, vv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    out, lse = kv.shared_prefix_attention(qq, kpp, vpp, kk, vv, return_lse=True, scale=0.2)
    check(q, kp, vp, k, v, [M] * B, out, lse, 0.2)


def test_equals_a_cache_that_holds_the_prefix_itself(cuda_device):
    """The same keys, once as a common prefix and once inside every sequence, differ by rounding only."""
    B, Hq, Hkv, P, M, d = 6, 8, 2, 900, 130, 128
    q, kp, vp, k, v = make(B, Hq, Hkv, P, M, d, torch.float32, 4)
    a = kv.shared_prefix_attention(q, kp, vp, k, v)
    kk, vv = (torch.cat([p.expand(B, -1, -1, -1), s], 2) for p, s in ((kp, k), (vp, v)))
    b = kv.window_attention(q[:, :, None], kk, vv)[:, :, 0]
    assert (a - b).abs().max() < 1e-5


def test_capture_and_streams(cuda_device):
    q, kp, vp, k, v = make(8, 8, 2, 3000, 500, 128, torch.bfloat16, 5)
    lens = torch.full((8,), 400, dtype=torch.int32, device="cuda")
    want = kv.shared_prefix_attention(q, kp, vp, k, v, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = kv.shared_prefix_attention(q, kp, vp, k, v, lens)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kv.shared_prefix_attention(q, kp, vp, k, v, lens)
    lens.fill_(17)
    g.replay()
    assert torch.equal(got, kv.shared_prefix_attention(q, kp, vp, k, v, lens))
