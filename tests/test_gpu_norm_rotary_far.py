"""norm_rotary at far positions. The fraction of a turn is computed as in rotary(), whose own tests hold it against exact
fractions; so in fp32 norm_rotary is rotary of the normed heads: the norm is rounded once more between the two (2^-24 of each
of the pair), and its products and the turn are taken in another order, six fp32 operations of a value each way (2^-21); bf16
is the same with half a step of the output."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [128, 64, 6])  # (both kernels)
@pytest.mark.parametrize("far", [2**20, 2**33, -2**33, 2**62, -2**62])
def test_far_positions(cuda_device, far, R, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn(41, 5, 128, generator=g, device="cuda", dtype=dtype) * 3
    w = (1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(dtype)
    pos = far + torch.randint(0, 100000, (41,), generator=g, device="cuda")
    f, _ = kv.rotary_frequencies(R)
    got = kv.norm_rotary(x, None, w, None, pos, f, interleaved=interleaved).double()
    normed = kv.norm_rotary(x.float(), None, w.float(), None)
    want = kv.rotary(normed, None, pos, f, interleaved=interleaved).double()
    size, n = normed.double().abs(), normed.double().abs()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    size[..., a] = size[..., b] = n[..., a] + n[..., b]
    assert ((got - want).abs() <= 2.0 ** -21 * size + torch.finfo(dtype).eps / 2 * want.abs()).all()
    assert not torch.allclose(want[..., :R], normed.double()[..., :R], atol=0.1)  # (they do turn)
