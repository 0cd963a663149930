"""The scale of an attention's logits is an fp32 number in the library, where 0 means the default: what fp32 does not hold is
refused, not taken for it."""
import pytest
import torch

from tests.test_paged_cpu import L, as_if_on_gpu, make  # noqa: F401


def calls():
    import kv_cache_eviction_decode_gb300 as kv
    c = make(dtype=torch.float32)
    q, p = torch.zeros(6, 8, 64), torch.zeros(2, 2, 8, 64)
    return {"paged": lambda s: kv.paged_attention(q, *c, scale=s), "window": lambda s: kv.window_attention(p, p, p, scale=s),
            "prefix": lambda s: kv.shared_prefix_attention(p[:, :, 0], p[0], p[0], p, p, scale=s)}


@pytest.mark.parametrize("name", ["paged", "window", "prefix"])
def test_scales_of_logits(as_if_on_gpu, name):  # noqa: F811
    for scale in (1e-50, 2.0 ** -150, 1e39, 1e300, 0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="^scale"):
            calls()[name](scale)
    for scale in (1e-45, 1e-40, 1, 3.4028234e38, None):
        with pytest.raises(RuntimeError, match="launched"):
            calls()[name](scale)
