"""4-bit pages in which single groups are not finite, in keys that some rows of a sequence see and others do not; V's groups of
any size; both over the kernels' row counts (few rows, 16, several tiles) and head sizes. Bounds: tests/paged_reference.py,
over the rows and channels that no such group reaches; the others are not finite."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref
from tests.paged_reference import Pool, attention_bounds, parts
from tests.test_gpu_paged_attention import check_sequence

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
# (heads of q a KV head, new tokens): 8 rows, 16 rows, 16 + 4, one row an item for fp32
ROWS = [(4, 2), (8, 2), (4, 5), (1, 3)]


def one_sequence(d, dtype, G, n, m, H, spoils, window, n_sink):
    """spoils: (key, head, group, which, base, step), which 0 for K, 1 for V. Checks every row and channel."""
    pool = Pool([m], H, 16, d, dtype, True, seed=m + d, garbage=True)
    dead_k = torch.zeros(H, m, dtype=torch.bool, device="cuda")
    dead_v = torch.zeros(H, m, d, dtype=torch.bool, device="cuda")
    for key, h, j, which, base, step in spoils:
        parts((pool.k, pool.v)[which], d)[1][int(pool.table[0, key // 16]), h, key % 16, j] = torch.tensor([base, step], device="cuda").bfloat16()
        if which:
            dead_v[h, key, 32 * j:32 * j + 32] = True
        else:
            dead_k[h, key] = True
    q = torch.randn(n, G * H, d, generator=torch.Generator(device="cuda").manual_seed(m), device="cuda", dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, n_sink=n_sink, window=window, return_lse=True, error_word=err)
    assert int(err) == 0
    see = ref.visible(n, m, n_sink, window, q.device)
    # a logit that is not finite spoils its row, a value its channels
    rows = (see[None] & dead_k[:, None]).any(-1).repeat_interleave(G, 0)              # [Hq][n]
    channels = (see.double() @ dead_v.double() > 0).repeat_interleave(G, 0) | rows[..., None]
    assert channels.any() and not rows.all() and not channels.all()
    (k, ks, kst), (v, vs, vst) = (pool.rows(0, m, w) for w in (0, 1))

    def clean(x, dead):
        return torch.where(dead.expand_as(x) if dead.dim() == x.dim() else dead[..., None].expand_as(x), torch.zeros_like(x), x).repeat_interleave(G, 0)
    k, ks, kst = (clean(x, dead_k) for x in (k, ks, kst))
    v, vs, vst = (clean(x, dead_v) for x in (v, vs, vst))
    qq = q.double().transpose(0, 1)
    r, l, _ = ref.rows(qq, k, v, see, d ** -0.5)
    p = torch.softmax((qq @ k.transpose(1, 2) * d ** -0.5).masked_fill(~see, -INF), -1)
    tol, tol_l = attention_bounds(dtype, True, qq, k, ks, kst, p @ vs, p @ vst, m, d ** -0.5, r, l)
    got, got_l = out.double().transpose(0, 1), lse.double().transpose(0, 1)
    assert not torch.isfinite(got[channels]).any() and not torch.isfinite(got_l[rows]).any()
    assert ((got - r).abs() <= tol)[~channels].all(), float(((got - r).abs() / tol)[~channels].max())
    assert ((got_l - l).abs() <= tol_l)[~rows].all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("m", [75, 91, 600])
def test_groups_that_are_not_finite(cuda_device, m, G, n, d, dtype):
    window, last = 30, d // 32 - 1
    first = m - n - window + 1  # the lowest key that the first token's window reaches: no other token sees it
    for which in (1, 0):
        for base, step in ((NAN, 0.0), (NAN, INF), (0.5, INF), (INF, 1.0)):
            one_sequence(d, dtype, G, n, m, 2, [(first, 0, 0, which, base, step)], window, 0)
            one_sequence(d, dtype, G, n, m, 2, [(m - 1, 1, last, which, base, step)], window, 3)  # the last token's own key
    # several at once, in K and in V, of both heads
    one_sequence(d, dtype, G, n, m, 2, [(first, 0, last, 1, NAN, 0.0), (m - 1, 0, 0, 1, NAN, 0.0), (m - 1, 1, 0, 0, NAN, 0.0),
                                        (first + 1, 1, last, 1, NAN, 0.0)], window, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", ROWS)
def test_values_of_any_size(cuda_device, G, n, d):
    """V's groups far from one: small, large, and growing or falling by 2^40 from tile to tile of one sequence."""
    for scale in ([2.0 ** -40], [2.0 ** 50], [2.0 ** -20, 2.0 ** 20], [2.0 ** 30, 2.0 ** -10], [2.0 ** -15, 1.0, 2.0 ** 15, 0.0]):
        lens = [400, 60, 1700]
        pool = Pool(lens, 2, 16, d, torch.bfloat16, True, seed=5)
        _, params = parts(pool.v, d)
        for b, m in enumerate(lens):
            for j in range(-(-m // 16)):
                params[int(pool.table[b, j])] *= scale[j % len(scale)]
        q = torch.randn(3 * n, 2 * G, d, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(6))
        out, lse = kv.paged_attention(q, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True)
        for b, m in enumerate(lens):
            rows = slice(b * n, b * n + n)
            check_sequence(pool, b, q[rows], out[rows], lse[rows], m, 0, None, d ** -0.5)
