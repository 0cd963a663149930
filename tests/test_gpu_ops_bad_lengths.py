"""window_attention where the lengths or starts on the device are out of range: the sound sequences' rows are right, the
same in every call, and no other row is written."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def packed(qs, ks, dtype, max_q, Hq=4, Hkv=2, d=64, repeats=5, q_rows=None, k_rows=None):
    """The call's out, lse and error word; unwritten rows hold 7. The same bits in every repeat."""
    g = torch.Generator(device="cuda").manual_seed(21)
    q_rows, k_rows = q_rows or max(qs), k_rows or max(ks)
    q = torch.randn(q_rows, Hq, d, generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn(k_rows, Hkv, d, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    a, b = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qs, ks))
    first = None
    for _ in range(repeats):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        kv.window_attention(q, k, v, q_starts=a, k_starts=b, max_q=max_q, max_k=k_rows, out=out, lse=lse, error_word=err)
        if first is None:
            first = (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    return q, k, v, out, lse, int(err)


def check_rows(q, k, v, out, lse, q0, n, k0, m, n_given=None):
    """Rows q0 .. q0 + n - 1, the first of n_given queries at the end of the keys k0 .. k0 + m - 1."""
    n_given = n if n_given is None else n_given
    pad = torch.zeros(n_given - n, *q.shape[1:], device=q.device, dtype=q.dtype)
    qq = torch.cat([q[q0:q0 + n], pad]).transpose(0, 1)
    kk, vv = (x[k0:k0 + m].transpose(0, 1) for x in (k, v))
    scale = q.shape[-1] ** -0.5
    r, l, A = ref.sequence(qq, kk, vv, 0, None, scale)
    tol, tol_l = ref.bounds(q.dtype, qq, kk, m, scale, r, A, l)
    ref.assert_close(out[q0:q0 + n].transpose(0, 1), r[:, :n], tol[:, :n], "out")
    ref.assert_close(lse[q0:q0 + n].transpose(0, 1), l[:, :n], tol_l[:, :n], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("starts,whole", [([0, 20, 10, 15, 40], 1), ([0, 10, 5, 7, 20], 1), ([0, 5, 20, 3, 9, 30], 2)])
def test_starts_that_go_back(cuda_device, starts, whole, dtype):
    """A later sequence that ascends again inside an earlier one's rows is left out."""
    q, k, v, out, lse, err = packed(starts, starts, dtype, max(starts))
    assert err == 0x10
    for b in range(whole):
        check_rows(q, k, v, out, lse, starts[b], starts[b + 1] - starts[b], starts[b], starts[b + 1] - starts[b])
    for t in (out, lse):
        assert (t[starts[whole]:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_starts_that_go_back_with_split_keys(cuda_device, dtype):
    """Few rows over many keys: the join leaves the same sequences out as the parts."""
    q, k, v, out, lse, err = packed([0, 2, 1, 3], [0, 5000, 6000, 11000], dtype, 2)
    assert err == 0x10
    check_rows(q, k, v, out, lse, 0, 2, 0, 5000)
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_starts_that_go_back_in_a_long_batch(cuda_device, dtype):
    """300 sequences of one row, of which the 201st goes back."""
    starts = list(range(201)) + [150] + list(range(151, 250))
    q, k, v, out, lse, err = packed(starts, [3 * x for x in starts], dtype, 1, q_rows=300, k_rows=900)
    assert err == 0x10
    for b in (0, 127, 128, 149, 150, 199):
        check_rows(q, k, v, out, lse, b, 1, 3 * b, 3)
    assert (out[200:] == 7).all() and (lse[200:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_more_queries_than_max_q(cuda_device, dtype):
    """The rows that are computed see what they would see with all of them; the others are not written."""
    q, k, v, out, lse, err = packed([0, 30, 40], [0, 30, 50], dtype, 20)
    assert err == 0x10
    check_rows(q, k, v, out, lse, 0, 20, 0, 30, n_given=30)
    check_rows(q, k, v, out, lse, 30, 10, 30, 20)
    assert (out[20:30] == 7).all() and (lse[20:30] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [30, 5000])
def test_more_queries_than_rows(cuda_device, m, dtype):
    """Padded: q_lens beyond the rows; with many keys split and joined."""
    n, given, d = 8, 11, 64
    g = torch.Generator(device="cuda").manual_seed(22)
    q = torch.randn(1, 4, n, d, generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn(1, 2, m, d, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kv.window_attention(q, k, v, q_lens=torch.tensor([given], dtype=torch.int32, device="cuda"), error_word=err, return_lse=True)
    assert int(err) == 0x10
    check_rows(*(x[0].transpose(0, 1) for x in (q, k, v, out)), lse[0].t(), 0, n, 0, m, n_given=given)


@pytest.mark.parametrize("dtype", TYPES)
def test_errors_without_a_word_of_the_callers(cuda_device, dtype):
    """They are kept on the device until they are asked for."""
    g = torch.Generator(device="cuda").manual_seed(23)
    q = torch.randn(2, 4, 3, 64, generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn(2, 2, 20, 64, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    good, bad = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([20, 7], [20, 70]))
    assert kv.operator_errors() == 0
    kv.window_attention(q, k, v, kv_lens=good)
    assert kv.operator_errors() == 0
    kv.window_attention(q, k, v, kv_lens=bad)
    kv.window_attention(q, k, v, kv_lens=good)
    assert kv.operator_errors() == kv.DEV_BAD_LENGTH and kv.operator_errors() == 0
    kv.shared_prefix_attention(q[:, :, 0], k[0], v[0], k, v, bad)
    assert kv.operator_errors(q.device) == kv.DEV_BAD_LENGTH and kv.operator_errors() == 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.window_attention(q, k, v, kv_lens=bad, error_word=err)
    assert int(err) == kv.DEV_BAD_LENGTH and kv.operator_errors() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.window_attention(q, k, v, kv_lens=good)
    assert kv.operator_errors() == 0
    good.copy_(bad)
    graph.replay()
    assert kv.operator_errors() == kv.DEV_BAD_LENGTH
