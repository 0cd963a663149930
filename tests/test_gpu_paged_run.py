"""The operators of a paged cache as a serving loop uses them: prompts in chunks, then decode steps, captured once and
replayed, on norms and rotary positions; every output against 64-bit attention over what the pages hold, and pages of the
keys' own type against the same run on plain tensors."""
import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from tests import attn_reference as ref
from tests.paged_reference import Pool
from tests.test_gpu_paged_attention import check_sequence, starts_of

pytestmark = pytest.mark.gpu
Hq, H, D, S = 8, 2, 64, 16


class Loop:
    def __init__(self, dtype, four, total):
        g = torch.Generator(device="cuda").manual_seed(13)
        self.dtype, self.four = dtype, four
        self.pool = Pool(total, H, S, D, dtype, four, seed=2, garbage=True)
        self.pool.kv_lens.zero_()
        self.q, self.k, self.v = ([torch.randn(m, h, D, generator=g, device="cuda", dtype=dtype) * 2 for m in total] for h in (Hq, H, H))
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2))
        self.f, _ = kv.rotary_frequencies(D)
        # the whole run's queries and keys, normed and turned at their places
        self.turned = [kv.norm_rotary(q, k, self.wq, self.wk, 0, self.f) for q, k in zip(self.q, self.k)]

    def check(self, b, first, n, out, lse):
        check_sequence(self.pool, b, self.turned[b][0][first:first + n], out, lse, first + n, 0, None, D ** -0.5)

    def keys_are_there(self, b, m):
        if not self.four:
            for which, x in enumerate((self.turned[b][1], self.v[b])):
                assert torch.equal(self.pool.rows(b, m, which)[0], x[:m].transpose(0, 1).double())


@pytest.mark.parametrize("dtype,four", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False), (torch.float32, True)])
def test_chunks_then_steps(cuda_device, dtype, four):
    total = [75, 40, 131]
    run = Loop(dtype, four, total)
    pool = run.pool
    done = [0, 0, 0]
    # prompts in chunks: normed, appended with the rotation on the way, read back for the chunk's attention
    for chunk in ([33, 40, 64], [30, 0, 50]):
        starts = starts_of(chunk)
        pool.kv_lens += torch.tensor(chunk, dtype=torch.int32, device="cuda")
        q, k, v = (torch.cat([x[b][done[b]:done[b] + n] for b, n in enumerate(chunk)]) for x in (run.q, run.k, run.v))
        pos = torch.cat([torch.arange(done[b], done[b] + n, device="cuda") for b, n in enumerate(chunk)])
        qn, kn = kv.norm_rotary(q, k, run.wq, run.wk, pos, run.f)
        if dtype == torch.float32:  # (rounded once either way: the same bits)
            kv.paged_append(kv.norm_rotary(k, None, run.wk, None), v, pool.k, pool.v, pool.table, pool.kv_lens, starts=starts, inv_freq=run.f)
        else:
            kv.paged_append(kn, v, pool.k, pool.v, pool.table, pool.kv_lens, starts=starts)
        m = [d + n for d, n in zip(done, chunk)]
        ks = starts_of(m)
        kk, vv = kv.paged_gather(pool.k, pool.v, pool.table, pool.kv_lens, k_starts=ks, rows=sum(m), dtype=dtype)
        out, lse = kv.window_attention(qn, kk, vv, q_starts=starts, k_starts=ks, max_q=max(chunk), max_k=max(m), return_lse=True)
        direct, dlse = kv.paged_attention(qn, pool.k, pool.v, pool.table, pool.kv_lens, q_starts=starts, max_q=max(chunk), return_lse=True)
        at = 0
        for b, n in enumerate(chunk):
            run.check(b, done[b], n, direct[at:at + n], dlse[at:at + n])
            if n:  # the chunk's attention, over the values that were read back
                qb, kb, vb = (x.transpose(0, 1) for x in (qn[at:at + n], kk[int(ks[b]):int(ks[b + 1])], vv[int(ks[b]):int(ks[b + 1])]))
                r, l, A = ref.sequence(qb, kb, vb, 0, None, D ** -0.5)
                tol, tol_l = ref.bounds(dtype, qb, kb, m[b], D ** -0.5, r, A, l)
                ref.assert_close(out[at:at + n].transpose(0, 1), r, tol, "out")
                ref.assert_close(lse[at:at + n].transpose(0, 1), l, tol_l, "lse")
            at += n
            if dtype == torch.bfloat16:
                run.keys_are_there(b, m[b])
        done = m
    # decode steps: one graph, lengths counted up on the device
    q1, k1, v1 = (torch.empty(3, h, D, device="cuda", dtype=dtype) for h in (Hq, H, H))
    pos = torch.empty(3, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pos.copy_(pool.kv_lens)
            pool.kv_lens += 1
            qn, kn = kv.norm_rotary(q1, k1, run.wq, run.wk, pos, run.f)
            kv.paged_append(kn, v1, pool.k, pool.v, pool.table, pool.kv_lens)
            out, lse = kv.paged_attention(qn, pool.k, pool.v, pool.table, pool.kv_lens, return_lse=True)
    torch.cuda.synchronize()
    order = [0, 2]  # (the second sequence has all its pages' tokens: its further ones find no page and are dropped)
    for step in range(12):
        for b in order:
            q1[b], k1[b], v1[b] = run.q[b][done[b]], run.k[b][done[b]], run.v[b][done[b]]
        q1[1], k1[1], v1[1] = 0, 0, 0
        g.replay()
        torch.cuda.synchronize()
        for b in order:
            run.check(b, done[b], 1, out[b:b + 1], lse[b:b + 1])
            done[b] += 1
    for b in order:
        if dtype == torch.bfloat16:
            run.keys_are_there(b, done[b])
    assert kv.operator_errors() == 0x20


def test_four_bit_pages_hold_two_calls_at_once(cuda_device):
    """Appends to different sequences and attention over others, on two streams, share nothing."""
    pool = Pool([300, 500], 2, 16, 64, torch.bfloat16, True, garbage=False)
    q = torch.randn(1, 8, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(300, 2, 64, device="cuda", dtype=torch.bfloat16)
    want = kv.paged_attention(q, pool.k, pool.v, pool.table[1:], pool.kv_lens[1:])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            kv.paged_append(x, x, pool.k, pool.v, pool.table[:1], pool.kv_lens[:1])
        with torch.cuda.stream(b):
            got = kv.paged_attention(q, pool.k, pool.v, pool.table[1:], pool.kv_lens[1:])
            assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert kv.operator_errors() == 0
