"""The operators on a cache's own path: a prompt attended and appended in one
call, positions rotated at the layer's next ones, decode steps behind a shared
prefix -- each against the formula in 64 bits over the tokens that the cache
holds, and one run of them together."""
import math

import pytest
import torch

import kv_cache_eviction_decode_gb300 as kv
from kv_cache_eviction_decode_gb300 import BF16, F32, H2O, H2O_BLOCK, RANDOM, SINK_WINDOW, KVEvictCache, KVEvictError
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
DT = {F32: torch.float32, BF16: torch.bfloat16}


def cache(policy, dtype, B=2, L=1, Hq=8, Hkv=2, d=64, **kw):
    base = dict(policy=policy, batch=B, n_layers=L, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, dtype=dtype)
    if policy == SINK_WINDOW:
        base.update(n_sink=4, n_recent=28, budget=32)
    elif policy == RANDOM:
        base.update(budget=24, r=8, max_prompt=64, seed=5)
    elif policy == H2O:
        base.update(n_sink=4, n_heavy=12, n_recent=16, budget=32)
    else:
        base.update(n_sink=4, n_heavy=28, n_recent=32, budget=64, r=8)
    base.update(kw)
    return KVEvictCache(device="cuda:0", **base)


def rnd(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def step_reference(q, keys, values, scale):
    """One token of every sequence: q [B][Hq][d]; keys[b][h], values[b][h] [m][d]: out, lse, A and the longest m."""
    B, Hq, d = q.shape
    outs, As, ms = [], [], 0
    for b in range(B):
        Hkv = len(keys[b])
        for h in range(Hkv):
            G = Hq // Hkv
            qq = q[b, h * G:(h + 1) * G][:, None].double()
            k, v = (x[b][h].double()[None].expand(G, -1, -1) for x in (keys, values))
            see = torch.ones(1, k.shape[1], dtype=torch.bool, device=q.device)
            r, _, A = ref.rows(qq, k, v, see, scale)
            outs.append(r)
            As.append(A)
            ms = max(ms, k.shape[1])
    return torch.cat(outs).view(B, Hq, d), torch.cat(As).view(B, Hq, d), ms


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("policy", [SINK_WINDOW, RANDOM, H2O, H2O_BLOCK])
@pytest.mark.parametrize("P", [1, 33, 64])
def test_prefill_attend(cuda_device, policy, dtype, P):
    """The outputs are the formula's, and the cache holds what prefill() puts there."""
    g = torch.Generator(device="cuda").manual_seed(P)
    a, b = cache(policy, dtype), cache(policy, dtype)
    t = DT[dtype]
    Q, K, V = rnd(g, 2, 8, P, 64, dtype=t), rnd(g, 2, 2, P, 64, dtype=t), rnd(g, 2, 2, P, 64, dtype=t)
    out, lse = a.prefill_attend(0, Q, K, V, return_lse=True)
    b.prefill(0, K, V)
    for i in range(2):
        n_sink, window = (4, 29) if policy == SINK_WINDOW else (0, None)
        r, l, A = ref.sequence(Q[i], K[i], V[i], n_sink, window, 0.125)
        tol, tol_l = ref.bounds(t, Q[i], K[i], P, 0.125, r, A, l)
        ref.assert_close(out[i], r, tol, "out")
        ref.assert_close(lse[i], l, tol_l, "lse")
    assert a.layer_state(0) == b.layer_state(0)
    assert torch.equal(a.slot_positions(0), b.slot_positions(0))
    q, k, v = rnd(g, 2, 8, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t)
    assert torch.equal(a.decode_step(0, q, k, v), b.decode_step(0, q, k, v))
    assert a.check() == 0 and b.check() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_attention_is_the_decode_steps(cuda_device, dtype):
    """The prompt's rows are what the SINK_WINDOW cache gives token by token: both within the bounds of one formula."""
    g = torch.Generator(device="cuda").manual_seed(3)
    t, P = DT[dtype], 90
    Q, K, V = rnd(g, 2, 8, P, 64, dtype=t), rnd(g, 2, 2, P, 64, dtype=t), rnd(g, 2, 2, P, 64, dtype=t)
    c = cache(SINK_WINDOW, dtype)
    steps = torch.stack([c.decode_step(0, Q[:, :, i].contiguous(), K[:, :, i].contiguous(), V[:, :, i].contiguous())
                         for i in range(P)], 2)
    out = cache(SINK_WINDOW, dtype).prefill_attend(0, Q, K, V)
    for i in range(2):
        r, l, A = ref.sequence(Q[i], K[i], V[i], 4, 29, 0.125)
        tol, _ = ref.bounds(t, Q[i], K[i], 33, 0.125, r, A, l)
        ref.assert_close(out[i], r, tol, "prompt")
        ref.assert_close(steps[i], r, tol, "steps")


@pytest.mark.parametrize("policy", [SINK_WINDOW, RANDOM])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,split", [(300, 0), (0, 0), (1, 2)])
def test_decode_step_shared(cuda_device, policy, dtype, P, split):
    """Steps through fills, evictions and cuts: every output against the formula over the prefix, the tokens that the
    cache held before the step, and the new one; the cache itself does what it does without a prefix."""
    g = torch.Generator(device="cuda").manual_seed(7)
    t, B, Hq, Hkv, d, T = DT[dtype], 3, 8, 2, 128, 70
    c, plain = (cache(policy, dtype, B=B, d=d) for _ in range(2))
    if split:
        c.set_split(split)
    kp, vp = rnd(g, Hkv, P, d, dtype=t), rnd(g, Hkv, P, d, dtype=t)
    K, V = rnd(g, T, B, Hkv, d, dtype=t), rnd(g, T, B, Hkv, d, dtype=t)
    for i in range(T):
        held = c.slot_positions(0)
        q = rnd(g, B, Hq, d, dtype=t)
        out = c.decode_step_shared(0, q, K[i], V[i], kp, vp)
        plain.decode_step(0, q, K[i], V[i])
        if i % 7 and i < T - 3:
            continue
        keys, values = [], []
        for b in range(B):
            rows = [held[b, h][held[b, h] >= 0].long().tolist() + [i] for h in range(Hkv)]
            keys.append([torch.cat([kp[h], K[rows[h], b, h]]) for h in range(Hkv)])
            values.append([torch.cat([vp[h], V[rows[h], b, h]]) for h in range(Hkv)])
        r, A, m = step_reference(q, keys, values, d ** -0.5)
        kk = torch.cat([kp.reshape(-1, d), K.reshape(-1, d)])
        tol, _ = ref.bounds(t, q.reshape(1, -1, d), kk[None], m, d ** -0.5, r, A, r[..., 0])
        ref.assert_close(out, r, tol, f"step {i}")
    assert torch.equal(c.slot_positions(0), plain.slot_positions(0)) and c.stats()["evictions"] == plain.stats()["evictions"]
    assert c.check() == 0


def test_rotate_uses_the_next_positions(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(9)
    c = cache(SINK_WINDOW, F32)
    f, s = kv.rotary_frequencies(64, scaling="yarn", factor=4.0)
    Q, K, V = rnd(g, 2, 8, 10, 64, dtype=torch.float32), rnd(g, 2, 2, 10, 64, dtype=torch.float32), rnd(g, 2, 2, 10, 64, dtype=torch.float32)
    q0, k0 = Q.clone(), K.clone()
    c.rotate(0, Q, K, f, scale=s, offset=7)
    wq, wk = kv.rotary(q0, k0, 7, f, scale=s)
    assert torch.equal(Q, wq) and torch.equal(K, wk)
    c.prefill(0, K, V)
    q, k, v = rnd(g, 2, 8, 64, dtype=torch.float32), rnd(g, 2, 2, 64, dtype=torch.float32), rnd(g, 2, 2, 64, dtype=torch.float32)
    c.decode_step(0, q, k, v)
    want = kv.rotary(q, k, torch.full((2,), 11, device="cuda"), f)
    got = c.rotate(0, q.clone(), k.clone(), f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_run_of_them_together(cuda_device, dtype):
    """Several answers to one prompt: the prompt is rotated and attended once (batch 1), its keys become the prefix of a
    batch; each step rotates, joins cache and prefix, and is checked against the formula from the unrotated inputs."""
    g = torch.Generator(device="cuda").manual_seed(11)
    t, B, Hq, Hkv, d, P, T = DT[dtype], 4, 8, 2, 64, 150, 12
    f, _ = kv.rotary_frequencies(d)
    Q, K, V = rnd(g, 1, Hq, P, d, dtype=t), rnd(g, 1, Hkv, P, d, dtype=t), rnd(g, 1, Hkv, P, d, dtype=t)
    first = cache(RANDOM, dtype, B=1, max_prompt=P)
    first.rotate(0, Q, K, f)
    out = first.prefill_attend(0, Q, K, V)
    r, l, A = ref.sequence(Q[0], K[0], V[0], 0, None, 0.125)
    tol, _ = ref.bounds(t, Q[0], K[0], P, 0.125, r, A, l)
    ref.assert_close(out[0], r, tol, "prompt")
    c = cache(RANDOM, dtype, B=B, max_prompt=0)
    hist_k, hist_v = [], []
    for i in range(T):
        q, k, v = rnd(g, B, Hq, d, dtype=t), rnd(g, B, Hkv, d, dtype=t), rnd(g, B, Hkv, d, dtype=t)
        c.rotate(0, q, k, f, offset=P)
        got = c.decode_step_shared(0, q, k, v, K[0], V[0])
        hist_k.append(k)
        hist_v.append(v)
        keys = [[torch.cat([K[0, h], torch.stack([x[b, h] for x in hist_k])]) for h in range(Hkv)] for b in range(B)]
        values = [[torch.cat([V[0, h], torch.stack([x[b, h] for x in hist_v])]) for h in range(Hkv)] for b in range(B)]
        r, A, m = step_reference(q, keys, values, 0.125)
        kk = torch.cat([K.reshape(-1, d)] + [x.reshape(-1, d) for x in hist_k])
        tol, _ = ref.bounds(t, q.reshape(1, -1, d), kk[None], m, 0.125, r, A, r[..., 0])
        ref.assert_close(got, r, tol, f"step {i}")
    assert c.check() == 0 and first.check() == 0


def test_refusals(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    t = torch.bfloat16
    Q, K, V = rnd(g, 2, 8, 70, 64, dtype=t), rnd(g, 2, 2, 70, 64, dtype=t), rnd(g, 2, 2, 70, 64, dtype=t)
    q, k, v = rnd(g, 2, 8, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t)
    c = cache(RANDOM, BF16)
    with pytest.raises(KVEvictError) as e:
        c.prefill_attend(0, Q, K, V)            # beyond max_prompt
    assert e.value.code == -2 and c.layer_state(0) == (0, 0, 0)
    with pytest.raises(KVEvictError) as e:
        c.prefill_attend(1, Q[:, :, :9].contiguous(), K[:, :, :9].contiguous(), V[:, :, :9].contiguous())
    assert e.value.code == -3
    c.decode_step(0, q, k, v)
    with pytest.raises(KVEvictError) as e:
        c.prefill_attend(0, Q[:, :, :9].contiguous(), K[:, :, :9].contiguous(), V[:, :, :9].contiguous())
    assert e.value.code == -3
    h = cache(H2O, BF16)
    with pytest.raises(KVEvictError) as e:
        h.decode_step_shared(0, q, k, v, K[0], V[0])  # scores would need the joint softmax
    assert e.value.code == -1 and h.layer_state(0) == (0, 0, 0)
    with pytest.raises(ValueError):
        c.decode_step_shared(0, q, k, v, K[0, :, :5], V[0, :, :5])  # not dense
    with pytest.raises(ValueError):
        c.decode_step_shared(0, q, k, v, K[0], V[0], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        c.rotate(0, q[:1], k, kv.rotary_frequencies(64)[0])


def test_on_the_handles_stream(cuda_device):
    """A handle with a stream of its own, calls made under another current stream, captured and replayed."""
    g = torch.Generator(device="cuda").manual_seed(2)
    s = torch.cuda.Stream()
    c = cache(SINK_WINDOW, BF16, stream=s)
    d = cache(SINK_WINDOW, BF16)
    t = torch.bfloat16
    Q, K, V = rnd(g, 2, 8, 40, 64, dtype=t), rnd(g, 2, 2, 40, 64, dtype=t), rnd(g, 2, 2, 40, 64, dtype=t)
    kp, vp = rnd(g, 2, 500, 64, dtype=t), rnd(g, 2, 500, 64, dtype=t)
    q, k, v = rnd(g, 2, 8, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t), rnd(g, 2, 2, 64, dtype=t)
    torch.cuda.synchronize()
    out = torch.empty_like(Q)
    step = torch.empty_like(q)
    c.prefill_attend(0, Q, K, V, out=out)
    c.decode_step_shared(0, q, k, v, kp, vp, out=step)
    want, want_step = d.prefill_attend(0, Q, K, V), d.decode_step_shared(0, q, k, v, kp, vp)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(step, want_step)
    # captured: the handle's host counters move once a capture, so one replay a capture
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(gr, stream=s):
            c.decode_step_shared(0, q, k, v, kp, vp, out=step)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(step, d.decode_step_shared(0, q, k, v, kp, vp))
