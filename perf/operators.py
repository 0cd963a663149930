"""Operators around the decode step, as a user's program calls them, with their plain forms.

- attention: `window_attention`, a prompt's (or a chunk's, or a single token's) attention in which a query sees the
  newest `window` keys up to its own position and the first `n_sink` keys; no window means all keys up to its position.
- shared: `shared_prefix_attention`, one token of every sequence over a prefix that all sequences share and a suffix of
  its own.
- rotary: `rotary`, the rotation of queries and keys by their positions.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- cases
def attention(name, dtype, form, batch, q_heads, kv_heads, head_dim, n, m, n_sink, window, ragged, lens_seed=1):
    """n queries (at most, where ragged) of every sequence at the end of m keys; window 0: none."""
    return {"name": name, "op": "attention", "dtype": dtype, "form": form, "batch": batch, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "n": n, "m": m, "n_sink": n_sink, "window": window,
            "ragged": ragged, "lens_seed": lens_seed}


def shared(name, dtype, batch, q_heads, kv_heads, head_dim, prefix, m, lens_seed=1):
    return {"name": name, "op": "shared", "dtype": dtype, "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "prefix": prefix, "m": m, "lens_seed": lens_seed}


def rotation(name, dtype, form, batch, tokens, q_heads, kv_heads, head_dim, rotary_dim, interleaved, factor, far, inverse):
    """form "tokens": [tokens][heads][d]; "heads": [batch][heads][tokens][d]. far: the largest position."""
    return {"name": name, "op": "rotary", "dtype": dtype, "form": form, "batch": batch, "tokens": tokens,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary_dim": rotary_dim,
            "interleaved": interleaved, "factor": factor, "far": far, "inverse": inverse}


def listed():
    return [
        # a small fp32 prompt in the shape of the smallest workload (8 heads of 64, 4 sinks, 64 recent tokens)
        attention("prompt_fp32_small", "fp32", "padded", 1, 8, 8, 64, 256, 256, 4, 65, False),
        # a StreamingLLM prompt, 32 MHA heads, 4 sinks and the 1020 tokens the cache keeps besides the new one
        attention("prompt_stream_mha", "bf16", "padded", 2, 32, 32, 128, 4096, 4096, 4, 1021, False),
        # the kept prompt of the long-reasoning workload: plain causal attention, 32 query heads over 8 KV heads
        attention("prompt_causal_gqa", "bf16", "padded", 1, 32, 8, 128, 8192, 8192, 0, 0, False),
        # a serving batch of packed prompts of uneven lengths, heads of 64
        attention("prompt_packed_ragged", "bf16", "packed", 13, 16, 4, 64, 1777, 1777, 4, 509, True),
        # one new token of each of 32 long sequences, 4 sinks and a window of 2044
        attention("step_window_gqa", "bf16", "padded", 32, 64, 8, 128, 1, 32768, 4, 2044, True),
        # five drafted tokens of a few sequences of odd lengths, all keys visible
        attention("step_drafted", "bf16", "padded", 3, 32, 8, 128, 5, 7777, 0, 0, True),
        # a few answers to a short common prompt, early in their decode: the launch is what costs
        shared("shared_small", "bf16", 4, 8, 8, 64, 250, 40),
        # 32 reasoning traces of one 8192-token prompt, 2048 + 128 kept tokens each
        shared("shared_reasoning", "bf16", 32, 32, 8, 128, 8192, 2176),
        # 64 sequences behind a 32768-token document, 64 query heads over 8 KV heads
        shared("shared_document", "bf16", 64, 64, 8, 128, 32768, 2048),
        # one decode step's queries and keys, 64 sequences at positions of their own
        rotation("rotary_step", "bf16", "tokens", 1, 64, 32, 32, 128, 128, False, 1.0, 16384, False),
        # a packed batch of prompts, 64 query heads over 8 KV heads, frequencies scaled for a longer context
        rotation("rotary_prompt", "bf16", "tokens", 1, 16384, 64, 8, 128, 128, False, 4.0, 131072, False),
        # gradients of fp32 queries and keys by head, a part of each head, neighbouring pairs, far positions
        rotation("rotary_partial_grad", "fp32", "heads", 3, 2049, 12, 4, 128, 48, True, 1.0, 1000003, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "shared", "rotary"])
    seed = rng.randrange(1 << 30)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128])
    if op == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
        window = rng.choice([0, _log(rng, 1, 4096), _log(rng, 16, 2048)])
        n_sink = rng.choice([0, 1, 4, rng.randrange(0, 200)])
        form = rng.choice(["padded", "packed", "step"])
        if form == "step":
            batch, n, m = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 3, 7]), _log(rng, 16, 32768)
            while batch * kv_heads * m > 1 << 20:
                batch, m = max(1, batch // 2), max(16, m * 3 // 4)
            c = attention("", dtype, "padded", batch, kv_heads * group, kv_heads, d, n, max(n, m), n_sink, window, True, seed)
        else:
            most = 2048 if dtype == "fp32" else 8192
            batch, n = _log(rng, 1, 16), _log(rng, 1, most)
            m = n + rng.choice([0, 0, _log(rng, 1, 1024)])
            while batch * kv_heads * group * n * m > (1 << (27 if dtype == "fp32" else 29)):
                if batch > 1:
                    batch //= 2
                else:
                    n, m = n * 3 // 4, m * 3 // 4 + 1
            c = attention("", dtype, form, batch, kv_heads * group, kv_heads, d, n, m, n_sink, window,
                          form == "packed" or rng.random() < 0.5, seed)
    elif op == "shared":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        batch, prefix, m = _log(rng, 1, 64), _log(rng, 1, 32768), _log(rng, 1, 2048)
        if dtype == "fp32":
            prefix = max(1, prefix // 8)
        c = shared("", dtype, batch, kv_heads * group, kv_heads, d, prefix, m, seed)
    else:
        kv_heads, group = _log(rng, 1, 8), rng.choice([1, 2, 4, 8])
        form = rng.choice(["tokens", "heads"])
        batch, tokens = (1, _log(rng, 1, 16384)) if form == "tokens" else (_log(rng, 1, 8), _log(rng, 1, 2048))
        c = rotation("", dtype, form, batch, tokens, kv_heads * group, kv_heads, d, rng.choice([d, d, d // 2, 16, 48, 10]),
                     rng.random() < 0.5, rng.choice([1.0, 1.0, 4.0, 32.0]), max(tokens * 2, _log(rng, 1024, 1 << 20)), rng.random() < 0.3)
    del c["name"]
    return c


def lengths(c):
    """Every sequence's queries and keys, from the case alone."""
    r = random.Random(c["lens_seed"])
    if c["op"] == "shared":
        return [1] * c["batch"], [r.randint(max(0, c["m"] // 2), c["m"]) for _ in range(c["batch"])]
    n, m, batch = c["n"], c["m"], c["batch"]
    if not c["ragged"]:
        return [n] * batch, [m] * batch
    if c["form"] == "padded":
        return [n] * batch, [r.randint(max(1, m // 2), m) for _ in range(batch)]
    ql = [r.randint(1, n) for _ in range(batch)]
    ql[0] = n
    if batch > 2:
        ql[2] = 0  # a sequence with nothing to do in this batch
    return ql, [q + r.randint(0, m - n) for q in ql]


# ------------------------------------------------------------------------------------------------------ inputs
def frequencies(c):
    """The angle per position of every pair of a head, base 10000; with a factor, the slow pairs (those that turn less
    than once in 4096 positions) are slowed by it and the fast ones are not, the ones between in proportion."""
    half = c["rotary_dim"] // 2
    f = 10000.0 ** (-np.arange(half, dtype=np.float64) * 2 / c["rotary_dim"])
    if c["factor"] != 1.0:
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    return f


def magnitude(c):
    return 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=t)

    if c["op"] == "rotary":
        if c["form"] == "tokens":
            q, k = normal(c["tokens"], c["q_heads"], c["head_dim"]), normal(c["tokens"], c["kv_heads"], c["head_dim"])
            pos = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=DEV, dtype=torch.int64)
        else:
            q = normal(c["batch"], c["q_heads"], c["tokens"], c["head_dim"])
            k = normal(c["batch"], c["kv_heads"], c["tokens"], c["head_dim"])
            start = torch.randint(0, c["far"] - c["tokens"], (c["batch"], 1), generator=g, device=DEV, dtype=torch.int64)
            pos = start + torch.arange(c["tokens"], device=DEV)
        return {"c": c, "q": q, "k": k, "pos": pos, "inv_freq": torch.tensor(frequencies(c), device=DEV), "scale": magnitude(c)}
    ql, kl = lengths(c)
    # trained heads send a good part of their attention to the first tokens: a common direction of all queries
    lean = torch.randn(c["head_dim"], generator=g, device=DEV, dtype=torch.float32) * 0.4
    if c["op"] == "shared":
        q = normal(c["batch"], c["q_heads"], c["head_dim"]) + lean.to(t)
        kp, vp = normal(c["kv_heads"], c["prefix"], c["head_dim"]), normal(c["kv_heads"], c["prefix"], c["head_dim"])
        kp[:, :4] += lean.to(t)
        k, v = (normal(c["batch"], c["kv_heads"], c["m"], c["head_dim"]) for _ in range(2))
        return {"c": c, "q": q, "kp": kp, "vp": vp, "k": k, "v": v, "lens": torch.tensor(kl, device=DEV, dtype=torch.int32)}
    s = {"c": c, "window": c["window"] or None}
    if c["form"] == "padded":
        q = normal(c["batch"], c["q_heads"], c["n"], c["head_dim"])
        k, v = (normal(c["batch"], c["kv_heads"], c["m"], c["head_dim"]) for _ in range(2))
        k[:, :, :max(1, c["n_sink"])] += lean.to(t)
        s["kv_lens"] = torch.tensor(kl, device=DEV, dtype=torch.int32) if c["ragged"] else None
    else:
        q = normal(sum(ql), c["q_heads"], c["head_dim"])
        k, v = (normal(sum(kl), c["kv_heads"], c["head_dim"]) for _ in range(2))
        for name, lens in (("q_starts", ql), ("k_starts", kl)):
            s[name] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=DEV, dtype=torch.int32)
        first = s["k_starts"][:-1].long()
        k[first[first < k.shape[0]]] += lean.to(t)
    q += lean.to(t)
    return {**s, "q": q, "k": k, "v": v}


# --------------------------------------------------------------------------------------------------- the passes
def softmax_times(z, visible, v):
    """softmax over the visible keys, times v; and the log of the sum. Rows that see nothing: 0 and -inf."""
    z = z.masked_fill(~visible, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (top + torch.log(total)).squeeze(-1)


def plain_attention(q, k, v, q_len, k_len, n_sink, window):
    """q [B][Hq][N][d], k and v [B][Hkv][M][d], q_len and k_len [B]: fp32 [B][Hq][N][d] and [B][Hq][N]."""
    B, Hq, N, d = q.shape
    Hkv, M = k.shape[1], k.shape[2]
    z = (q.float() * d ** -0.5).reshape(B, Hkv, Hq // Hkv * N, d) @ k.float().transpose(2, 3)
    i, j = torch.arange(N, device=DEV), torch.arange(M, device=DEV)
    p = (k_len - q_len)[:, None] + i
    visible = (j <= p[..., None]) & (j < k_len[:, None, None])
    if window:
        visible &= (j < n_sink) | (j > p[..., None] - window)
    visible = visible[:, None, None].expand(B, Hkv, Hq // Hkv, N, M).reshape(B, Hkv, Hq // Hkv * N, M)
    out, lse = softmax_times(z, visible, v.float())
    return out.view(B, Hq, N, d), lse.view(B, Hq, N)


def run(s):
    c = s["c"]
    if own:
        import kv_cache_eviction_decode_gb300 as kv

        if c["op"] == "rotary":
            return kv.rotary(s["q"], s["k"], s["pos"], s["inv_freq"], interleaved=c["interleaved"], scale=s["scale"],
                             inverse=c["inverse"])
        if c["op"] == "shared":
            return kv.shared_prefix_attention(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], return_lse=True)
        if c["form"] == "padded":
            return kv.window_attention(s["q"], s["k"], s["v"], n_sink=c["n_sink"], window=s["window"],
                                       kv_lens=s["kv_lens"], return_lse=True)
        return kv.window_attention(s["q"], s["k"], s["v"], n_sink=c["n_sink"], window=s["window"],
                                   q_starts=s["q_starts"], k_starts=s["k_starts"], max_q=c["n"], max_k=c["m"],
                                   return_lse=True)
    t = s["q"].dtype
    if c["op"] == "rotary":
        return plain_rotary(s, s["q"]), plain_rotary(s, s["k"])
    if c["op"] == "shared":
        B, Hq, d = s["q"].shape
        Hkv, P, G, M = c["kv_heads"], c["prefix"], c["q_heads"] // c["kv_heads"], c["m"]
        q = (s["q"].float() * d ** -0.5).view(B, Hkv, G, d)
        kp, vp = s["kp"].float(), s["vp"].float()
        zp = (q.transpose(0, 1).reshape(Hkv, B * G, d) @ kp.transpose(1, 2)).view(Hkv, B, G, P).transpose(0, 1)
        zs = q @ s["k"].float().transpose(2, 3)
        zs = zs.masked_fill((torch.arange(M, device=DEV) >= s["lens"][:, None])[:, None, None], -math.inf)
        top = torch.maximum(zp.amax(-1, keepdim=True), zs.amax(-1, keepdim=True))
        ep, es = torch.exp(zp - top), torch.exp(zs - top)
        total = ep.sum(-1, keepdim=True) + es.sum(-1, keepdim=True)
        over_prefix = (ep.transpose(0, 1).reshape(Hkv, B * G, P) @ vp).view(Hkv, B, G, d).transpose(0, 1)
        out = (over_prefix + es @ s["v"].float()) / total
        return out.reshape(B, Hq, d).to(t), (top + torch.log(total)).view(B, Hq)
    if c["form"] == "padded":
        B, M = c["batch"], c["m"]
        k_len = torch.full((B,), M, device=DEV) if s["kv_lens"] is None else s["kv_lens"]
        out, lse = plain_attention(s["q"], s["k"], s["v"], torch.full_like(k_len, c["n"]), k_len, c["n_sink"], c["window"])
        return out.to(t), lse
    # packed: gathered into rows of one length, and back
    qs, ks = s["q_starts"].long(), s["k_starts"].long()
    ql, kl = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    qi, ki = torch.arange(c["n"], device=DEV), torch.arange(c["m"], device=DEV)
    at = (ks[:-1, None] + ki).clamp(max=max(0, s["k"].shape[0] - 1))
    q = s["q"][(qs[:-1, None] + qi).clamp(max=max(0, s["q"].shape[0] - 1))].transpose(1, 2)
    k, v = s["k"][at].transpose(1, 2), s["v"][at].transpose(1, 2)
    out, lse = plain_attention(q, k, v, ql, kl, c["n_sink"], c["window"])
    real = qi < ql[:, None]
    return out.transpose(1, 2)[real].to(t), lse.transpose(1, 2)[real]


def plain_rotary(s, x):
    c, R = s["c"], s["c"]["rotary_dim"]
    angle = s["pos"].double()[..., None] * s["inv_freq"]
    if c["inverse"]:
        angle = -angle
    head = 1 if c["form"] == "tokens" else -3
    cos, sin = ((f(angle) * s["scale"]).float().unsqueeze(head) for f in (torch.cos, torch.sin))
    y = x.float()
    turned, rest = y[..., :R], y[..., R:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :R // 2], turned[..., R // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


# ------------------------------------------------------------------------------------------- what a pass cannot do without
def seen(c, ql, kl):
    """Visible (query, key) pairs of one head, and the keys that any query of a sequence sees, over all sequences."""
    pairs = keys = 0
    for n, m in zip(ql, kl):
        p = np.arange(max(0, m - n), m, dtype=np.int64)
        if c["window"]:
            near = np.minimum(p + 1, c["window"])
            pairs += int((near + np.minimum(c["n_sink"], p + 1 - near)).sum())
            first = max(0, max(0, m - n) - c["window"] + 1)
            keys += m - first + min(c["n_sink"], first) if len(p) else 0
        else:
            pairs += int((p + 1).sum())
            keys += m if len(p) else 0
    return pairs, keys


def work(c):
    e, d = (2 if c["dtype"] == "bf16" else 4), c["head_dim"]
    if c["op"] == "rotary":
        n = c["batch"] * c["tokens"]
        values = n * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 2 * values * d * e + 8 * n, "flops": 3 * values * c["rotary_dim"]}
    ql, kl = lengths(c)
    if c["op"] == "shared":
        B = c["batch"]
        pairs = B * c["prefix"] + sum(kl)
        return {"bytes": 2 * c["kv_heads"] * d * e * (c["prefix"] + sum(kl)) + B * c["q_heads"] * (2 * d * e + 4) + 4 * B,
                "flops": 4 * d * c["q_heads"] * pairs}
    pairs, keys = seen(c, ql, kl)
    return {"bytes": sum(ql) * c["q_heads"] * (2 * d * e + 4) + 2 * keys * c["kv_heads"] * d * e,
            "flops": 4 * d * c["q_heads"] * pairs}


# ------------------------------------------------------------------------------------- the definitions, in 64 bits
def exact_rows(q, k, v, first, n_sink, window):
    """q [H][n][d] at positions first.., k and v [H][m][d], all fp64, a block of queries at a time over the keys that one
    of them can see."""
    H, n, d = q.shape
    out = torch.zeros(H, n, d, dtype=torch.float64, device=DEV)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=DEV)
    for i0 in range(0, n, 256):
        i1 = min(n, i0 + 256)
        last = min(first + i1 - 1, k.shape[1] - 1)
        if last < 0:
            continue
        low = max(0, first + i0 - window + 1) if window else 0
        cols = torch.cat([torch.arange(0, min(n_sink, low), device=DEV), torch.arange(low, last + 1, device=DEV)])
        pos = first + torch.arange(i0, i1, device=DEV)
        z = torch.einsum("hid,hjd->hij", q[:, i0:i1], k[:, cols]) / math.sqrt(d)
        dead = cols > pos[:, None]
        if window:
            dead |= (cols >= n_sink) & (cols <= pos[:, None] - window)
        z = z + torch.zeros_like(z).masked_fill(dead, -math.inf)
        s = torch.logsumexp(z, -1)
        w = torch.exp(z - s[..., None])
        w = torch.where(dead.all(-1)[:, None], torch.zeros_like(w), w)
        out[:, i0:i1] = torch.einsum("hij,hjd->hid", w, v[:, cols])
        lse[:, i0:i1] = s
    return out, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        return [exact_rotary(s, s["q"].double()), exact_rotary(s, s["k"].double())]
    ql, kl = lengths(c)
    G = c["q_heads"] // c["kv_heads"]
    if c["op"] == "shared":
        outs, sums = [], []
        for b in range(c["batch"]):
            k = torch.cat([s["kp"], s["k"][b, :, :kl[b]]], 1).double()
            v = torch.cat([s["vp"], s["v"][b, :, :kl[b]]], 1).double()
            z = torch.einsum("hgd,hjd->hgj", s["q"][b].double().view(-1, G, c["head_dim"]), k) / math.sqrt(c["head_dim"])
            lse = torch.logsumexp(z, -1)
            outs.append(torch.einsum("hgj,hjd->hgd", torch.exp(z - lse[..., None]), v).flatten(0, 1))
            sums.append(lse.flatten())
        return [torch.stack(outs), torch.stack(sums)]
    outs, sums, q0, k0 = [], [], 0, 0
    for b, (n, m) in enumerate(zip(ql, kl)):
        if c["form"] == "padded":
            q, k, v = s["q"][b], s["k"][b, :, :m], s["v"][b, :, :m]
        else:
            q, k, v = (x[i:i + w].transpose(0, 1) for x, i, w in ((s["q"], q0, n), (s["k"], k0, m), (s["v"], k0, m)))
            q0, k0 = q0 + n, k0 + m
        parts = [exact_rows(q[h * G:(h + 1) * G].double(), k[h:h + 1].double().expand(G, -1, -1),
                            v[h:h + 1].double().expand(G, -1, -1), m - n, c["n_sink"], c["window"]) for h in range(c["kv_heads"])]
        outs.append(torch.cat([p[0] for p in parts]))
        sums.append(torch.cat([p[1] for p in parts]))
    if c["form"] == "padded":
        return [torch.stack(outs), torch.stack(sums)]
    return [torch.cat([o.transpose(0, 1) for o in outs]), torch.cat([x.t() for x in sums])]


def exact_rotary(s, x):
    """Each pair as a complex number, times scale e^(+-i angle)."""
    c, R = s["c"], s["c"]["rotary_dim"]
    angle = s["pos"].double().unsqueeze(-1) * s["inv_freq"].double()
    turn = torch.polar(torch.full_like(angle, s["scale"]), -angle if c["inverse"] else angle)
    turn = turn.unsqueeze(1)  # the heads' axis, in both forms
    y = x.clone()
    if c["interleaved"]:
        pairs = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous())
        y[..., :R] = torch.view_as_real(pairs * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y
