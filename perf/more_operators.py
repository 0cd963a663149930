"""A paged cache, what is written into it and what reads it, as a user's program calls it, with the plain forms.

- norm: `norm_rotary`, the root-mean-square norm of every head of queries and keys, then their rotation by positions.
- append: `paged_append`, new keys (turned by their positions on the way) and values into the pages of their sequences.
- gather: `paged_gather`, the keys and values of whole sequences out of their pages, as attention over a prompt's next
  chunk takes them.
- attention: `paged_attention`, a few tokens of every sequence over its pages.

Pages hold the keys' own type, or 4 bits a channel ("q4"): every 32 channels of a token and head have a base and a step in
bf16, and a channel is base + (code - 8) * step, code 0 .. 15.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- cases
def norm(name, dtype, form, batch, tokens, q_heads, kv_heads, head_dim, rotary_dim, interleaved, far):
    """form "tokens": [tokens][heads][d]; "heads": [batch][heads][tokens][d]. far: positions are below it."""
    return {"name": name, "op": "norm", "dtype": dtype, "form": form, "batch": batch, "tokens": tokens, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rotary_dim": rotary_dim, "interleaved": interleaved, "far": far}


def append(name, dtype, pages, batch, kv_heads, head_dim, page, new, m, rotary_dim, interleaved, ragged, read, lens_seed=1):
    """`new` tokens (at most, where ragged) of every sequence, which then has up to m; pages "own" or "q4"; rotary_dim 0:
    keys as they are. read: and the sequences read back out of the pages."""
    return {"name": name, "op": "append", "dtype": dtype, "pages": pages, "batch": batch, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "new": new, "m": m, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "ragged": ragged, "read": read, "lens_seed": lens_seed}


def gather(name, dtype, pages, form, batch, kv_heads, head_dim, page, m, lens_seed=1):
    """form "padded": [batch][heads][m][d]; "packed": [tokens][heads][d]."""
    return {"name": name, "op": "gather", "dtype": dtype, "pages": pages, "form": form, "batch": batch, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "m": m, "lens_seed": lens_seed}


def attention(name, dtype, pages, batch, q_heads, kv_heads, head_dim, page, new, m, n_sink, window, ragged, lens_seed=1):
    """`new` tokens (at most, where ragged) at the end of every sequence's up to m; window 0: none."""
    return {"name": name, "op": "attention", "dtype": dtype, "pages": pages, "batch": batch, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "new": new, "m": m, "n_sink": n_sink,
            "window": window, "ragged": ragged, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step's queries and keys, 64 sequences at positions of their own, 32 heads over 8
        norm("norm_step", "bf16", "tokens", 1, 64, 32, 8, 128, 128, False, 16384),
        # a packed batch of prompts, 64 query heads over 8 KV heads
        norm("norm_prompt", "bf16", "tokens", 1, 16384, 64, 8, 128, 128, False, 131072),
        # fp32 queries and keys by head, a part of each head turned, neighbouring pairs, far positions
        norm("norm_partial", "fp32", "heads", 3, 2049, 12, 4, 128, 48, True, 1000003),
        # one new token of each of 64 sequences into pages of 16
        append("append_step", "bf16", "own", 64, 8, 128, 16, 1, 4096, 128, False, False, False),
        # a serving batch of uneven prompts, into pages of 64
        append("append_prompt", "bf16", "own", 13, 8, 128, 64, 4097, 8192, 128, False, True, False),
        # the next chunk of a few long prompts into 4-bit pages, and the sequences read back for the chunk's attention
        append("append_q4_chunk", "bf16", "q4", 8, 8, 128, 16, 512, 8192, 128, False, True, True),
        # whole 4-bit sequences, padded to the longest
        gather("gather_q4", "bf16", "q4", "padded", 16, 8, 128, 32, 16384),
        # a few sequences of odd lengths, heads of 64, one behind the other
        gather("gather_packed", "bf16", "own", "packed", 5, 4, 64, 16, 1777),
        # a few short answers, early in their decode, 8 heads of 64: the launch is what costs
        attention("attend_q4_small", "bf16", "q4", 4, 8, 8, 64, 16, 1, 300, 0, 0, False),
        # a decode step of 32 long 4-bit sequences, 64 query heads over 8 KV heads
        attention("attend_q4_long", "bf16", "q4", 32, 64, 8, 128, 16, 1, 32768, 0, 0, False),
        # five drafted tokens of 16 sequences, 4 sinks and a window of 2044, 4-bit pages of 32
        attention("attend_q4_drafted", "bf16", "q4", 16, 32, 8, 128, 32, 5, 32768, 4, 2044, True),
        # a decode step over bf16 pages, 32 query heads over 8 KV heads
        attention("attend_bf16", "bf16", "own", 32, 32, 8, 128, 64, 1, 10240, 0, 0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "gather", "attention", "attention", "attention"])
    seed = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    kv_heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    page = rng.choice([16, 16, 32, 64, 128])
    kind = rng.choice(["q4", "q4", "q4", "bf16", "bf16", "fp32"])
    dtype, pages = ("bf16", "q4") if kind == "q4" else (kind, "own")
    if op == "norm":
        form = rng.choice(["tokens", "heads"])
        batch, tokens = (1, _log(rng, 1, 16384)) if form == "tokens" else (_log(rng, 1, 8), _log(rng, 1, 2048))
        c = norm("", rng.choice(["bf16", "bf16", "fp32"]), form, batch, tokens, min(64, kv_heads * group), min(8, kv_heads), d,
                 rng.choice([d, d, d // 2, 16, 48, 10]), rng.random() < 0.4, max(tokens * 2, _log(rng, 1024, 1 << 20)))
    elif op == "append":
        batch, new = _log(rng, 1, 64), rng.choice([1, 1, 3, _log(rng, 1, 4096)])
        while batch * new * kv_heads > 1 << 18:
            batch, new = max(1, batch // 2), max(1, new * 3 // 4)
        m = new + _log(rng, 1, 4096)
        while batch * m * kv_heads > 1 << 20:
            m = max(new, m // 2)
            if m == new:
                break
        c = append("", dtype, pages, batch, kv_heads, d, page, new, m, rng.choice([0, d, d, d // 2, 16]), rng.random() < 0.3,
                   rng.random() < 0.5, pages == "q4", seed)
    elif op == "gather":
        batch, m = _log(rng, 1, 32), _log(rng, 1, 16384)
        while batch * m * kv_heads > 1 << 20:
            batch, m = max(1, batch // 2), max(1, m * 3 // 4)
        c = gather("", dtype, pages, rng.choice(["padded", "packed"]), batch, kv_heads, d, page, m, seed)
    else:
        batch, new, m = _log(rng, 1, 64), rng.choice([1, 1, 1, 1, 2, 3, 5, 8]), _log(rng, 1, 32768)
        most = 1 << (18 if dtype == "fp32" else 21)
        while batch * kv_heads * m * max(8, new * group) > 8 * most:
            batch, m = max(1, batch // 2), max(1, m * 3 // 4)
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        c = attention("", dtype, pages, batch, kv_heads * group, kv_heads, d, page, new, max(new, m),
                      rng.choice([0, 1, 4, rng.randrange(0, 200)]), window, rng.random() < 0.4, seed)
    del c["name"]
    return c


def lengths(c):
    """Every sequence's new tokens and tokens in all, from the case alone."""
    r = random.Random(c["lens_seed"])
    kl = [r.randint(max(1, c["m"] // 2), c["m"]) for _ in range(c["batch"])]
    if c["op"] == "gather":
        kl[0] = c["m"]
        return [0] * c["batch"], kl
    if not c["ragged"]:
        return [c["new"]] * c["batch"], [max(k, c["new"]) for k in kl]
    nl = [r.randint(1, c["new"]) for _ in range(c["batch"])]
    nl[0] = c["new"]
    if c["batch"] > 2:
        nl[2] = 0  # a sequence with nothing to do in this batch
    return nl, [max(k, n) for k, n in zip(kl, nl)]


# ------------------------------------------------------------------------------------------------------ inputs
def frequencies(rotary_dim):
    """The angle per position of every pair of a head, base 10000."""
    half = rotary_dim // 2
    return torch.tensor(10000.0 ** (-np.arange(half, dtype=np.float64) * 2 / rotary_dim), device=DEV)


def four_bit(x):
    """x [...][d] to (codes as whole numbers [...][d], base and step [...][d/32] in bf16). The base is the value nearest
    8/15 of the way up, the step the least that reaches both ends from it, rounded up."""
    x = x.unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    base = (hi * (8 / 15) + lo * (7 / 15)).to(torch.bfloat16)
    b = base.to(x.dtype)
    step = torch.maximum((hi - b) / 7, (b - lo) / 8).float()
    step = ((step.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    by = torch.where(step > 0, step, torch.ones_like(step)).to(x.dtype)
    code = torch.round((x - b[..., None]) / by[..., None]) + 8
    return code.clamp(0, 15).to(torch.uint8).flatten(-2), base, step.to(torch.bfloat16)


def parts(pages, d):
    """The codes [pages][heads][page][d/2] and the bases and steps [pages][heads][page][d/32][2] of 4-bit pages: in a
    page, a head's codes of all tokens come first."""
    page = pages.shape[2]
    flat = pages.flatten(2)
    return (flat[..., :page * d // 2].unflatten(-1, (page, d // 2)),
            flat[..., page * d // 2:].unflatten(-1, (page, d // 8)).view(torch.bfloat16).unflatten(-1, (d // 32, 2)))


def codes_to_bytes(code):
    """Channel 32 j + 4 g + i of a row is in byte (d / 16) g + 2 j + i / 2, the even ones in the low half."""
    d = code.shape[-1]
    c = code.unflatten(-1, (d // 32, 8, 4)).transpose(-3, -2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-3)


def bytes_to_codes(b):
    d = 2 * b.shape[-1]
    c = torch.stack([b & 15, b >> 4], -1).unflatten(-2, (8, d // 32, 2)).flatten(-2)
    return c.transpose(-3, -2).flatten(-3)


def values(code_bytes, base_step):
    """What rows of 4-bit pages stand for, in fp32."""
    u = bytes_to_codes(code_bytes).float().unflatten(-1, (-1, 32)) - 8
    p = base_step.float()
    return (p[..., 0:1] + u * p[..., 1:2]).flatten(-2)


def pool(c, g, n_pages):
    """Pages full of keys or values."""
    t, H, S, d = TYPES[c["dtype"]], c["kv_heads"], c["page"], c["head_dim"]
    if c["pages"] == "own":
        return torch.randn((n_pages, H, S, d), generator=g, device=DEV, dtype=t)
    out = torch.empty((n_pages, H, S, 5 * d // 8), device=DEV, dtype=torch.uint8)
    codes, base_step = parts(out, d)
    some = max(1, (1 << 26) // (H * S * d))
    for i in range(0, n_pages, some):
        x = torch.randn((min(some, n_pages - i), H, S, d), generator=g, device=DEV)
        code, base, step = four_bit(x)
        codes[i:i + some] = codes_to_bytes(code)
        base_step[i:i + some] = torch.stack([base, step], -1)
    return out


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    t, d, Hkv = TYPES[c["dtype"]], c["head_dim"], c["kv_heads"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=t)

    def int32(x):
        return torch.tensor(np.asarray(x), device=DEV, dtype=torch.int32)

    if c["op"] == "norm":
        if c["form"] == "tokens":
            q, k = normal(c["tokens"], c["q_heads"], d), normal(c["tokens"], Hkv, d)
            pos = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=DEV, dtype=torch.int64)
        else:
            q, k = normal(c["batch"], c["q_heads"], c["tokens"], d), normal(c["batch"], Hkv, c["tokens"], d)
            start = torch.randint(0, c["far"] - c["tokens"], (c["batch"], 1), generator=g, device=DEV, dtype=torch.int64)
            pos = start + torch.arange(c["tokens"], device=DEV)
        wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t), (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t)
        return {"c": c, "q": q * 3, "k": k * 2, "wq": wq, "wk": wk, "pos": pos, "inv_freq": frequencies(c["rotary_dim"])}
    nl, kl = lengths(c)
    S = c["page"]
    width = -(-c["m"] // S)
    used = [-(-k // S) for k in kl]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["batch"], width), -1, device=DEV, dtype=torch.int32)  # entries that no token needs name no page
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    s = {"c": c, "kp": pool(c, g, n_pages), "vp": pool(c, g, n_pages), "table": table, "lens": int32(kl),
         "starts": int32(np.concatenate([[0], np.cumsum(nl)]))}
    if c["op"] == "append":
        s["k"], s["v"] = normal(sum(nl), Hkv, d), normal(sum(nl), Hkv, d)
        s["inv_freq"] = frequencies(c["rotary_dim"]) if c["rotary_dim"] else None
    if c["op"] == "gather" or (c["op"] == "append" and c["read"]):
        if c.get("form") == "packed":
            s["k_starts"] = int32(np.concatenate([[0], np.cumsum(kl)]))
            shape = (sum(kl), Hkv, d)
        else:
            s["k_starts"], shape = None, (c["batch"], Hkv, c["m"], d)
        s["k_out"], s["v_out"] = torch.zeros(shape, device=DEV, dtype=t), torch.zeros(shape, device=DEV, dtype=t)
    if c["op"] == "attention":
        # trained heads send a good part of their attention to the first tokens: a common direction of queries and first keys
        lean = torch.randn(d, generator=g, device=DEV) * 0.4
        first = table[:, 0].long()
        if c["pages"] == "own":
            s["kp"][first, :, :4] += lean.to(t)
        else:
            code, base, step = four_bit(torch.randn((c["batch"], Hkv, 4, d), generator=g, device=DEV) + lean)
            codes, base_step = parts(s["kp"], d)
            codes[first, :, :4] = codes_to_bytes(code)
            base_step[first, :, :4] = torch.stack([base, step], -1)
        s["q"] = normal(sum(nl), c["q_heads"], d) + lean.to(t)
        s["window"] = c["window"] or None
    return s


# --------------------------------------------------------------------------------------------------- the passes
def turned(x, pos, inv_freq, interleaved, head):
    """x in fp32 (or fp64) turned by its positions; `head`: where the heads' axis goes among the angles."""
    R = 2 * inv_freq.shape[0]
    angle = pos.double()[..., None] * inv_freq
    cos, sin = (f(angle).to(x.dtype).unsqueeze(head) for f in (torch.cos, torch.sin))
    y, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, rest], -1)


def plain_norm(s, x, w):
    c = s["c"]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return turned(y, s["pos"], s["inv_freq"], c["interleaved"], 1 if c["form"] == "tokens" else -3).to(x.dtype)


def places(s):
    """Of every new token: its sequence and its index in it."""
    starts = s["starts"].long()
    t = torch.arange(s["k"].shape[0], device=DEV)
    b = torch.searchsorted(starts[1:], t, right=True)
    return b, s["lens"].long()[b] - starts[b + 1] + t


def plain_append(s):
    c, S = s["c"], s["c"]["page"]
    b, pos = places(s)
    page, slot = s["table"][b, pos // S].long()[:, None], (pos % S)[:, None]
    heads = torch.arange(c["kv_heads"], device=DEV)[None]
    # (codes are whole numbers: a value next to a border is taken in 64 bits)
    k = s["k"].double() if c["pages"] == "q4" else s["k"].float()
    if c["rotary_dim"]:
        k = turned(k, pos, s["inv_freq"], c["interleaved"], 1)
    if c["pages"] == "own":
        s["kp"][page, heads, slot] = k.to(s["kp"].dtype)
        s["vp"][page, heads, slot] = s["v"]
        return
    for pages, x in ((s["kp"], k), (s["vp"], s["v"].double())):
        code, base, step = four_bit(x)
        codes, base_step = parts(pages, c["head_dim"])
        codes[page, heads, slot] = codes_to_bytes(code)
        base_step[page, heads, slot] = torch.stack([base, step], -1)


def rows_of(pages, c, page, slot):
    """Rows of pages as fp32: page and slot [...], result [...][heads][d]."""
    if c["pages"] == "own":
        return pages[page, :, slot].float()
    codes, base_step = parts(pages, c["head_dim"])
    return values(codes[page, :, slot], base_step[page, :, slot])


def plain_gather(s):
    c, S, lens = s["c"], s["c"]["page"], s["lens"].long()
    if s["k_starts"] is not None:
        starts = s["k_starts"].long()
        t = torch.arange(s["k_out"].shape[0], device=DEV)
        b = torch.searchsorted(starts[1:], t, right=True)
        i = t - starts[b]
        page = s["table"][b, i // S].long()
        for out, pages in ((s["k_out"], s["kp"]), (s["v_out"], s["vp"])):
            out.copy_(rows_of(pages, c, page, i % S))
        return
    i = torch.arange(c["m"], device=DEV)
    page, real = s["table"][:, i // S].long().clamp(min=0), i < lens[:, None]
    for out, pages in ((s["k_out"], s["kp"]), (s["v_out"], s["vp"])):
        x = rows_of(pages, c, page, (i % S).expand_as(page)).transpose(1, 2)
        out.copy_(torch.where(real[:, None, :, None], x.to(out.dtype), out))


def plain_attention(s):
    c, q, S = s["c"], s["q"], s["c"]["page"]
    B, Hq, Hkv, d, N, M = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["new"], c["m"]
    starts, m = s["starts"].long(), s["lens"].long()
    n = starts[1:] - starts[:-1]
    i, j = torch.arange(N, device=DEV), torch.arange(M, device=DEV)
    page = s["table"][:, j // S].long().clamp(min=0)
    k, v = (rows_of(x, c, page, (j % S).expand_as(page)).transpose(1, 2) for x in (s["kp"], s["vp"]))  # [B][Hkv][M][d]
    qr = q[(starts[:-1, None] + i).clamp(max=max(0, q.shape[0] - 1))].transpose(1, 2).float()          # [B][Hq][N][d]
    z = (qr * d ** -0.5).reshape(B, Hkv, Hq // Hkv * N, d) @ k.transpose(2, 3)
    p = (m - n)[:, None] + i
    visible = (j <= p[..., None]) & (j < m[:, None, None])
    if c["window"]:
        visible &= (j < c["n_sink"]) | (j > p[..., None] - c["window"])
    visible = visible[:, None, None].expand(B, Hkv, Hq // Hkv, N, M).reshape(B, Hkv, Hq // Hkv * N, M)
    z = z.masked_fill(~visible, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(B, Hq, N)
    real = i < n[:, None]
    return out.view(B, Hq, N, d).transpose(1, 2)[real].to(q.dtype), lse.transpose(1, 2)[real]


def run(s):
    c = s["c"]
    if own:
        import kv_cache_eviction_decode_gb300 as kv

        if c["op"] == "norm":
            return kv.norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"], eps=1e-6,
                                  interleaved=c["interleaved"])
        if c["op"] == "append":
            kv.paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], starts=s["starts"] if c["ragged"] else None,
                            inv_freq=s["inv_freq"], interleaved=c["interleaved"])
            if not c["read"]:
                return s["kp"], s["vp"]
        if c["op"] != "attention":
            return kv.paged_gather(s["kp"], s["vp"], s["table"], s["lens"], k_starts=s["k_starts"], k_out=s["k_out"],
                                   v_out=s["v_out"])
        return kv.paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["lens"], q_starts=s["starts"] if c["ragged"] else None,
                                  max_q=c["new"], n_sink=c["n_sink"], window=s["window"], return_lse=True)
    if c["op"] == "norm":
        return plain_norm(s, s["q"], s["wq"]), plain_norm(s, s["k"], s["wk"])
    if c["op"] == "append":
        plain_append(s)
        if not c["read"]:
            return s["kp"], s["vp"]
    if c["op"] != "attention":
        plain_gather(s)
        return s["k_out"], s["v_out"]
    return plain_attention(s)


# ------------------------------------------------------------------------------------------- what a pass cannot do without
def seen(c, nl, kl):
    """Visible (query, key) pairs of one head, and the keys that any query of a sequence sees, over all sequences."""
    pairs = keys = 0
    for n, m in zip(nl, kl):
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
    e, d, H = (2 if c["dtype"] == "bf16" else 4), c["head_dim"], c["kv_heads"]
    if c["op"] == "norm":
        n = c["batch"] * c["tokens"]
        rows = n * (c["q_heads"] + H)
        return {"bytes": 2 * rows * d * e + 8 * n + 2 * d * e, "flops": rows * (4 * d + 3 * c["rotary_dim"])}
    nl, kl = lengths(c)
    row = 5 * d / 8 if c["pages"] == "q4" else d * e  # bytes of a token and head in a page
    if c["op"] == "attention":
        pairs, keys = seen(c, nl, kl)
        return {"bytes": sum(nl) * c["q_heads"] * (2 * d * e + 4) + 2 * keys * H * row, "flops": 4 * d * c["q_heads"] * pairs}
    w = {"bytes": 0, "flops": 0}
    if c["op"] == "append":
        w = {"bytes": 2 * sum(nl) * H * (d * e + row), "flops": sum(nl) * H * (3 * c["rotary_dim"] + (8 * d if c["pages"] == "q4" else 0))}
    if c["op"] == "gather" or c["read"]:
        w = {"bytes": w["bytes"] + 2 * sum(kl) * H * (d * e + row), "flops": w["flops"] + (4 * d * sum(kl) * H if c["pages"] == "q4" else 0)}
    return w


# ------------------------------------------------------------------------------------- the definitions, in 64 bits
def exact_turn(x, pos, inv_freq, interleaved):
    """x [tokens][heads][d] fp64: each pair as a complex number, times e^(i angle)."""
    R = 2 * inv_freq.shape[0]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double().unsqueeze(-1) * inv_freq).unsqueeze(1)
    y = x.clone()
    if interleaved:
        pairs = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous())
        y[..., :R] = torch.view_as_real(pairs * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def exact_norm(s, x, w):
    c = s["c"]
    if c["form"] == "heads":
        x = x.transpose(1, 2).flatten(0, 1)
    x = x.double()
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True).pow(2) / c["head_dim"] + 1e-6).sqrt()
    y = exact_turn(x / rms * w.double(), s["pos"].flatten(), s["inv_freq"], c["interleaved"])
    return y if c["form"] == "tokens" else y.unflatten(0, (c["batch"], c["tokens"])).transpose(1, 2)


def exact_rows(raw, page, d):
    """One head's rows of 4-bit pages: raw [pages in order][page * 5 d / 8] bytes, to [rows][d] fp64."""
    r = raw.reshape(raw.shape[0], -1)
    codes, rest = r[:, :page * d // 2].reshape(-1, d // 2), r[:, page * d // 2:].contiguous().view(torch.bfloat16).reshape(-1, d // 32, 2)
    c = torch.arange(d, device=DEV)
    at, high = d // 16 * (c % 32 // 4) + 2 * (c // 32) + c % 4 // 2, c % 2
    code = (codes[:, at].long() >> (4 * high)) & 15
    return rest[:, c // 32, 0].double() + (code - 8) * rest[:, c // 32, 1].double()


def exact_sequence(s, pages, b, m):
    """A sequence's first m rows out of its pages, [heads][m][d] fp64."""
    c, S, d = s["c"], s["c"]["page"], s["c"]["head_dim"]
    mine = pages[s["table"][b, :-(-m // S)].long()]  # [pages][heads][S][...]
    if c["pages"] == "own":
        return mine.transpose(0, 1).flatten(1, 2)[:, :m].double()
    return torch.stack([exact_rows(mine[:, h], S, d)[:m] for h in range(c["kv_heads"])])


def exact_append(s, nl, kl):
    """The new rows, [tokens][heads][d] fp64, as the pages hold them (4 bits: as the values they stand for)."""
    c, pos = s["c"], torch.cat([torch.arange(k - n, k, device=DEV) for n, k in zip(nl, kl)])
    k, v = s["k"].double(), s["v"].double()
    if c["rotary_dim"]:
        k = exact_turn(k, pos, s["inv_freq"], c["interleaved"])
    if c["pages"] == "own":
        return k, v
    got = []
    for x in (k, v):
        y = x.clone()
        for j in range(0, c["head_dim"], 32):
            z = x[..., j:j + 32]
            lo, hi = z.min(-1, keepdim=True).values, z.max(-1, keepdim=True).values
            base = ((8 * hi + 7 * lo) / 15).bfloat16().double()
            need = torch.maximum((hi - base) / 7, (base - lo) / 8)
            near = need.bfloat16()
            step = torch.where(near.double() < need, (near.view(torch.int16) + 1).view(torch.bfloat16), near).double()  # upwards
            y[..., j:j + 32] = base + torch.where(step > 0, ((z - base) / step).round().clamp(-8, 7) * step, 0.0)
        got.append(y)
    return got


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        return [exact_norm(s, s["q"], s["wq"]), exact_norm(s, s["k"], s["wk"])]
    nl, kl = lengths(c)
    S = c["page"]
    if c["op"] == "attention":
        G, outs, sums, at = c["q_heads"] // c["kv_heads"], [], [], 0
        for b, (n, m) in enumerate(zip(nl, kl)):
            if not n:
                continue
            k, v = (exact_sequence(s, x, b, m) for x in (s["kp"], s["vp"]))
            q = s["q"][at:at + n].double().unflatten(1, (c["kv_heads"], G))
            at += n
            i, j = torch.arange(m - n, m, device=DEV)[:, None], torch.arange(m, device=DEV)
            dead = j > i
            if c["window"]:
                dead |= (j >= c["n_sink"]) & (j <= i - c["window"])
            z = torch.einsum("nhgd,hjd->nhgj", q, k) / math.sqrt(c["head_dim"])
            z = z + torch.zeros_like(z).masked_fill(dead[:, None, None], -math.inf)
            lse = torch.logsumexp(z, -1)
            outs.append(torch.einsum("nhgj,hjd->nhgd", torch.exp(z - lse[..., None]), v).flatten(1, 2))
            sums.append(lse.flatten(1))
        return [torch.cat(outs), torch.cat(sums)]
    if c["op"] == "append":
        new = exact_append(s, nl, kl)
    if c["op"] == "append" and not c["read"]:
        whole = [s["kp"].double(), s["vp"].double()]
        for pages, x in zip(whole, new):
            at = 0
            for b, (n, m) in enumerate(zip(nl, kl)):
                i = torch.arange(m - n, m, device=DEV)
                pages[s["table"][b, i // S].long(), :, i % S] = x[at:at + n]
                at += n
        return whole
    got = []
    for which, pages in enumerate((s["kp"], s["vp"])):
        rows, at = [], 0
        out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV)
        for b, (n, m) in enumerate(zip(nl, kl)):
            x = exact_sequence(s, pages, b, m)
            if n:
                x[:, m - n:] = new[which][at:at + n].transpose(0, 1)
                at += n
            if s["k_starts"] is None:
                out[b, :, :m] = x
            else:
                rows.append(x.transpose(0, 1))
        got.append(out if s["k_starts"] is None else torch.cat(rows))
    return got
