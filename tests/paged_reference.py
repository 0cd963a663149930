"""A paged cache in plain Python for the tests: tables, the 4-bit format read back in 64 bits, and error bounds.

4 bits: a group's base is within half a step of bf16 (2^-9 of its size; 2^-8 with the fp32 sum's own rounding far
inside) of (8 hi + 7 lo) / 15; its step is the least s with base + 7 s >= hi and base - 8 s <= lo, rounded up to bf16 (at
most 2^-7 more) after fp32 operations (2^-22 together); and every value is within half a step, plus fp32's rounding of
x - base and of the quotient, of its channel.
"""
import random

import torch

BF16_HALF = 2.0 ** -9  # relative: half a step of bf16 is at most 2^-8 of the value's power of two, 2^-9 of twice that


class Pool:
    """Pages with every sequence's places in them. `strides`: "dense", "joint" (keys and values in one tensor) or "tokens"
    (token before head)."""

    def __init__(self, lens, H, S, d, dtype, four, seed=0, width=None, strides="dense", spare=3, garbage=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = random.Random(seed)
        self.lens, self.H, self.S, self.d, self.four, self.dtype = lens, H, S, d, four, dtype
        used = [-(-max(n, 0) // S) for n in lens]
        self.width = max(used + [1]) if width is None else width
        n = sum(used) + spare
        order = list(range(n))
        r.shuffle(order)
        table, at = [], 0
        for u in used:
            row = order[at:at + u] + [r.choice([-1, -7, n, n + 5, 2**31 - 1]) for _ in range(self.width - u)]
            at += u
            table.append(row)
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda").reshape(len(lens), self.width)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        row, t = (5 * d // 8, torch.uint8) if four else (d, dtype)
        if strides == "joint":
            both = torch.empty(n, 2, H, S, row, dtype=t, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        elif strides == "tokens" and not four:
            self.k, self.v = (torch.empty(n, S, H, row, dtype=t, device="cuda").transpose(1, 2) for _ in range(2))
        else:
            self.k, self.v = (torch.empty(n, H, S, row, dtype=t, device="cuda") for _ in range(2))
        for p in (self.k, self.v):
            if not four:
                p.copy_(torch.randn(n, H, S, d, generator=g, device="cuda"))
            else:
                codes, params = parts(p, d)
                codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda"))
                params[..., 0] = (0.3 * torch.randn(params.shape[:-1], generator=g, device="cuda")).bfloat16()
                params[..., 1] = (0.27 * torch.exp(0.2 * torch.randn(params.shape[:-1], generator=g, device="cuda"))).bfloat16()
        if garbage:  # rows that hold no token: infinities and NaN
            for b, m in enumerate(lens):
                for i in range(max(m, 0), used[b] * S):
                    self.spoil(b, i)

    def spoil(self, b, i):
        page, slot = int(self.table[b, i // self.S]), i % self.S
        for p in (self.k, self.v):
            if self.four:
                parts(p, self.d)[1][page, :, slot] = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16()
            else:
                p[page, :, slot] = torch.tensor([float("nan"), float("inf")], device="cuda").to(p.dtype).repeat(self.d // 2)

    def rows(self, b, m, which):
        """The first m rows of a sequence, [H][m][d] fp64, and (4 bits) |base| + |code - 8| step, else the values' size, and
        the steps."""
        p = (self.k, self.v)[which]
        pages = self.table[b, :-(-m // self.S)].long()
        if not self.four:
            x = p[pages].transpose(0, 1).reshape(self.H, -1, self.d)[:, :m].double()
            return x, x.abs(), None
        codes, params = parts(p, self.d)
        c = unpack(codes[pages].transpose(0, 1).reshape(self.H, -1, self.d // 2)[:, :m])
        q = params[pages].transpose(0, 1).reshape(self.H, -1, self.d // 32, 2)[:, :m].double()
        base, step = (q[..., i].repeat_interleave(32, -1) for i in (0, 1))
        u = (c - 8).double()
        return base + u * step, base.abs() + u.abs() * step, step


def parts(pages, d):
    """Codes [..][H][S][d / 2] and (base, step) [..][H][S][d / 32][2] of 4-bit pages, views."""
    n, H, S = pages.shape[:3]
    s0, s1 = pages.stride()[:2]
    codes = pages.as_strided((n, H, S, d // 2), (s0, s1, d // 2, 1), pages.storage_offset())
    raw = pages.as_strided((n, H, S, d // 32, 4), (s0, s1, d // 8, 4, 1), pages.storage_offset() + S * d // 2)
    return codes, raw.view(torch.bfloat16)


def unpack(codes):
    """[...][d / 2] bytes to whole numbers [...][d], one channel after another."""
    d = 2 * codes.shape[-1]
    out = torch.empty(*codes.shape[:-1], d, dtype=torch.int64, device=codes.device)
    for c in range(d):
        j, g, i = c // 32, c % 32 // 4, c % 4
        out[..., c] = (codes[..., d // 16 * g + 2 * j + i // 2].long() >> (4 * (i % 2))) & 15
    return out


def check_groups(x, slack, codes, params):
    """x [n][d] fp64, of which the kernel saw values within slack; codes [n][d], params [n][d / 32][2] as stored."""
    x, slack, c = (t.unflatten(-1, (-1, 32)) for t in (x, slack, codes.double()))
    base, step = params[..., 0].double(), params[..., 1].double()
    lo, hi, s = x.amin(-1), x.amax(-1), slack.amax(-1)
    size = lo.abs() + hi.abs()
    assert ((base - (8 * hi + 7 * lo) / 15).abs() <= 2.0 ** -8 * base.abs() + 2.0 ** -20 * size + s + 1e-38).all()
    need = torch.maximum((hi - base) / 7, (base - lo) / 8)
    fuzz = 2.0 ** -20 * (size + base.abs()) + s + 1e-38
    assert (step >= need - fuzz).all() and (step <= need * (1 + 2.0 ** -7) + 2 * fuzz).all()
    v = base[..., None] + (c - 8) * step[..., None]
    assert ((v - x).abs() <= 0.5 * step[..., None] + fuzz[..., None]).all(), float(((v - x).abs() / step[..., None].clamp_min(1e-30)).max())
    assert (c[(step == 0)[..., None].expand_as(c)] == 8).all()


U = 2.0 ** -23


def attention_bounds(dtype, four, q, k, k_size, k_step, A, A_step, n_keys, scale, ref, lse):
    """Bounds of one sequence's out and lse, as derived in tests/attn_reference.py, for q and k [H][..][d] fp64. 4 bits: the
    codes enter a product as they are (at most 15), and 8 times the other factor's sum is taken away, in fp32. Of a
    logit's group of 32: 34 operations, each off by a step of at most (15 + 8) step sum |q|; the bases 32 more of their
    own size; sum them over the groups. Of an output: 80 operations a run of keys at most, the same with the probabilities,
    which are rounded after they are multiplied with the step. A: p @ |v| (4 bits: |base| + |code - 8| step), A_step: p @ step."""
    d = q.shape[-1]
    half = torch.finfo(dtype).eps / 2
    r_p = half if dtype == torch.bfloat16 else 0.0
    if four:
        S, T = (scale * float((q.abs() @ x.transpose(-1, -2)).max()) if x.numel() and q.numel() else 0.0 for x in (k_size, k_step))
        dz = U * ((d + 6) * S + 34 * 23 * T)
        tol = A * (r_p + 2 * dz + n_keys * U + 2.0 ** -20) + 80 * 23 * U * A_step
    else:
        S = scale * float((q.norm(dim=-1).max() * k.norm(dim=-1).max())) if k.numel() and q.numel() else 0.0
        dz = (d + 6) * U * S
        tol = A * (r_p + 2 * dz + n_keys * U + 2.0 ** -20)
    tol_l = dz + n_keys * U + 2.0 ** -20 + U * torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    return tol + half * ref.abs() + 1e-30, tol_l
