"""Plain 64-bit attention for the operator tests, and error bounds derived from
the arithmetic of the kernels.

With A_i = sum_j p_ij |v_j| (p the exact softmax), every output element obeys
  |out - exact| <= A (r_p + 2 dz + n u) + r_out |exact| + tiny,
where
  dz     bounds a logit's error: (d + 4) u S, S = scale * max_ij sum_e |q_ie k_je|, u = 2^-23 (an fp32 chain of d
         products and sums, each off by at most one step: tensor cores may truncate), plus 2 steps of S for the
         scaling; it enters the numerator and the denominator;
  r_p    the rounding of the probabilities for the product with V: half a step of bf16, 2^-8, else 0;
  n u    the fp32 sums over n keys (numerator and denominator), and 2^-20 for the exponential and the division;
  r_out  the output's own rounding, half a step: 2^-8 for bf16, 2^-24 for fp32.
lse: dz + n u + 2^-20 + 2^-23 |lse|.
"""
import math

import torch

U = 2.0 ** -23


def rows(q, k, v, visible, scale):
    """q [H][n][d], k, v [H][m][d] (fp64), visible [n][m]: out, lse, A, all fp64."""
    z = torch.einsum("hid,hjd->hij", q, k) * scale
    z = z.masked_fill(~visible, -math.inf)
    top = z.amax(-1, keepdim=True) if z.shape[-1] else torch.full(z.shape[:-1] + (1,), -math.inf, dtype=z.dtype, device=z.device)
    e = torch.exp(z - top.masked_fill(top == -math.inf, 0))
    s = e.sum(-1, keepdim=True)
    p = e / s.masked_fill(s == 0, 1)
    v = torch.where(visible.any(0)[None, :, None], v, torch.zeros_like(v))  # rows nobody sees may hold anything
    return p @ v, (top + torch.log(s)).squeeze(-1), p @ v.abs()


def visible(n, m, n_sink, window, device):
    p = (m - n + torch.arange(n, device=device))[:, None]
    j = torch.arange(m, device=device)[None]
    see = j <= p
    if window:
        see &= (j < n_sink) | (j > p - window)
    return see


def sequence(q, k, v, n_sink, window, scale):
    """One sequence: q [Hq][n][d], k, v [Hkv][m][d] of any type."""
    G = q.shape[0] // k.shape[0]
    see = visible(q.shape[1], k.shape[1], n_sink, window, q.device)
    kd, vd = (x.double().repeat_interleave(G, 0) for x in (k, v))
    kd = torch.where(see.any(0)[None, :, None], kd, torch.zeros_like(kd))
    return rows(q.double(), kd, vd, see, scale)


def bounds(dtype, q, k, n_keys, scale, ref, A, lse):
    d = q.shape[-1]
    kk = k.double()
    kk = torch.where(torch.isfinite(kk), kk, torch.zeros_like(kk))
    S = scale * (q.double().norm(dim=-1).max() * kk.norm(dim=-1).max()).item() if k.numel() and q.numel() else 0.0
    dz = (d + 6) * U * S
    half = torch.finfo(dtype).eps / 2
    r_p = half if dtype == torch.bfloat16 else 0.0
    tol = A * (r_p + 2 * dz + n_keys * U + 2.0 ** -20) + half * ref.abs() + 1e-30
    tol_l = dz + n_keys * U + 2.0 ** -20 + U * torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    return tol, tol_l


def assert_close(got, ref, tol, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same_inf = (got.double() == ref) & torch.isinf(ref)
    err = torch.where(same_inf, torch.zeros_like(ref), (got.double() - ref).abs())
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.3g} of the bound"
