"""Plain FP64 implementations of the operators between a decode step's projections, and the
bounds that their GPU results are held to.  Nothing here uses the package.

Rounding facts used below: BF16 round-to-nearest is off by at most 2^-8 |v| (half a unit in the
last place of 8 significant bits) or 2^-134 near zero; e4m3 by at most 2^-4 |v| (half a unit of 4
significant bits) or 2^-10 (half the spacing of its subnormals); one FP32 operation by 2^-24 |v|,
or 2^-23 |v| where the tensor core truncates; CUDA's rsqrtf, division and exp2 approximations by a
few units of 2^-22.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24


# ------------------------------------------------------------------------------------ RMS norm
def add_rmsnorm(x, weight, residual=None, eps=1e-6):
    """(y, h) in FP64."""
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    mean = (h * h).sum(-1, keepdim=True) / x.shape[-1]
    return h / torch.sqrt(mean + eps) * weight.double(), h


def scales_of(y, group):
    """FP64 scales max|y| / 448 of each group of columns (0: the whole row); 1 where that is 0."""
    D = y.shape[-1]
    parts = y.split(group if group else D, -1)
    top = torch.stack([p.abs().amax(-1) for p in parts], -1) / 448.0
    return torch.where(top == 0, torch.ones_like(top), top)


def spread(scales, D, group):
    """Scales repeated to one per column."""
    return scales.repeat_interleave(group, -1)[:, :D] if group else scales.expand(-1, D)


def norm_rel(D):
    """Relative error of the FP32 y before its rounding: h is one addition (2^-24); the sum of D
    squares and its mean are off by (D + 2) 2^-24 relatively (all terms positive), half of that
    after the root; rsqrt and the two products add a few units."""
    return (D / 2 + 16) * U32


def norm_y_bound(y, D):
    return y.abs() * (2.0 ** -8 + norm_rel(D)) * (1 + 2.0 ** -8) + 2.0 ** -133


def residual_bound(h):
    """h is rounded to FP32, then to BF16."""
    return h.abs() * (2.0 ** -8 + 2 * U32) + 2.0 ** -133


# ------------------------------------------------------------------------------- latent append
def rotate(x, cos, sin, interleaved):
    """Rotate the pairs of x's last dimension, FP64; also the sum of the products' magnitudes."""
    x = x.double()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
    else:
        a, b = x.chunk(2, -1)
    first, second = a * cos - b * sin, b * cos + a * sin
    m1, m2 = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    if interleaved:
        return torch.stack([first, second], -1).flatten(-2), torch.stack([m1, m2], -1).flatten(-2)
    return torch.cat([first, second], -1), torch.cat([m1, m2], -1)


def rotate_bound(v, magnitude):
    """Two products and a sum in FP32 (3 roundings of the magnitudes at most), then BF16."""
    return v.abs() * 2.0 ** -8 + magnitude * 4 * U32 + 2.0 ** -133


# ----------------------------------------------------------------------------- latent attention
def latent_attention(q, cache, table, lens, rank, scale, cu_q):
    """(out, lse, out bound, lse bound) in FP64, token by token from the definition.

    Bounds.  A score's FP32 sum of W products is off by e = W 2^-23 scale sum|q||k| at most, so
    its weight by the factor exp(e); 2 e covers numerator and denominator.  The weights' rounding
    to BF16 (the products' operands; the denominator keeps FP32) costs 2^-8 of
    A = sum_j p_j |v_j|; FP32 sums over n keys and the exponential 2^-20 + n 2^-23 of A; rounding
    the result 2^-8 |out|.  Shares of a split context are joined in FP32: inside the 2^-20.
    """
    total, H, W = q.shape
    page = cache.shape[1]
    out = torch.zeros((total, H, rank), dtype=torch.float64)
    lse = torch.full((total, H), -math.inf, dtype=torch.float64)
    ob = torch.zeros_like(out)
    lb = torch.zeros_like(lse)
    for b in range(len(lens)):
        n, first, last = int(lens[b]), int(cu_q[b]), int(cu_q[b + 1])
        used = table[b, : -(-n // page)].long()
        keys = cache[used].reshape(-1, W)[:n].double()
        for t in range(first, last):
            sees = n - (last - first) + (t - first) + 1
            if sees <= 0:
                continue
            k = keys[:sees]
            qt = q[t].double()
            s = (qt @ k.T) * scale
            e = (abs(scale) * (qt.abs() @ k.abs().T) * W * 2.0 ** -23).amax(1)
            lse[t] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[t][:, None])
            out[t] = p @ k[:, :rank]
            A = p @ k[:, :rank].abs()
            rel = 2 * e + 2.0 ** -20 + sees * 2.0 ** -23
            ob[t] = (2.0 ** -8 + rel[:, None]) * A * (1 + 2.0 ** -8) + 2.0 ** -8 * out[t].abs() + 2.0 ** -133
            lb[t] = e + 2.0 ** -20 + sees * 2.0 ** -23 + lse[t].abs() * 2.0 ** -22
    return out, lse, ob, lb


def check(got, want, bound, what=""):
    """Every element within its bound; what is not finite has to be alike."""
    got = got.detach().cpu().double()
    fine = torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert torch.all(fine | same), f"{what}: infinities or NaN differ"
    assert torch.all(torch.isfinite(got) | ~fine), f"{what}: infinities or NaN where none belong"
    d = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    over = torch.where(fine, d / bound.clamp(min=1e-300), torch.zeros_like(want))
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound, {int((over > 1).sum())} of {over.numel()} elements"
    return worst
