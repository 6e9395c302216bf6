"""Plain FP64 implementations of the operators that make whole layers, and the bounds that their GPU
results are held to.  Nothing here uses the package.

Rounding facts: as in decode_oracle (BF16 off by at most 2^-8 |v|, one FP32 operation by 2^-24 |v|,
or 2^-23 |v| where the tensor core truncates, CUDA's exp and division by a few units of 2^-22).
"""
from __future__ import annotations

import math

import torch

ACC = 2.0 ** -23  # an addition in the tensor core, relative to the sum of magnitudes
TINY = 2.0 ** -133


# ------------------------------------------------------------------------------------------ router
def route(x, w, bias=None, scoring="softmax"):
    """(scores, keys, error of a key) in FP64.  A logit's FP32 sum of D products is off by
    e = D 2^-23 sum |x||w| at most.  Sigmoid: a derivative of 1/4 at most, and 2^-20 of itself.
    Softmax: factors exp(e) above and below, 2 e + 2^-20 (and the sum's E 2^-24) of itself."""
    x, w = x.double(), w.double()
    logits = x @ w.T
    e = (x.abs() @ w.abs().T) * x.shape[1] * ACC
    worst = e.amax(1, keepdim=True)
    if scoring == "softmax":
        s = torch.softmax(logits, 1)
        err = s * (torch.expm1(2 * worst) + 2.0 ** -20 + w.shape[0] * 2.0 ** -24)
    else:
        s = torch.sigmoid(logits)
        err = e / 4 + s * 2.0 ** -20
    if bias is None:
        return s, logits, worst.expand_as(logits), err  # chosen by the logits
    return s, s + bias.double(), err + (s + bias.double()).abs() * 2.0 ** -23, err


def check_route(ids, weights, x, w, k, bias=None, scoring="softmax", renormalize=True, scale=1.0):
    """Each choice is as good as the exact one but for the keys' errors, and no expert comes twice."""
    s, key, key_err, s_err = route(x, w, bias, scoring)
    ids, weights = ids.cpu().long(), weights.cpu().double()
    best = key.sort(1, descending=True)[0][:, :k]
    slack = 2 * key_err.amax(1, keepdim=True)
    got = key.gather(1, ids)
    assert torch.all((got - best).abs() <= slack), "chosen experts"
    assert all(len(set(row)) == k for row in ids.tolist()), "an expert twice"
    c, ce = s.gather(1, ids), s_err.gather(1, ids)
    if renormalize:
        total = c.sum(1, keepdim=True)
        want, err = c / total, ce / total + c / total ** 2 * ce.sum(1, keepdim=True)
    else:
        want, err = c, ce
    bound = abs(scale) * (err * 1.01 + want * (k + 4) * 2.0 ** -22)
    assert torch.all((weights - want * scale).abs() <= bound + 2.0 ** -140), "weights"


# ----------------------------------------------------------------------------------------- experts
def experts(x, gate_up, down, ids, weights):
    """(y, bound).  gate and up are off by D 2^-23 sum |x||w| each (eg, eu); |silu'| <= 1.1, so that
    w h is off by |w| (1.1 eg |u| + |silu| eu + 1.1 eg eu) and 2^-8 + 2^-19 of itself; y by that times
    |Wd|, by n 2^-23 sum |w h||Wd| for its n = experts x F summands, and 2^-8 |y|."""
    T, D = x.shape
    E, F = down.shape[0], down.shape[2]
    x = x.double()
    y = torch.zeros((T, D), dtype=torch.float64)
    err, mag = torch.zeros_like(y), torch.zeros_like(y)
    used = sorted({int(e) for e in ids.flatten() if 0 <= e < E})
    for e in used:
        w = (weights.double() * (ids == e)).sum(1, keepdim=True)
        on = (ids == e).any(1, keepdim=True).double()
        g64, u64 = gate_up[e, :F].double(), gate_up[e, F:].double()
        g, u = x @ g64.T, x @ u64.T
        eg, eu = (x.abs() @ g64.abs().T) * D * ACC, (x.abs() @ u64.abs().T) * D * ACC
        silu = g * torch.sigmoid(g)
        h = w * silu * u * on
        dh = w.abs() * on * (1.1 * eg * u.abs() + silu.abs() * eu + 1.1 * eg * eu) + h.abs() * (2.0 ** -8 + 2.0 ** -19)
        d64 = down[e].double()
        y += h @ d64.T
        err += dh @ d64.abs().T
        mag += (h.abs() + dh) @ d64.abs().T
    bound = err + mag * (len(used) * F + 16) * ACC + (y.abs() + err) * 2.0 ** -8 * 1.01 + TINY
    return y, bound


# ------------------------------------------------------------------------- attention by mask
def tree_attention(q, cache, table, lens, rank, scale, cu_q, masks):
    """(out, lse, out bound, lse bound), token by token; ``masks``: a set of new tokens for each.  The
    bounds are those of decode_oracle.latent_attention."""
    total, H, W = q.shape
    page = cache.shape[1]
    out = torch.zeros((total, H, rank), dtype=torch.float64)
    lse = torch.full((total, H), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(lens)):
        n, first, last = int(lens[b]), int(cu_q[b]), int(cu_q[b + 1])
        base = n - (last - first)
        rows = cache[table[b, : -(-n // page)].long()].reshape(-1, W)[:n].double()
        for t in range(first, last):
            see = list(range(max(0, base))) + [base + j for j in sorted(masks[t]) if 0 <= j < last - first and base + j >= 0]
            if not see:
                continue
            k, qt = rows[see], q[t].double()
            s = (qt @ k.T) * scale
            e = (abs(scale) * (qt.abs() @ k.abs().T) * W * ACC).amax(1)
            lse[t] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[t][:, None])
            out[t] = p @ k[:, :rank]
            A = p @ k[:, :rank].abs()
            rel = 2 * e + 2.0 ** -20 + len(see) * ACC
            ob[t] = (2.0 ** -8 + rel[:, None]) * A * (1 + 2.0 ** -8) + 2.0 ** -8 * out[t].abs() + TINY
            lb[t] = e + 2.0 ** -20 + len(see) * ACC + lse[t].abs() * 2.0 ** -22
    return out, lse, ob, lb


# -------------------------------------------------------------------------------- linear attention
def linear(q, k, v, g, state, scale, chunked):
    """One sequence from ``state`` ([Hv, Dk, Dv]), token by token: (out, last state, their bounds).

    Magnitudes go through the same recurrence: M = exp(g) M + |k||v|, and |q|^T M for the outputs.
    One token at a time, S is off by 2^-22 (exp) and two FP32 roundings of M; the output by that,
    Dk 2^-24 for its sum, and 2^-8 of itself.
    In chunks the decayed keys are off by 2^-17, sums over n tokens and Dk products, and the chunks'
    factors, by (n + Dk) 2^-23 + n 2^-22 / 64; the outputs' operands (S, and the weights of a chunk)
    are rounded to BF16, 2^-8 of |q|^T M together at most, the products q.k before by Dk 2^-23."""
    n, Hv = v.shape[:2]
    r = Hv // q.shape[1]
    q, k, v = q.double().repeat_interleave(r, 1), k.double().repeat_interleave(r, 1), v.double()
    Dk = q.shape[2]
    S, M = state.double().clone(), state.double().abs()
    out, mag = torch.zeros((n, Hv, v.shape[2]), dtype=torch.float64), torch.zeros((n, Hv, v.shape[2]), dtype=torch.float64)
    for t in range(n):
        e = torch.exp(g[t].double())[:, None, None]
        S = e * S + k[t][:, :, None] * v[t][:, None, :]
        M = e * M + (k[t][:, :, None] * v[t][:, None, :]).abs()
        out[t] = scale * torch.einsum("hk,hkv->hv", q[t], S)
        mag[t] = abs(scale) * torch.einsum("hk,hkv->hv", q[t].abs(), M)
    if chunked:
        rel = 2.0 ** -17 + 2.0 ** -20 + (n + Dk) * ACC + n * 2.0 ** -22 / 64
        return out, S, mag * (2.0 ** -8 + 2 * rel) * 1.01 + out.abs() * 2.0 ** -8 + TINY, M * rel + 2.0 ** -140
    rel = 2.0 ** -21 * max(n, 1)
    return out, S, mag * (rel + Dk * 2.0 ** -23) + out.abs() * 2.0 ** -8 + TINY, M * rel + 2.0 ** -140
