"""What the limits of layers_tight and the tests of tails tell apart, on the CPU: results with a mistake in them, made
here, pass them where they should not."""
from __future__ import annotations

import pytest
import torch

import decode_oracle as D
import layers_oracle as L
import layers_tight as R


def problem(T, E, k, width, F, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(torch.bfloat16)
    x, gu, dn = n(T, width), n(E, 2 * F, width, std=width ** -0.5), n(E, width, F, std=F ** -0.5)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    return x, gu, dn, ids, torch.rand((T, k), generator=g) + 0.05


def rounded(x, gu, dn, ids, weights, lose=None):
    """The products with the roundings that the kernels make; without the last 8 of D or F where ``lose`` says so."""
    if lose == "D":
        x = x.clone()
        x[:, -8:] = 0
    y = torch.zeros(x.shape, dtype=torch.float64)
    F = dn.shape[2]
    for e in range(dn.shape[0]):
        w = (weights.double() * (ids == e)).sum(1, keepdim=True)
        g, u = x.double() @ gu[e, :F].double().T, x.double() @ gu[e, F:].double().T
        h = (w * g * torch.sigmoid(g) * u).to(torch.bfloat16).double()
        if lose == "F":
            h[:, -8:] = 0
        y += h @ dn[e].double().T
    return y.to(torch.bfloat16)


WIDTHS = [(8, 1000), (72, 56), (200, 136), (1000, 24), (1032, 520), (4104, 264), (512, 2048)]


@pytest.mark.parametrize("width,F", WIDTHS)
@pytest.mark.parametrize("T,E,k", [(70, 9, 4), (128, 3, 3)])
def test_experts_limit(width, F, T, E, k):
    p = problem(T, E, k, width, F, width + F + T)
    want, bound = L.experts(*p)
    good = rounded(*p)
    D.check(good, want, bound)
    assert R.rms(good, want) <= R.EXPERTS
    for lose in "DF":
        assert R.rms(rounded(*p, lose=lose), want) > R.EXPERTS


@pytest.mark.parametrize("width,F", WIDTHS)
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (5, 9, 4), (40, 3, 3)])
def test_tails_alone(width, F, T, E, k):
    """Inputs that are 0 but in the last 8 of D, or of F: without them the result is 0, and outside the bound."""
    x, gu, dn, ids, weights = problem(T, E, k, width, F, width + F + T)
    tail = x.clone()
    tail[:, :-8] = 0
    want, bound = L.experts(tail, gu, dn, ids, weights)
    with pytest.raises(AssertionError, match="times the bound"):
        D.check(torch.zeros_like(want), want, bound)
    tail = dn.clone()
    tail[:, :, :-8] = 0
    want, bound = L.experts(x, gu, tail, ids, weights)
    with pytest.raises(AssertionError, match="times the bound"):
        D.check(torch.zeros_like(want), want, bound)


@pytest.mark.parametrize("n", [64, 300, 1000])
def test_states_limit(n):
    """Keys in three numbers keep the limit, in two they do not."""
    g = torch.Generator().manual_seed(n)
    k = (torch.randn((n, 1, 64), generator=g) / 8).to(torch.bfloat16)
    v = torch.randn((n, 1, 64), generator=g).to(torch.bfloat16)
    decay = -torch.exp(-torch.rand((n, 1), generator=g) * 6.9)
    want = L.linear(torch.zeros_like(k), k, v, decay, torch.zeros((1, 64, 64)), 1.0, True)[1][0]
    behind = decay.double().flip(0).cumsum(0).flip(0) - decay.double()  # the sum of g behind a token
    for numbers, fine in ((3, True), (2, False), (1, False)):
        got = R.cut_keys(k[:, 0], torch.exp(behind), numbers).T @ v[:, 0].double()
        assert (R.rms(got, want) <= R.STATES) == fine
