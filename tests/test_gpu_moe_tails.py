"""GPU: the ends of long rows in the experts' products, and their error over many elements."""
from __future__ import annotations

import pytest
import torch

import layers_oracle as L
import layers_tight as R
from test_gpu_moe import compare, problem
from test_layers_tight import WIDTHS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width,F", WIDTHS)
@pytest.mark.parametrize("T,E,k", [(70, 9, 4), (128, 3, 3)])
def test_error_over_many_elements(width, F, T, E, k):
    p = problem(T, E, k, width, F, width + F + T)
    y = compare(*p)
    assert R.rms(y, L.experts(*p)[0]) <= R.EXPERTS


@pytest.mark.parametrize("T,E,k", [(5, 9, 4), (20, 5, 2), (40, 3, 3)])
def test_error_at_a_layers_widths(T, E, k):
    p = problem(T, E, k, 2048, 1408, T)
    y = compare(*p)
    assert R.rms(y, L.experts(*p)[0]) <= R.EXPERTS


@pytest.mark.parametrize("width,F", WIDTHS)
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (5, 9, 4), (40, 3, 3)])
def test_tails_alone(width, F, T, E, k):
    """Inputs that are 0 but in the last 8 of D, or of F."""
    x, gu, dn, ids, weights = problem(T, E, k, width, F, width + F + T)
    tail = x.clone()
    tail[:, :-8] = 0
    assert compare(tail, gu, dn, ids, weights).abs().max() > 0
    tail = dn.clone()
    tail[:, :, :-8] = 0
    assert compare(x, gu, tail, ids, weights).abs().max() > 0
