"""GPU: infinities and NaN in an expert's weights reach the tokens that chose it, and no others."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L
from test_gpu_moe import problem

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def check(x, gu, dn, ids, weights, spoil):
    """``spoil(gu, dn)`` puts them into expert 1, and says which elements of y they reach (a mask of D)."""
    chose = (ids == 1).any(1)
    want, bound = L.experts(x, gu, dn, ids, weights)  # of the tokens that did not choose it the same
    bad_gu, bad_dn = gu.clone(), dn.clone()
    reached = spoil(bad_gu, bad_dn)
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), bad_gu.to(DEV), bad_dn.to(DEV), ids.to(DEV), weights.to(DEV))
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    assert chose.any() and not chose.all()
    D.check(y[~chose], want[~chose], bound[~chose], "tokens that did not choose it")
    got = y.cpu()[chose]
    assert not torch.isfinite(got[:, reached]).any()
    if not reached.all():
        D.check(got[:, ~reached], want[chose][:, ~reached], bound[chose][:, ~reached], "its other rows")


def rows_of_down(value):
    def spoil(gu, dn):
        D_, F = dn.shape[1:]
        reached = torch.zeros(D_, dtype=torch.bool)
        for i, d in enumerate((0, 5, D_ // 2, D_ - 1)):
            dn[1, d, (7 * i) % F if i else F - 1] = value  # (a product of 0 and an infinity is NaN, others infinite)
            reached[d] = True
        return reached
    return spoil


def all_of_down(gu, dn):
    dn[1] = NAN
    return torch.ones(dn.shape[1], dtype=torch.bool)


def of_gate_and_up(gu, dn):
    gu[1, 0, 3], gu[1, gu.shape[1] // 2, 1] = NAN, INF
    return torch.ones(dn.shape[1], dtype=torch.bool)


@pytest.mark.parametrize("spoil", [rows_of_down(NAN), rows_of_down(INF), rows_of_down(-INF), all_of_down, of_gate_and_up],
                         ids=["nan", "inf", "minus_inf", "all", "gate_up"])
@pytest.mark.parametrize("T,E,k,width,F", [(2, 4, 1, 64, 40), (9, 6, 2, 256, 192), (20, 40, 3, 136, 1000), (40, 5, 2, 512, 64),
                                           (70, 70, 8, 64, 72), (128, 12, 3, 200, 136)])
def test_weights_that_are_not_finite(spoil, T, E, k, width, F):
    p = problem(T, E, k, width, F, T + E)
    p[3][0, 0], p[3][1] = 1, torch.tensor([2, 3, 0, *range(4, 4 + k)])[:k]  # the first token chooses it, the second does not
    check(*p, spoil)


def test_an_expert_twice_and_entries_that_are_not_used():
    p = problem(5, 6, 3, 96, 48, 1)
    ids = p[3]
    ids[:] = torch.tensor([[1, 4, 1], [2, 5, 2], [-1, 3, 3], [0, -1, -1], [4, 0, 5]])
    check(*p, rows_of_down(NAN))


def test_strided_weights_and_the_same_bits_again():
    x, gu, dn, ids, weights = problem(6, 5, 2, 64, 40, 2)
    ids[:, 0] = torch.tensor([1, 2, 3, 4, 0, 2])
    ids[:, 1] = torch.tensor([0, 3, 4, 0, 2, 4])
    dn[1, 7] = NAN
    wide = torch.full((5, 66, 48), NAN, dtype=torch.bfloat16, device=DEV)
    wide[:, :64, 8:] = dn.to(DEV)
    args = x.to(DEV), gu.to(DEV)
    a = sk.sgemm_bf16_moe_experts(*args, dn.to(DEV), ids.to(DEV), weights.to(DEV))
    b = sk.sgemm_bf16_moe_experts(*args, wide[:, :64, 8:], ids.to(DEV), weights.to(DEV))
    torch.cuda.synchronize()
    assert torch.isnan(a[0, 7]) and torch.isfinite(a[1:]).all()
    assert torch.equal(a[1:], b[1:]) and torch.equal(a.isnan(), b.isnan())
