"""GPU: the short way from tensors to the layers' operators (native/marshal.cpp) and the long one
(layers.py) are the same call: same bits, same refusals."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import layers
from test_gpu_marshal import Never, Only

pytestmark = pytest.mark.gpu
DEV = "cuda"


def both(monkeypatch, call, outputs, again=()):
    """Runs the call both ways on outputs filled alike (``again``: what it updates, as it was)."""
    layers._short.linear_step(*[None] * 10)  # loads the module
    module, got = layers._short, []
    before = [t.clone() for t in again]
    for way in (Only(module), Never()):
        for t in outputs:
            t.fill_(3)
        for t, b in zip(again, before):
            t.copy_(b)
        monkeypatch.setattr(layers, "_short", way)
        call()
        torch.cuda.synchronize()
        monkeypatch.setattr(layers, "_short", module)
        got.append([t.clone() for t in (*outputs, *again)])
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


@pytest.mark.parametrize("T", [1, 5])
def test_route_both_ways(monkeypatch, T):
    x, w, bias = bf(T, 200)[:, 8:136], bf(1, 3, 20, 128, seed=1)[0, 1], torch.rand(20, device=DEV)
    ids, weights = torch.zeros((T, 9), dtype=torch.int32, device=DEV), torch.zeros((T, 4), device=DEV)
    for b in (bias, None):
        both(monkeypatch, lambda: sk.sgemm_bf16_moe_route(x, w, 4, b, "sigmoid", False, 2.0, ids=ids[:, 2:6], weights=weights,
                                                          stream=torch.cuda.current_stream()), [ids, weights])


@pytest.mark.parametrize("T,E", [(1, 1), (1, 4), (5, 4)])
def test_experts_both_ways(monkeypatch, T, E):
    x, gu, dn = bf(T, 72)[:, 8:], bf(E, 2 * 40 + 2, 72, seed=1, std=0.1)[:, :80, :64], bf(E, 64, 40, seed=2, std=0.1)
    ids = torch.zeros((T, 3), dtype=torch.int32, device=DEV)
    weights = torch.rand((T, 3), device=DEV)
    y = torch.zeros((T, 70), dtype=torch.bfloat16, device=DEV)[:, 3:67]
    ws = torch.empty(sk.sgemm_moe_experts_workspace(T, E, 3, 64, 40), dtype=torch.uint8, device=DEV)
    both(monkeypatch, lambda: sk.sgemm_bf16_moe_experts(x, gu, dn, ids, weights, y=y, workspace=ws), [y])


@pytest.mark.parametrize("cu", [True, False])
def test_tree_both_ways(monkeypatch, cu):
    q, cache = bf(4, 6, 192), bf(9, 16, 192, seed=2)
    table = torch.arange(8, device=DEV, dtype=torch.int32).view(2, 4)
    lens = torch.tensor([50, 33], dtype=torch.int32, device=DEV)
    cu_q = torch.tensor([0, 1, 4], dtype=torch.int32, device=DEV) if cu else None
    tree = torch.tensor([[1, 0], [1, 0], [3, 0], [5, 0]], device=DEV)
    out, lse = torch.zeros((4, 6, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 6), device=DEV)
    ws = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
    for l in (lse, None):
        both(monkeypatch, lambda: sk.sgemm_bf16_latent_tree_attention(q, cache, table, lens, 128, 0.1, tree, cu_q=cu_q, max_q=3 if cu else 2,
                                                                      out=out, lse=l, workspace=ws), [out] + ([lse] if l is not None else []))


@pytest.mark.parametrize("N,Hk,Hv", [(1, 1, 1), (1, 2, 4), (7, 2, 2)])
def test_linear_both_ways(monkeypatch, N, Hk, Hv):
    q, k, v = bf(N, Hk, 80)[..., :64], bf(N, Hk, 64, seed=1), bf(N, Hv, 128, seed=2)
    out, state = torch.zeros((N, Hv, 128), dtype=torch.bfloat16, device=DEV), torch.rand((N + 1, Hv, 64, 128), device=DEV)
    slots = torch.arange(N, device=DEV)
    for g in (-torch.rand((N, Hv), device=DEV), -torch.rand(Hv, device=DEV).expand(N, Hv), -torch.rand((Hv, N), device=DEV).T):
        both(monkeypatch, lambda: sk.sgemm_bf16_linear_step(q, k, v, g, state, slots, 0.5, out=out), [out], [state])
        cu = torch.tensor([0, N], dtype=torch.int32, device=DEV)
        ws = torch.empty(max(16, sk.sgemm_linear_attention_workspace(N, 1, Hv, 64, 128)), dtype=torch.uint8, device=DEV)
        for fresh in (None, torch.ones(1, dtype=torch.int32, device=DEV)):
            both(monkeypatch, lambda: sk.sgemm_bf16_linear_attention(q, k, v, g, state, slots[:1], cu, 0.5, fresh=fresh, out=out, workspace=ws),
                 [out], [state])


def test_what_is_not_well_formed_is_left_to_the_checks():
    x, w = bf(2, 64), bf(8, 64)
    ids, weights = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.zeros((2, 2), device=DEV)
    for bad in (dict(w=w.float()), dict(w=w[:, :32]), dict(bias=weights), dict(ids=ids.long()), dict(weights=weights.T[:1]), dict(x=x.cpu()),
                dict(scoring="max")):
        with pytest.raises((TypeError, ValueError)):
            sk.sgemm_bf16_moe_route(**(dict(x=x, w=w, k=2, ids=ids, weights=weights) | bad))
    q, k, v, g = bf(2, 2, 64), bf(2, 2, 64), bf(2, 2, 64), torch.zeros((2, 2), device=DEV)
    state, slots, out = torch.zeros((3, 2, 64, 64), device=DEV), torch.arange(2, device=DEV), bf(2, 2, 64)
    for bad in (dict(g=g[:1]), dict(state=state.transpose(2, 3)), dict(slots=slots.int()), dict(out=out.float()), dict(k=k[:, :1]), dict(v=3)):
        with pytest.raises((TypeError, ValueError)):
            sk.sgemm_bf16_linear_step(**(dict(q=q, k=k, v=v, g=g, state=state, slots=slots, out=out) | bad))
