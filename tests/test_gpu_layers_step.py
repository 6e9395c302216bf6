"""GPU: the layers' operators together, as a step calls them, captured into one graph that is replayed
on other inputs.  Each operator's result is held against FP64 on what its call was given."""
from __future__ import annotations

import torch
import pytest

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHAIN = sk.SGEMM_FLAG_PDL | sk.SGEMM_FLAG_WEIGHTS_READONLY


def weight(g, *shape):
    return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(torch.bfloat16).to(DEV)


def buf(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def captured(step):
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


def test_a_linear_attention_layer_with_experts():
    """norm, projections, one token of linear attention, output projection, norm, router, experts (one
    of them for every token), norm of the sum: four sequences, one of them padded."""
    M, hidden, H, dk, E, k, width = 4, 512, 4, 64, 12, 3, 192
    g = torch.Generator().manual_seed(1)
    ones = torch.ones(hidden, dtype=torch.bfloat16, device=DEV)
    w_qkv, w_o = weight(g, 3 * H * dk, hidden), weight(g, hidden, H * dk)
    w_r, w_gu, w_dn = weight(g, E, hidden), weight(g, E + 1, 2 * width, hidden), weight(g, E + 1, hidden, width)
    x, res = buf(M, hidden), buf(M, hidden)
    h, res1, qkv, o, y, h2, res2, z, h3, res3 = (buf(M, hidden), buf(M, hidden), buf(M, 3 * H * dk), buf(M, H, dk), buf(M, hidden),
                                                 buf(M, hidden), buf(M, hidden), buf(M, hidden), buf(M, hidden), buf(M, hidden))
    q, kk, v = (t.unflatten(1, (H, dk)) for t in qkv.split(H * dk, 1))
    decay, state, before = buf(M, H, dtype=torch.float32), buf(6, H, dk, dk, dtype=torch.float32), buf(6, H, dk, dk, dtype=torch.float32)
    slots = torch.tensor([5, 0, -1, 2], device=DEV)
    ids = torch.full((M, k + 1), E, dtype=torch.int32, device=DEV)
    weights = torch.ones((M, k + 1), device=DEV)
    work = torch.empty(sk.sgemm_moe_experts_workspace(M, E + 1, k + 1, hidden, width), dtype=torch.uint8, device=DEV)

    def step():
        sk.sgemm_bf16_add_rmsnorm(x, ones, res, y=h, residual_out=res1, flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(h, w_qkv, qkv, flags=CHAIN)
        sk.sgemm_bf16_linear_step(q, kk, v, decay, state, slots, dk ** -0.5, out=o, flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(o.view(M, -1), w_o, y, flags=CHAIN)
        sk.sgemm_bf16_add_rmsnorm(y, ones, res1, y=h2, residual_out=res2, flags=CHAIN)
        sk.sgemm_bf16_moe_route(h2, w_r, k, ids=ids[:, :k], weights=weights[:, :k], flags=CHAIN)
        sk.sgemm_bf16_moe_experts(h2, w_gu, w_dn, ids, weights, y=z, workspace=work, flags=CHAIN)
        sk.sgemm_bf16_add_rmsnorm(z, ones, res2, y=h3, residual_out=res3, flags=CHAIN)

    graph = captured(step)
    for seed in range(3):
        g = torch.Generator().manual_seed(10 + seed)
        x.copy_(torch.randn((M, hidden), generator=g))
        res.copy_(torch.randn((M, hidden), generator=g))
        decay.copy_(-torch.rand((M, H), generator=g))
        state.copy_(torch.randn(state.shape, generator=g))
        before.copy_(state)
        graph.replay()
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0
        for b, slot in enumerate(slots.tolist()):
            if slot < 0:
                assert torch.all(o[b] == 0)
                continue
            r = slice(b, b + 1)
            want, last, ob, sb = L.linear(q[r].cpu(), kk[r].cpu(), v[r].cpu(), decay[r].cpu(), before[slot].cpu(), dk ** -0.5, False)
            D.check(o[r], want, ob, "linear attention")
            D.check(state[slot], last, sb, "state")
        assert torch.equal(state[[1, 3, 4]], before[[1, 3, 4]])
        L.check_route(ids[:, :k], weights[:, :k], h2.cpu(), w_r.cpu(), k)
        assert torch.all(ids[:, k] == E) and torch.all(weights[:, k] == 1)
        want, bound = L.experts(h2.cpu(), w_gu.cpu(), w_dn.cpu(), ids.cpu(), weights.cpu())
        D.check(z, want, bound, "experts")
        n64, s64 = D.add_rmsnorm(z.cpu(), ones.cpu(), res2.cpu())
        D.check(h3, n64, D.norm_y_bound(n64, hidden), "norm")
        D.check(res3, s64, D.residual_bound(s64), "residual")


def test_a_tree_of_drafts_over_the_cache_with_experts():
    """Drafted tokens: their rows into the cache (at the positions of their depth), attention by the
    tree, router and experts over all of them."""
    H, R, E, page, n, context = 8, 128, 32, 16, 9, 70
    hidden, experts, k, width = 256, 6, 2, 64
    g = torch.Generator().manual_seed(2)
    parents = [-1, 0, 0, 1, 1, 2, 3, 5, 6]
    masks, depth = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else set()) | {i})
        depth.append(depth[p] + 1 if p >= 0 else 0)
    pages = torch.randperm(8, generator=g)[:6].to(torch.int32)
    cache = buf(8, page, R + E)
    at = torch.arange(context, context + n)
    slots = (pages[at // page].long() * page + at % page).to(DEV)
    positions = (context + torch.tensor(depth)).to(DEV)
    angle = torch.arange(200)[:, None] * 1e4 ** (-torch.arange(E // 2) / (E // 2))
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    kv, q = buf(n, R + E), buf(n, H, R + E)
    tree = torch.tensor([sum(1 << j for j in m) for m in masks], device=DEV)[:, None]
    lens = torch.tensor([context + n], dtype=torch.int32, device=DEV)
    table = pages[None].to(DEV)
    out, lse = buf(n, H, R), buf(n, H, dtype=torch.float32)
    w_o, w_r, w_gu, w_dn = weight(g, hidden, H * R), weight(g, experts, hidden), weight(g, experts, 2 * width, hidden), weight(g, experts, hidden, width)
    h, z = buf(n, hidden), buf(n, hidden)
    ids, weights = buf(n, k, dtype=torch.int32), buf(n, k, dtype=torch.float32)
    ws = torch.empty(sk.sgemm_latent_tree_attention_workspace(1, H, R, E, page, 6, n), dtype=torch.uint8, device=DEV)
    work = torch.empty(sk.sgemm_moe_experts_workspace(n, experts, k, hidden, width), dtype=torch.uint8, device=DEV)
    scale = (R + E) ** -0.5

    def step():
        sk.sgemm_bf16_latent_append(kv, cache, slots, positions, cos_sin, q=q[..., R:], q_out=q[..., R:], flags=CHAIN)
        sk.sgemm_bf16_latent_tree_attention(q, cache, table, lens, R, scale, tree, max_q=n, out=out, lse=lse, workspace=ws, flags=CHAIN)
        for i in range(0, n, 8):
            sk.sgemm_bf16_skinny_ex(out.view(n, -1)[i : i + 8], w_o, h[i : i + 8], flags=CHAIN)
        sk.sgemm_bf16_moe_route(h, w_r, k, ids=ids, weights=weights, flags=CHAIN)
        sk.sgemm_bf16_moe_experts(h, w_gu, w_dn, ids, weights, y=z, workspace=work, flags=CHAIN)

    graph = captured(step)
    for seed in range(2):
        g = torch.Generator().manual_seed(20 + seed)
        cache.copy_(torch.randn(cache.shape, generator=g))
        kv.copy_(torch.randn(kv.shape, generator=g))
        q.copy_(torch.randn(q.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0
        assert torch.equal(cache.view(-1, R + E)[slots, :R], kv[:, :R])
        want, wlse, ob, lb = L.tree_attention(q.cpu(), cache.cpu(), table.cpu(), [context + n], R, scale, [0, n], masks)
        D.check(out, want, ob, "attention")
        D.check(lse, wlse, lb, "lse")
        L.check_route(ids, weights, h.cpu(), w_r.cpu(), k)
        want, bound = L.experts(h.cpu(), w_gu.cpu(), w_dn.cpu(), ids.cpu(), weights.cpu())
        D.check(z, want, bound, "experts")
