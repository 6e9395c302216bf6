"""GPU: the layers' operators where element offsets pass 32 bits, and where a call's first run is a captured one."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L
from test_gpu_linear import expect, problem
from test_gpu_latent_attention import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def done():
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0


def test_experts_far_apart():
    """The last experts' weights lie behind 2^31 elements."""
    T, E, k, width, F = 5, 16, 2, 256, 136
    g = torch.Generator().manual_seed(1)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(torch.bfloat16)
    x, gu, dn = n(T, width), n(E, 2 * F, width, std=width ** -0.5), n(E, width, F, std=F ** -0.5)
    step = (1 << 31) // (E - 2) + 8
    step -= step % 8
    far = torch.empty((E - 1) * step + gu[0].numel(), dtype=torch.bfloat16, device=DEV)
    far_gu = far.as_strided(gu.shape, (step, width, 1))
    far_dn = far.as_strided(dn.shape, (step, F, 1), gu[0].numel() - dn[0].numel())
    ids = torch.tensor([[15, 0], [14, 15], [3, 13], [15, 14], [1, 15]], dtype=torch.int32)
    weights = torch.rand((T, k), generator=g) + 0.05
    far_gu.copy_(gu)
    want, bound = L.experts(x, gu, dn, ids, weights)
    near_dn = dn.to(DEV)
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), far_gu, near_dn, ids.to(DEV), weights.to(DEV))
    done()
    D.check(y, want, bound, "gate and up far apart")
    far_dn.copy_(dn)
    near_gu = gu.to(DEV)
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), near_gu, far_dn, ids.to(DEV), weights.to(DEV))
    done()
    D.check(y, want, bound, "down far apart")
    far_dn[14, 7] = float("nan")  # outputs that are summed again: tokens that chose expert 15
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), near_gu, far_dn, ids.to(DEV), weights.to(DEV))
    done()
    for t in (0, 2, 4):
        D.check(y[t], want[t], bound[t], "summed again")


@pytest.mark.parametrize("n", [1, 300, 1500])
def test_states_far_apart(n):
    """Slots behind 2^31 elements of the pool."""
    p = problem([n, n], 2, 4, 128, 128, n, pool=7)
    p[5][:] = torch.tensor([6, 5])
    step = (1 << 29) - 4 * 128 * 128
    assert 5 * step > 1 << 31
    far = torch.zeros(6 * step + 4 * 128 * 128, device=DEV)
    s = far.as_strided((7, 4, 128, 128), (step, 128 * 128, 128, 1))
    s.copy_(p[4])
    if n == 1:
        out = sk.sgemm_bf16_linear_step(*(t.to(DEV) for t in p[:4]), s, p[5].to(DEV))
    else:
        cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)
        out = sk.sgemm_bf16_linear_attention(*(t.to(DEV) for t in p[:4]), s, p[5].to(DEV), cu)
    done()
    want, last, ob, sb = expect(*p, [n, n], 1.0, n > 1)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


@pytest.mark.parametrize("n", [100, 1500])
def test_tokens_far_apart(n):
    """Rows of q, k, v and out behind 2^31 elements: token strides of 2^22 and more."""
    p = problem([n], 1, 1, 64, 64, n)
    step = (1 << 31) // (n - 20) // 8 * 8
    far = torch.zeros(n * step, dtype=torch.bfloat16, device=DEV)
    views = []
    for i, t in enumerate(p[:3]):
        views.append(far.as_strided(t.shape, (step, 64, 1), 64 * i))
        views[-1].copy_(t)
    out = far.as_strided((n, 1, 64), (step, 64, 1), 64 * 3)
    s, cu = p[4].to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    sk.sgemm_bf16_linear_attention(*views, p[3].to(DEV), s, p[5].to(DEV), cu, out=out)
    done()
    want, last, ob, sb = expect(*p, [n], 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_a_tree_over_pages_far_apart():
    q, cache, table, ln, cu = make([900], [6], 16, seed=3)
    masks = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {4}, {0, 2, 5}]
    pages, page, W = cache.shape
    step = (1 << 31) // (pages - 2) // 8 * 8
    far = torch.zeros((pages - 1) * step + page * W, dtype=torch.bfloat16, device=DEV)
    c = far.as_strided(cache.shape, (step, W, 1))
    c.copy_(cache)
    tree = torch.tensor([[sum(1 << j for j in m)] for m in masks])
    out, _ = sk.sgemm_bf16_latent_tree_attention(q.to(DEV), c, table.to(DEV), ln.to(DEV), 512, 0.05, tree.to(DEV),
                                                 cu_q=cu.to(DEV), max_q=6)
    done()
    want, _, ob, _ = L.tree_attention(q, cache, table, ln, 512, 0.05, cu, masks)
    D.check(out, want, ob, "out")


FIRST = """
import torch
import bf16_skinny_gemm_gb300 as sk
dev, bf = "cuda", torch.bfloat16
g = torch.Generator(device=dev).manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)
x, w, gu, dn = r(3, 256), r(16, 256), r(16, 256, 256) / 16, r(16, 256, 128) / 16
ids, wt, y = torch.zeros((3, 4), dtype=torch.int32, device=dev), torch.zeros((3, 4), device=dev), torch.zeros_like(x)
q, k, v, decay = r(1500, 2, 64) / 8, r(1500, 2, 64) / 8, r(1500, 4, 64), -torch.rand((1500, 4), generator=g, device=dev)
state, slots, cu, o = torch.zeros((1, 4, 64, 64), device=dev), torch.zeros(1, dtype=torch.int64, device=dev), torch.tensor([0, 1500], dtype=torch.int32, device=dev), torch.zeros_like(v)
tok = torch.zeros((1, 4, 64), dtype=bf, device=dev)
lq, cache, table, ln = r(4, 8, 192), r(8, 64, 192), torch.arange(8, dtype=torch.int32, device=dev)[None], torch.tensor([300], dtype=torch.int32, device=dev)
tree, lo = torch.tensor([[1], [3], [5], [9]], device=dev), torch.zeros((4, 8, 128), dtype=bf, device=dev)
work = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=dev)
def calls():
    sk.sgemm_bf16_moe_route(x, w, 4, ids=ids, weights=wt)
    sk.sgemm_bf16_moe_experts(x, gu, dn, ids, wt, y=y, workspace=work)
    sk.sgemm_bf16_linear_attention(q, k, v, decay, state, slots, cu, out=o, workspace=work)
    sk.sgemm_bf16_linear_step(q[:1], k[:1], v[:1], decay[:1], state, slots, out=tok)
    sk.sgemm_bf16_latent_tree_attention(lq, cache, table, ln, 128, 0.1, tree, max_q=4, out=lo, workspace=work)
outs = (ids, wt, y, o, tok, state, lo)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
a = [t.clone() for t in outs]
state.zero_()
calls()
torch.cuda.synchronize()
assert sk.sgemm_device_errors() == 0
assert all(torch.equal(s, t) for s, t in zip(a, outs)) and all(bool(t.any()) for t in a)
print("alike")
"""


def test_a_first_call_that_is_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=200)
    assert out.returncode == 0 and "alike" in out.stdout, out.stderr[-2000:]
