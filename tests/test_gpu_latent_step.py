"""GPU: one attention layer of a decode step as examples/latent_decode_step.py runs it, against the
same step in FP64, step by step.

Each kernel's output is compared with FP64 arithmetic on the inputs that it really had (the
buffers before it), so that the bounds are those of the single operators; what is new here is
that they run together: one stream, programmatic dependents, a graph, strided views of one
another's buffers, a cache that grows.
"""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_decode_step.py")
_spec = importlib.util.spec_from_file_location("latent_decode_step", _path)
example = importlib.util.module_from_spec(_spec)
import sys  # noqa: E402

sys.modules["latent_decode_step"] = example
_spec.loader.exec_module(example)


def gemm_bound(x, w, y):
    """FP32 sums of K exact products, each addition off by 2^-23 of the terms' sum at most; BF16."""
    return (x.abs() @ w.abs().transpose(-1, -2)) * x.shape[-1] * 2.0 ** -23 + y.abs() * 2.0 ** -8 + 2.0 ** -133


def check_gemm(x, w, y, what):
    x, w = x.cpu().double(), w.cpu().double()
    want = x @ w.transpose(-1, -2)
    D.check(y, want, gemm_bound(x, w, want), what)


@pytest.mark.parametrize("lens,qs", [([100, 1, 64, 333], [1, 1, 1, 1]), ([70, 200], [3, 2]), ([128], [8])])
def test_a_step_in_a_graph_against_fp64(lens, qs):
    """`lens`: rows of each sequence with its new tokens, `qs` of them."""
    s = example.Sizes(hidden=1024, q_rank=512, heads=12, page=16)
    M, B = sum(qs), len(lens)
    layer = example.Layer(s, M, seed=3)
    g = torch.Generator(device=DEV).manual_seed(5)
    W = s.rank + s.rope
    width = max(-(-n // s.page) for n in lens)
    pages = torch.randperm(B * width, generator=g, device=DEV).to(torch.int32).view(B, width)
    cache = torch.randn((B * width, s.page, W), generator=g, device=DEV).to(torch.bfloat16)
    before = cache.clone()
    table = example.rotation_table(512, s.rope)
    x, residual = [torch.randn((M, s.hidden), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    positions = torch.tensor([n_ - q + i for n_, q in zip(lens, qs) for i in range(q)], device=DEV)
    seq = torch.tensor([b for b, q in enumerate(qs) for _ in range(q)], device=DEV)
    slots = pages[seq, positions // s.page].long() * s.page + positions % s.page

    def step():
        return layer.step(x, residual, cache, pages, n, slots, positions, table, cu, max(qs))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8, scales, stream = step()
    for t in (layer.h, layer.res, layer.qa, layer.qn, layer.kv, layer.q, layer.q_full, layer.o, layer.v, layer.y,
              layer.res2, layer.scales):
        t.fill_(float("nan"))
    cache.copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0

    c = {k: v.cpu() for k, v in vars(layer).items() if isinstance(v, torch.Tensor)}
    want, h = D.add_rmsnorm(x.cpu(), c["g_in"], residual.cpu())
    D.check(c["h"], want, D.norm_y_bound(want, s.hidden), "h")
    D.check(c["res"], h, D.residual_bound(h), "residual")
    check_gemm(c["h"], c["w_qa"], c["qa"], "qa")
    check_gemm(c["h"], c["w_kv"], c["kv"], "kv")
    want, _ = D.add_rmsnorm(c["qa"], c["g_q"])
    D.check(c["qn"], want, D.norm_y_bound(want, s.q_rank), "qn")
    check_gemm(c["qn"], c["w_qb"], c["q"].flatten(1), "q")
    for i in range(s.heads):
        check_gemm(c["q"][:, i, : s.nope], c["w_uk"][i], c["q_full"][:, i, : s.rank], f"absorbed query {i}")
        check_gemm(c["o"][:, i], c["w_uv"][i], c["v"][:, i], f"value {i}")
    cos, sin = table.cpu()[positions.cpu()].double().chunk(2, 1)
    want, mag = D.rotate(c["q"][..., s.nope :], cos[:, None], sin[:, None], True)
    D.check(c["q_full"][..., s.rank :], want, D.rotate_bound(want, mag), "rotated query")
    latent, _ = D.add_rmsnorm(c["kv"][:, : s.rank], c["g_kv"])
    key, mag = D.rotate(c["kv"][:, s.rank :], cos, sin, True)
    rows = cache.cpu().flatten(0, 1)
    at = slots.cpu()
    D.check(rows[at], torch.cat([latent, key], 1),
            torch.cat([D.norm_y_bound(latent, s.rank), D.rotate_bound(key, mag)], 1), "cached rows")
    untouched = torch.ones(rows.shape[0], dtype=torch.bool)
    untouched[at] = False
    assert torch.equal(rows[untouched], before.cpu().flatten(0, 1)[untouched])
    want, _, ob, _ = D.latent_attention(c["q_full"], cache.cpu(), pages.cpu(), n.cpu(), s.rank, s.scale, cu.cpu())
    D.check(c["o"], want, ob, "o")
    check_gemm(c["v"].flatten(1), c["w_o"], c["y"], "y")
    want, h = D.add_rmsnorm(c["y"], c["g_out"], c["res"])
    D.check(stream, h, D.residual_bound(h), "stream")
    top = D.scales_of(want, 128)
    D.check(scales, top, top * (D.norm_rel(s.hidden) + 2 * D.U32), "scales")
    v = want / D.spread(scales.cpu().double(), s.hidden, 128)
    D.check(q8, v, v.abs() * (2.0 ** -4 + 4 * D.norm_rel(s.hidden)) + 2.0 ** -10, "q8")


def test_the_example_runs(capsys):
    example.main(4)
    assert "4 steps of 4 sequences" in capsys.readouterr().out
