"""GPU: the operators of a decode step keep the stream's order.

Their kernels are launched as programmatic dependents, so each of them may be there before the
work in front of it is done.  Here that work is slow, writes what the operator reads, reads what
the operator writes, or is no kernel at all (a copy, a fill, an event of another stream), eagerly
and in a graph.  What comes out has to be, bit for bit, what comes out with a synchronisation
before and after each call.
"""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Norm:
    def __init__(self, g):
        self.w = torch.randn(1024, generator=g, device=DEV).to(torch.bfloat16)
        self.inputs = [torch.empty((5, 1024), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        self.outputs = [torch.zeros_like(self.inputs[0]) for _ in range(2)]

    def __call__(self, flags=0):
        sk.sgemm_bf16_add_rmsnorm(self.inputs[0], self.w, self.inputs[1], 1e-6, y=self.outputs[0],
                                  residual_out=self.outputs[1], flags=flags)


class Append:
    def __init__(self, g):
        self.table = torch.randn((64, 64), generator=g, device=DEV)
        self.at = torch.tensor([3, 40, 17, 9], device=DEV)
        self.inputs = [torch.empty((4, 576), dtype=torch.bfloat16, device=DEV),
                       torch.empty((4, 6, 64), dtype=torch.bfloat16, device=DEV)]
        self.outputs = [torch.zeros((4, 16, 576), dtype=torch.bfloat16, device=DEV), torch.zeros_like(self.inputs[1])]

    def __call__(self, flags=0):
        sk.sgemm_bf16_latent_append(self.inputs[0], self.outputs[0], self.at, self.at, self.table, q=self.inputs[1],
                                    q_out=self.outputs[1], flags=flags)


class Attention:
    def __init__(self, g):
        self.inputs = [torch.empty((3, 6, 576), dtype=torch.bfloat16, device=DEV),
                       torch.empty((64, 16, 576), dtype=torch.bfloat16, device=DEV)]
        self.table = torch.randperm(63, generator=g, device=DEV).to(torch.int32).view(3, 21)
        self.lens = torch.tensor([300, 336, 1], dtype=torch.int32, device=DEV)
        self.ws = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
        self.outputs = [torch.zeros((3, 6, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((3, 6), device=DEV)]

    def __call__(self, flags=0):
        sk.sgemm_bf16_latent_attention(self.inputs[0], self.inputs[1], self.table, self.lens, 512, 0.05,
                                       out=self.outputs[0], lse=self.outputs[1], workspace=self.ws, flags=flags)


def make(kind):
    """The operator, data for its inputs (four sets), and its outputs for each, one call at a time."""
    g = torch.Generator(device=DEV).manual_seed(7)
    op = kind(g)
    data = [[torch.randn(x.shape, generator=g, device=DEV).to(torch.bfloat16) for x in op.inputs] for _ in range(4)]
    want = []
    for d in data:
        for x, v in zip(op.inputs, d):
            x.copy_(v)
        for y in op.outputs:
            y.zero_()
        torch.cuda.synchronize()
        op()
        torch.cuda.synchronize()
        want.append([y.clone() for y in op.outputs])
    return op, data, want


def same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def slow():
    """About a tenth of a millisecond of kernels."""
    a = torch.ones((2048, 2048), device=DEV)
    return (a @ a)[0, 0] * 0.0


@pytest.mark.parametrize("kind", [Norm, Append, Attention])
@pytest.mark.parametrize("flags", [0, sk.SGEMM_FLAG_PDL])
def test_after_kernels_that_write_inputs_and_read_outputs(kind, flags):
    op, data, want = make(kind)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kept = []
        for d in data * 3:
            zero = slow().to(torch.bfloat16)
            for x, v in zip(op.inputs, d):
                torch.add(v, zero, out=x)      # a kernel, ready late
            for y in op.outputs:
                y.zero_()
            op(flags)
            zero = slow()
            kept.append([torch.add(y, zero.to(y.dtype)) for y in op.outputs])  # read late, then written again
            for x in op.inputs:
                x.fill_(float("nan"))
        stream.synchronize()
    for i, k in enumerate(kept):
        # x + 0 turns a -0 into 0, so values are compared
        assert all(torch.equal(a, b) for a, b in zip(k, want[i % len(data)])), i


@pytest.mark.parametrize("kind", [Norm, Append, Attention])
@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "host copy", "event", "itself"])
def test_in_a_graph_after_each_kind_of_node(kind, before):
    op, data, want = make(kind)
    source = [torch.empty_like(x) for x in op.inputs]
    host = [x.cpu().pin_memory() for x in source]
    other, stream = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        if before == "copy":
            for x, v in zip(op.inputs, source):
                x.copy_(v)
        elif before == "host copy":
            for x, v in zip(op.inputs, host):
                x.copy_(v, non_blocking=True)
        elif before == "fill":
            for y in op.outputs:
                y.zero_()
        elif before == "event":
            # inputs from two streams at once: one written here, one there
            other.wait_stream(stream)
            with torch.cuda.stream(other):
                op.inputs[1].copy_(source[1])
            op.inputs[0].copy_(source[0])
            stream.wait_stream(other)
        elif before == "itself":
            op(sk.SGEMM_FLAG_PDL)
        op()
        if before == "itself":
            op()
    for i in (1, 3, 0, 2):
        for x, s, h, v in zip(op.inputs, source, host, data[i]):
            s.copy_(v)
            h.copy_(v)
            if before not in ("copy", "host copy", "event"):
                x.copy_(v)
        for y in op.outputs:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(op.outputs, want[i]), i
