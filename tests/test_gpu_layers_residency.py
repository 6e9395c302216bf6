"""GPU: kernels that take half of an SM's tensor memory or all of it have the SM to themselves.

A CTA that waits for so much must not lie beside CTAs of other streams that hold some while they wait for one
that has none yet.  What a call launches is read from its captured graph; nothing of it runs."""
from __future__ import annotations

import ctypes

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk

pytestmark = pytest.mark.gpu
DEV = "cuda"
PER_CTA = 227 << 10  # shared memory that a CTA can have
TWO = 64 << 10       # what two CTAs of the GEMM that uses tensor memory need at least: rings of two stages of 16 KiB


class Kernel(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS"""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launched(call):
    """The kernels of a captured call: (threads a CTA, dynamic shared memory)."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    raw, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(raw, 2) == 0  # (relaxed)
    call(stream)
    assert cu.cuStreamEndCapture(raw, ctypes.byref(graph)) == 0
    n = ctypes.c_size_t()
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    got = []
    for node in nodes:
        k = Kernel()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        got.append((k.block[0], k.shared))
    assert cu.cuGraphDestroy(graph) == 0
    return got


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_prompts(Dk, Dv):
    n = 2000
    q, k = (torch.zeros((n, 2, Dk), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    v, g = torch.zeros((n, 2, Dv), dtype=torch.bfloat16, device=DEV), torch.zeros((n, 2), device=DEV)
    state, slots = torch.zeros((1, 2, Dk, Dv), device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    cu, out = torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.zeros_like(v)
    work = torch.empty(sk.sgemm_linear_attention_workspace(n, 1, 2, Dk, Dv), dtype=torch.uint8, device=DEV)

    def call(stream):
        sk.sgemm_bf16_linear_attention(q, k, v, g, state, slots, cu, out=out, workspace=work, stream=stream)

    call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    kernels = launched(call)
    assert len(kernels) == 3
    whole = [shared for threads, shared in kernels if threads != 256]  # (the joining kernel takes none)
    assert len(whole) == 2 and all(shared > PER_CTA - TWO for shared in whole), kernels


@pytest.mark.parametrize("T", [33, 64, 65, 128])
@pytest.mark.parametrize("width,F", [(64, 40), (512, 256), (2048, 1408), (4096, 1024)])
def test_experts_of_many_tokens(width, F, T):
    """(The down kernel takes a quarter of it at most.)"""
    E, k = 4, 2
    x = torch.zeros((T, width), dtype=torch.bfloat16, device=DEV)
    gu, dn = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((E, 2 * F, width), (E, width, F)))
    ids, weights = torch.zeros((T, k), dtype=torch.int32, device=DEV), torch.zeros((T, k), device=DEV)
    y, work = torch.zeros_like(x), torch.empty(sk.sgemm_moe_experts_workspace(T, E, k, width, F), dtype=torch.uint8, device=DEV)

    def call(stream):
        sk.sgemm_bf16_moe_experts(x, gu, dn, ids, weights, y=y, workspace=work, stream=stream)

    call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    kernels = launched(call)
    assert len(kernels) == 2 and kernels[0][1] > PER_CTA - TWO, kernels
