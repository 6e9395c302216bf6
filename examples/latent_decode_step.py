"""One attention layer of a decode step, from the library's own kernels only.

For M <= 8 new tokens (a few sequences, or one sequence's drafted tokens):

    h        = norm(x + residual)                        sgemm_bf16_add_rmsnorm
    q        = norm(h Wqa^T) Wqb^T,  kv = h Wkv^T        sgemm_bf16_skinny_ex, sgemm_bf16_add_rmsnorm
    q_abs    = q_nope W_uk  (per head)                   sgemm_bf16_skinny_batched_ex
    cache   += [norm(kv latent) | rot(kv rest)],
    q_rot    = rot(q rest)                               sgemm_bf16_latent_append
    o        = attention(q_abs | q_rot, cache)           sgemm_bf16_latent_attention
    y        = (o W_uv per head) Wo^T                    sgemm_bf16_skinny_batched_ex, sgemm_bf16_skinny_ex
    next     = norm(y + residual), 8 bits                sgemm_bf16_add_rmsnorm_e4m3

Every launch is a programmatic dependent of the one before, and the step is captured into a CUDA
graph that is replayed as the sequences grow: lengths, positions, slots and the page table are
read on the device.

    python examples/latent_decode_step.py [steps]
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bf16_skinny_gemm_gb300 as sk  # noqa: E402

CHAIN = sk.SGEMM_FLAG_PDL | sk.SGEMM_FLAG_WEIGHTS_READONLY


@dataclass
class Sizes:
    hidden: int = 4096
    q_rank: int = 1536
    heads: int = 32
    nope: int = 128      # elements of a head's query and value without rotation
    rank: int = 512      # latent vector
    rope: int = 64       # rotated elements
    page: int = 64

    @property
    def scale(self) -> float:
        return (self.nope + self.rope) ** -0.5


class Layer:
    """Weights of the layer, and the buffers of a step for M tokens."""

    def __init__(self, s: Sizes, tokens: int, seed: int = 0, device="cuda"):
        self.s, self.M = s, tokens
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn((n, k), generator=g, device=device) * k ** -0.5).to(torch.bfloat16)

        def gamma(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device=device)).to(torch.bfloat16)

        H, D = s.heads, s.hidden
        self.w_qa, self.w_kv = weight(s.q_rank, D), weight(s.rank + s.rope, D)
        self.w_qb = weight(H * (s.nope + s.rope), s.q_rank)
        self.w_uk = torch.stack([weight(s.rank, s.nope) for _ in range(H)])  # [H, rank, nope]
        self.w_uv = torch.stack([weight(s.nope, s.rank) for _ in range(H)])  # [H, nope, rank]
        self.w_o = weight(D, H * s.nope)
        self.g_in, self.g_q, self.g_kv, self.g_out = gamma(D), gamma(s.q_rank), gamma(s.rank), gamma(D)

        def buf(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=device)

        M = tokens
        self.h, self.res, self.res2, self.y = buf(M, D), buf(M, D), buf(M, D), buf(M, D)
        self.qa, self.qn, self.kv = buf(M, s.q_rank), buf(M, s.q_rank), buf(M, s.rank + s.rope)
        self.q = buf(M, H, s.nope + s.rope)
        self.q_full, self.o = buf(M, H, s.rank + s.rope), buf(M, H, s.rank)
        self.v = buf(M, H, s.nope)
        self.q8 = torch.empty((M, D), dtype=torch.float8_e4m3fn, device=device)
        self.scales = torch.empty((M, D // 128), dtype=torch.float32, device=device)
        self.workspace = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=device)

    def step(self, x, residual, cache, table, lens, slots, positions, cos_sin, cu_q, max_q):
        """Returns (next input in 8 bits, its scales, the residual stream)."""
        s, H = self.s, self.s.heads
        sk.sgemm_bf16_add_rmsnorm(x, self.g_in, residual, y=self.h, residual_out=self.res, flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(self.h, self.w_qa, self.qa, flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(self.h, self.w_kv, self.kv, flags=CHAIN)
        sk.sgemm_bf16_add_rmsnorm(self.qa, self.g_q, y=self.qn, flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(self.qn, self.w_qb, self.q.view(self.M, -1), flags=CHAIN)
        for h in range(0, H, sk.MAX_BATCH):
            sk.sgemm_bf16_skinny_batched_ex(
                [(self.q[:, i, : s.nope], self.w_uk[i], self.q_full[:, i, : s.rank])
                 for i in range(h, min(H, h + sk.MAX_BATCH))], flags=CHAIN)
        sk.sgemm_bf16_latent_append(self.kv, cache, slots, positions, cos_sin, self.g_kv, q=self.q[..., s.nope :],
                                    q_out=self.q_full[..., s.rank :], flags=CHAIN)
        sk.sgemm_bf16_latent_attention(self.q_full, cache, table, lens, s.rank, s.scale, cu_q=cu_q, max_q=max_q,
                                       out=self.o, workspace=self.workspace, flags=CHAIN)
        for h in range(0, H, sk.MAX_BATCH):
            sk.sgemm_bf16_skinny_batched_ex([(self.o[:, i], self.w_uv[i], self.v[:, i])
                                             for i in range(h, min(H, h + sk.MAX_BATCH))], flags=CHAIN)
        sk.sgemm_bf16_skinny_ex(self.v.view(self.M, -1), self.w_o, self.y, flags=CHAIN)
        return sk.sgemm_bf16_add_rmsnorm_e4m3(self.y, self.g_out, self.res, q=self.q8, scales=self.scales,
                                              residual_out=self.res2, flags=CHAIN)


def rotation_table(length: int, rope: int, device="cuda") -> torch.Tensor:
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * (
        10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=device) / rope))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def main(steps: int = 16) -> None:
    s, lens = Sizes(), [1000, 37, 2047, 64]
    B, dev = len(lens), "cuda"
    layer = Layer(s, B)
    width = -(-(max(lens) + steps) // s.page)
    pages = torch.randperm(B * width)[: B * width].to(torch.int32).view(B, width).to(dev)
    cache = torch.randn((B * width, s.page, s.rank + s.rope), device=dev).to(torch.bfloat16)
    table = rotation_table(max(lens) + steps + 1, s.rope)
    x, residual = [torch.randn((B, s.hidden), device=dev).to(torch.bfloat16) for _ in range(2)]
    n = torch.tensor(lens, dtype=torch.int32, device=dev)  # rows cached before the step
    slots, positions = [torch.zeros(B, dtype=torch.int64, device=dev) for _ in range(2)]
    rows = torch.arange(B, device=dev)

    def place():
        """Where this step's token of each sequence goes; the lengths then count it."""
        positions.copy_(n)
        slots.copy_(pages[rows, positions // s.page].long() * s.page + positions % s.page)
        n.add_(1)

    def step():
        return layer.step(x, residual, cache, pages, n, slots, positions, table, None, 1)

    place()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps - 1):
        place()
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if sk.sgemm_device_errors():
        raise RuntimeError("the device error word is set")
    q8, scales, stream = out
    print(f"{steps} steps of {B} sequences, lengths now {n.tolist()}; "
          f"{start.elapsed_time(end) / max(1, steps - 1) * 1e3:.1f} us a step with its bookkeeping; "
          f"residual stream rms {stream.float().square().mean().sqrt().item():.3f}, "
          f"8-bit scales up to {scales.max().item():.4f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 16)
