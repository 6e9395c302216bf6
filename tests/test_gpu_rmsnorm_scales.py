"""GPU: the 8-bit norm's scales and quotients at the ends of FP32's range.  The inputs are such that
y, its scale and y / scale are exact, so what has to come out is known bit for bit."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNIT = 2.0 ** -149  # the smallest positive FP32
SMALL = 2.0 ** -133  # the smallest positive BF16


def view(rows, shift):
    """The rows on the device, starting `shift` elements off 16 bytes."""
    T, width = rows.shape
    buf = torch.zeros((T, width + 16), dtype=torch.bfloat16, device=DEV)
    buf[:, shift : shift + width] = rows.to(DEV)
    return buf[:, shift : shift + width]


@pytest.mark.parametrize("width,shift", [(512, 0), (512, 2), (512, 1), (20480, 0)])
@pytest.mark.parametrize("times", [1, 3, 4])
def test_a_group_of_subnormal_values_beside_large_ones(width, shift, times):
    """A quarter of the columns is 2^10, so that the root mean square is 2^9.  The first group holds
    0 and +-times 2^-133: y = +-times 128 units.  The scale is the smallest FP32 that is no less than
    times 128 / 448 units."""
    x = torch.zeros((3, width), dtype=torch.float64)
    x[:, width // 4 : width // 2] = 2.0 ** 10
    x[1, 5], x[1, 70], x[2, :128:2] = times * SMALL, -times * SMALL, times * SMALL
    want = x[:, :128] * 2.0 ** -9
    s = 1 if times < 4 else 2
    q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(view(x.to(torch.bfloat16), shift), torch.ones(width, dtype=torch.bfloat16, device=DEV),
                                                  eps=0.0)
    torch.cuda.synchronize()
    q, scales = q.cpu().double(), scales.cpu().double()
    assert scales[0, 0] == 1 and torch.all(scales[1:, 0] == s * UNIT)
    assert torch.equal(q[:, :128] * scales[:, :1], want)
    assert torch.all(q[:, width // 4 : width // 2] == 448) and torch.all(torch.isfinite(q))


@pytest.mark.parametrize("width,shift", [(512, 0), (512, 2), (512, 1), (20480, 0)])
@pytest.mark.parametrize("group", [0, 128])
def test_rows_of_subnormal_values(width, shift, group):
    """x is 0 and +-1 in equal parts, eps makes the root 2^10, the weight is 2^-133: y = +-64 units,
    and its scale is one unit."""
    x = torch.zeros((2, width), dtype=torch.float64)
    x[0, ::2], x[1, 1::4], x[1, 3::4] = 1, -1, 1
    w = torch.full((width,), SMALL, dtype=torch.float64).to(torch.bfloat16)
    q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(view(x.to(torch.bfloat16), shift), w.to(DEV), eps=2.0 ** 20 - 0.5, group=group)
    torch.cuda.synchronize()
    assert torch.all(scales.cpu().double() == UNIT)
    assert torch.equal(q.cpu().double(), 64 * x)


@pytest.mark.parametrize("width,shift", [(512, 0), (512, 1), (4096, 0), (20480, 0)])
@pytest.mark.parametrize("group", [0, 128])
def test_each_quotient_is_rounded_to_the_nearest(width, shift, group):
    """x is +-1 and eps 0, so that y is +-the weight.  A quotient within 2^-22 of the middle of two
    values (two roundings of FP32 come within 2^-23) may round to either, every other one does not."""
    g = torch.Generator().manual_seed(width + group)
    w = torch.randn(width, generator=g).to(torch.bfloat16)
    x = torch.where(torch.rand((40, width), generator=g) < 0.5, -1.0, 1.0)
    q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(view(x.to(torch.bfloat16), shift), w.to(DEV), eps=0.0, group=group)
    torch.cuda.synchronize()
    y = x * w.float()
    top = torch.stack([p.abs().amax(1) for p in y.split(group or width, 1)], 1)
    assert torch.equal(scales.cpu(), top / 448)  # FP32 division, as the kernel's
    s = scales.cpu().double()
    v = y.double() / (s.repeat_interleave(group, 1)[:, :width] if group else s)
    low, high = [(v * (1 + d)).clamp(-448, 448).float().to(torch.float8_e4m3fn).float() for d in (-2.0 ** -22, 2.0 ** -22)]
    got = q.cpu().float()
    assert torch.all((got == low) | (got == high))
