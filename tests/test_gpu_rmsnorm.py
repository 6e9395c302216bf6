"""GPU: residual add and RMS norm, BF16 and 8-bit outputs, against the FP64 definition."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def inputs(T, width, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, width), generator=g) * std).to(torch.bfloat16)
    r = (torch.randn((T, width), generator=g) * 3 * std).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(torch.bfloat16)
    return x, r, w


def check_q(q, scales, y, group, width):
    """Scales to a few units of FP32; each q within the rounding of e4m3 (y / s with y's own
    relative error on top), of the scale the kernel wrote."""
    want = D.scales_of(y, group)
    rel = D.norm_rel(width) + 2 * D.U32
    D.check(scales, want, want.abs() * rel, "scales")
    s = D.spread(scales.cpu().double(), width, group)
    v = y / s
    D.check(q, v, v.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10, "q")
    assert float(q.float().abs().max()) <= 448


# widths: one chunk and less, a warp's and a block's worth, ends inside a group and inside a
# 16-byte piece, odd ones, rows beyond a block's registers
WIDTHS = [1, 2, 7, 8, 64, 120, 127, 128, 130, 136, 256, 257, 1000, 1024, 1537, 4096, 4100, 8192, 12576, 16384, 16392, 20001]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("add", [True, False])
def test_bf16(T, width, add):
    x, r, w = inputs(T, width, seed=T * 31 + width)
    y, kept = sk.sgemm_bf16_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV) if add else None)
    want, h = D.add_rmsnorm(x, w, r if add else None)
    D.check(y, want, D.norm_y_bound(want, width), "y")
    if add:
        D.check(kept, h, D.residual_bound(h), "residual")
    else:
        assert kept is None


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_e4m3(T, width, group):
    x, r, w = inputs(T, width, seed=T * 37 + width)
    q, scales, kept = sk.sgemm_bf16_add_rmsnorm_e4m3(x.to(DEV), w.to(DEV), r.to(DEV), group=group)
    y, h = D.add_rmsnorm(x, w, r)
    check_q(q, scales, y, group, width)
    D.check(kept, h, D.residual_bound(h), "residual")


@pytest.mark.parametrize("T", [608, 609, 3001])
@pytest.mark.parametrize("width", [96, 200, 512, 768, 1023, 2048])
def test_many_rows(T, width):
    x, r, w = inputs(T, width, seed=width)
    y, h = D.add_rmsnorm(x, w, r)
    got, kept = sk.sgemm_bf16_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV))
    D.check(got, y, D.norm_y_bound(y, width), "y")
    D.check(kept, h, D.residual_bound(h), "residual")
    for group in (0, 128):
        q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(x.to(DEV), w.to(DEV), r.to(DEV), group=group)
        check_q(q, scales, y, group, width)


def test_strided_rows_leave_gaps_alone():
    T, width = 4, 300
    x, r, w = inputs(T, width, seed=1)
    bufs = [torch.full((T, 700), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    views = [b[:, 3 * i + 1 : 3 * i + 1 + width] for i, b in enumerate(bufs)]
    views[0].copy_(x)
    views[1].copy_(r)
    sk.sgemm_bf16_add_rmsnorm(views[0], w.to(DEV), views[1], y=views[2], residual_out=views[3])
    torch.cuda.synchronize()
    want, h = D.add_rmsnorm(x, w, r)
    D.check(views[2], want, D.norm_y_bound(want, width), "y")
    D.check(views[3], h, D.residual_bound(h), "residual")
    for i, b in enumerate(bufs):
        assert torch.all(b[:, : 3 * i + 1] == 9) and torch.all(b[:, 3 * i + 1 + width :] == 9)
    # 8 bits into a view, scales with a stride, and two column ranges of one buffer
    qb = torch.zeros((T, 700), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    sb = torch.full((T, 9), 4.0, device=DEV)
    two = torch.zeros((T, 2 * width), dtype=torch.bfloat16, device=DEV)
    two[:, :width] = x.to(DEV)
    sk.sgemm_bf16_add_rmsnorm_e4m3(two[:, :width], w.to(DEV), r.to(DEV), q=qb[:, 5 : 5 + width], scales=sb[:, 2:5],
                                   residual_out=two[:, width:])
    torch.cuda.synchronize()
    check_q(qb[:, 5 : 5 + width], sb[:, 2:5], want, 128, width)
    D.check(two[:, width:], h, D.residual_bound(h), "residual")
    assert torch.all(sb[:, :2] == 4) and torch.all(sb[:, 5:] == 4)
    assert torch.all(qb[:, :5].float() == 0) and torch.all(qb[:, 5 + width :].float() == 0)


@pytest.mark.parametrize("width", [1000, 4096, 20001])
def test_in_place(width):
    x, r, w = inputs(3, width, seed=2)
    want, h = D.add_rmsnorm(x, w, r)
    xd, rd = x.to(DEV), r.to(DEV)
    y, kept = sk.sgemm_bf16_add_rmsnorm(xd, w.to(DEV), rd, y=xd, residual_out=rd)
    assert y is xd and kept is rd
    D.check(xd, want, D.norm_y_bound(want, width), "y")
    D.check(rd, h, D.residual_bound(h), "residual")


def test_zero_rows_and_eps():
    x, r, w = inputs(3, 256, seed=3)
    x[1] = 0
    r[1] = 0
    x[2] *= 1e-3
    r[2] *= 1e-3
    for eps in (0.0, 1e-6, 1e-2):
        want, _ = D.add_rmsnorm(x, w, r, eps if eps else 1e-300)
        if not eps:
            want[1] = NAN  # 0 / sqrt(0)
        y, _ = sk.sgemm_bf16_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), eps)
        D.check(y, want, D.norm_y_bound(want, 256), f"eps {eps}")
    q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(x.to(DEV), w.to(DEV), r.to(DEV))
    assert torch.all(scales[1] == 1) and torch.all(q[1].float() == 0)
    empty, _ = sk.sgemm_bf16_add_rmsnorm(x.to(DEV)[:0], w.to(DEV))
    assert empty.shape == (0, 256)


@pytest.mark.parametrize("width", [256, 257])
def test_nan_and_infinities_stay_in_their_row(width):
    x, _, w = inputs(4, width, seed=4)
    x[0, 5] = NAN
    x[1, 200] = INF
    x[2, 7] = 3e38  # the square overflows FP32: the row's norm is infinite
    want, _ = D.add_rmsnorm(x, w)
    y, _ = sk.sgemm_bf16_add_rmsnorm(x.to(DEV), w.to(DEV))
    assert torch.all(torch.isnan(y[0]))
    assert torch.isnan(y[1, 200]) and torch.all(y[1, :200] == 0)
    assert torch.all(y[2] == 0)
    D.check(y[3], want[3], D.norm_y_bound(want[3], width), "y")
    for group in (0, 128):
        q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(x.to(DEV), w.to(DEV), group=group)
        assert torch.all(torch.isnan(scales[0])) and torch.all(torch.isnan(q[0].float()))
        assert torch.isnan(scales[1, -1 if not group else 1]) and torch.isnan(q[1, 200].float())
        check_q(q[3:], scales[3:], want[3:], group, width)


def test_large_and_small_values():
    x, r, w = inputs(2, 512, seed=5, std=2.0 ** 40)
    want, h = D.add_rmsnorm(x, w, r)
    y, kept = sk.sgemm_bf16_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV))
    D.check(y, want, D.norm_y_bound(want, 512), "y")
    D.check(kept, h, D.residual_bound(h), "residual")
    x, r, w = inputs(2, 512, seed=6, std=2.0 ** -60)
    want, _ = D.add_rmsnorm(x, w, r, 1e-6)
    q, scales, _ = sk.sgemm_bf16_add_rmsnorm_e4m3(x.to(DEV), w.to(DEV), r.to(DEV), 1e-6)
    check_q(q, scales, want, 128, 512)


def test_other_stream_graph_and_pdl():
    x, r, w = inputs(8, 4096, seed=7)
    want, _ = D.add_rmsnorm(x, w, r)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    y, ro = torch.empty_like(xd), torch.empty_like(xd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sk.sgemm_bf16_add_rmsnorm(xd, wd, rd, y=y, residual_out=ro, stream=s)
    s.synchronize()
    D.check(y, want, D.norm_y_bound(want, 4096), "y")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        for _ in range(3):
            sk.sgemm_bf16_add_rmsnorm(xd, wd, rd, y=y, residual_out=ro,
                                      flags=sk.SGEMM_FLAG_PDL | sk.SGEMM_FLAG_WEIGHTS_READONLY)
    y.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    D.check(y, want, D.norm_y_bound(want, 4096), "y")


def test_refusals_of_the_library():
    x, r, w = [t.to(DEV) for t in inputs(3, 64, seed=8)]
    with pytest.raises(sk.SgemmError) as e:
        sk.sgemm_bf16_add_rmsnorm(x, w, r, residual_out=r[:, :].as_strided((3, 64), (64, 1), 0)[torch.tensor([0, 1, 2])][:, :], eps=NAN)
    assert e.value.status == sk.SGEMM_ERR_INVALID_ARG
    buf = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sk.SgemmError):  # y one row below x
        sk.sgemm_bf16_add_rmsnorm(buf[:3], w, y=buf[1:])
    with pytest.raises(sk.SgemmError):  # y over the residual's copy
        sk.sgemm_bf16_add_rmsnorm(x, w, r, y=buf[:3], residual_out=buf[:3])
    with pytest.raises(sk.SgemmError):
        sk.sgemm_bf16_add_rmsnorm(x, w, r, flags=1 << 10)
