"""GPU: the short way from tensors to the decode operators' calls (native/marshal.cpp) and the long
one (decode.py) are the same call: same bits, same refusals."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Never:
    """A short way that leaves every call to the long one."""

    def __getattr__(self, name):
        return lambda *args: -1


class Only:
    """The short way, which must not leave the call."""

    def __init__(self, module):
        self.module = module

    def __getattr__(self, name):
        def call(*args):
            status = getattr(self.module, name)(*args)
            assert status >= 0, f"{name} was left to the long way"
            return status
        return call


def both(monkeypatch, call, outputs):
    """Runs the call both ways on outputs filled alike; the bits of each way's outputs."""
    decode._short.add_rmsnorm(None, None, None, 0.0, 0, None, None, None, 0, None)  # loads the module
    module, got = decode._short, []
    for way in (Only(module), Never()):
        for t in outputs:
            t.view(torch.uint8).fill_(17) if t.is_contiguous() else t.fill_(17)
        monkeypatch.setattr(decode, "_short", way)
        call()
        torch.cuda.synchronize()
        monkeypatch.setattr(decode, "_short", module)
        got.append([t.clone() for t in outputs])
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def bf(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("form", ["bf16", 0, 128])
def test_norm_both_ways(monkeypatch, T, form):
    x, w, r = bf(T, 900, seed=1)[:, 7:607], bf(600, seed=2), bf(T, 600, seed=3)
    y, kept = torch.zeros_like(r), torch.zeros((T, 2, 600), dtype=torch.bfloat16, device=DEV)[:, 1]
    q = torch.zeros((T, 600), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros((T, 5 if form == 128 else 1), device=DEV)
    if form == "bf16":
        both(monkeypatch, lambda: sk.sgemm_bf16_add_rmsnorm(x, w, r, 1e-5, y=y, residual_out=kept), [y, kept])
        both(monkeypatch, lambda: sk.sgemm_bf16_add_rmsnorm(x, w, y=y), [y])
    else:
        both(monkeypatch, lambda: sk.sgemm_bf16_add_rmsnorm_e4m3(x, w, r, group=form, q=q, scales=scales, residual_out=kept,
                                                                 stream=torch.cuda.current_stream()), [q, scales, kept])


@pytest.mark.parametrize("T,H", [(1, 0), (1, 3), (5, 4)])
def test_append_both_ways(monkeypatch, T, H):
    kv, w = bf(T, 192, seed=1), bf(128, seed=2)
    cache = bf(3, 2, 8, 192, seed=3)[:, 1]
    slots, pos = torch.arange(T, device=DEV) * 3, torch.arange(T, device=DEV)
    cs = torch.rand((9, 64), device=DEV)
    q, q_out = (bf(T, H, 100, seed=4)[..., 30:94], torch.zeros((H, T, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1)) \
        if H else (None, None)
    for weight in (w, None):
        both(monkeypatch, lambda: sk.sgemm_bf16_latent_append(kv, cache, slots, pos, cs, weight, q=q, q_out=q_out,
                                                              interleaved=weight is None,
                                                              stream=torch.cuda.current_stream().cuda_stream),
             [cache] + ([q_out] if H else []))


@pytest.mark.parametrize("cu", [True, False])
def test_attention_both_ways(monkeypatch, cu):
    q, cache = bf(4, 6, 192, seed=1), bf(9, 16, 192, seed=2)
    table = torch.arange(8, device=DEV, dtype=torch.int32).view(2, 4)
    lens = torch.tensor([50, 33], dtype=torch.int32, device=DEV)
    cu_q = torch.tensor([0, 1, 4] if cu else [0, 2, 4], dtype=torch.int32, device=DEV)
    out, lse = torch.zeros((4, 6, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 6), device=DEV)
    ws = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=DEV)
    for l in (lse, None):
        both(monkeypatch, lambda: sk.sgemm_bf16_latent_attention(q, cache, table, lens, 128, 0.1, cu_q=cu_q if cu else None,
                                                                 max_q=3 if cu else 2, out=out, lse=l, workspace=ws),
             [out] + ([lse] if l is not None else []))


def test_what_is_not_well_formed_is_left_to_the_checks():
    x, w, y = bf(2, 64), bf(64), bf(2, 64)
    for bad in (dict(weight=w.float()), dict(weight=w[:60]), dict(weight=w.cpu()), dict(x=x.t()), dict(y=y[:1]), dict(y=3),
                dict(residual=bf(2, 32)), dict(x=x.view(2, 8, 8))):
        args = dict(x=x, weight=w, y=y) | bad
        with pytest.raises((TypeError, ValueError)):
            sk.sgemm_bf16_add_rmsnorm(**args)
    with pytest.raises(sk.SgemmError) as e:  # well formed, but y lies one row below x
        b = bf(3, 64)
        sk.sgemm_bf16_add_rmsnorm(b[:2], w, y=b[1:])
    assert e.value.status == sk.SGEMM_ERR_INVALID_ARG
