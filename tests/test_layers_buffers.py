"""Buffers that the layers' calls make for themselves belong to the stream they run on, and all
tensors have to be on the current device, where the library launches."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import layers
from test_buffers_of_a_call import BF16, F32, HERE, I32, I64, THERE, Stream, log  # noqa: F401
from test_decode_devices import Fake

HIDDEN, WIDTH = 64, 40
# each operator's tensors by name, the call, and what it makes for itself where it is not given
CASES = {
    "route": (dict(x=((2, HIDDEN), BF16), w=((8, HIDDEN), BF16), bias=((8,), F32), ids=((2, 3), I32), weights=((2, 3), F32)),
              sk.sgemm_bf16_moe_route, dict(k=3), {"ids": ((2, 3), True), "weights": ((2, 3), True)}),
    "experts": (dict(x=((2, HIDDEN), BF16), w_gate_up=((4, 2 * WIDTH, HIDDEN), BF16), w_down=((4, HIDDEN, WIDTH), BF16), ids=((2, 3), I32),
                     weights=((2, 3), F32), y=((2, HIDDEN), BF16), workspace=((1 << 20,), torch.uint8)),
                sk.sgemm_bf16_moe_experts, {}, {"y": ((2, HIDDEN), True), "workspace": ((4 * 2 * WIDTH * 2,), False)}),
    "tree": (dict(q=((2, 8, 192), BF16), cache=((6, 16, 192), BF16), block_table=((2, 3), I32), seq_lens=((2,), I32), tree=((2, 1), I64),
                  cu_q=((3,), I32), out=((2, 8, 128), BF16), lse=((2, 8), F32), workspace=((64 << 20,), torch.uint8)),
             sk.sgemm_bf16_latent_tree_attention, dict(rank=128, scale=0.1), {"out": ((2, 8, 128), True), "workspace": ((7 << 10,), False)}),
    "step": (dict(q=((3, 2, 64), BF16), k=((3, 2, 64), BF16), v=((3, 4, 128), BF16), g=((3, 4), F32), state=((5, 4, 64, 128), F32),
                  slots=((3,), I64), out=((3, 4, 128), BF16)), sk.sgemm_bf16_linear_step, {}, {"out": ((3, 4, 128), True)}),
    "prompt": (dict(q=((9, 2, 64), BF16), k=((9, 2, 64), BF16), v=((9, 4, 128), BF16), g=((9, 4), F32), state=((5, 4, 64, 128), F32),
                    slots=((3,), I64), cu=((4,), I32), fresh=((3,), I32), out=((9, 4, 128), BF16), workspace=((1 << 20,), torch.uint8)),
               sk.sgemm_bf16_linear_attention, {}, {"out": ((9, 4, 128), True), "workspace": ((9 << 10,), False)}),
}
EACH = [(name, t) for name, (tensors, *_) in CASES.items() for t in tensors]


@pytest.fixture
def calls(monkeypatch):
    calls = []
    monkeypatch.setattr(layers, "_call", lambda name, *args: calls.append(name))
    monkeypatch.setattr(layers, "sgemm_latent_tree_attention_workspace", lambda *a: 7 << 10)
    monkeypatch.setattr(layers, "sgemm_linear_attention_workspace", lambda *a: 9 << 10)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, Fake))
    return calls


@pytest.mark.parametrize("name,other", EACH)
def test_one_tensor_on_another_device(monkeypatch, calls, name, other):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    tensors, function, more, _ = CASES[name]
    with pytest.raises(ValueError, match=f"{other} is on cuda:0, the current device is cuda:1"):
        function(**{t: Fake(*a, 0 if t == other else 1) for t, a in tensors.items()}, **more)
    assert not calls


@pytest.mark.parametrize("name", CASES)
def test_all_on_the_current_device(monkeypatch, calls, name):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    tensors, function, more, _ = CASES[name]
    function(**{t: Fake(*a, 1) for t, a in tensors.items()}, **more)
    assert len(calls) == 1


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("stream", [None, HERE, THERE, "there"])
def test_what_a_call_makes_comes_from_its_stream(monkeypatch, calls, name, stream):
    made = []

    def empty(shape, dtype, device, stream=None, returned=True):
        made.append((tuple(shape), stream, returned))
        return Fake(shape, dtype, 0)

    monkeypatch.setattr(layers, "_empty", empty)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    tensors, function, more, own = CASES[name]
    s = Stream(THERE) if stream == "there" else stream
    monkeypatch.setattr(layers, "_raw", lambda x: x)
    function(**{t: Fake(*a, 0) for t, a in tensors.items() if t not in own}, **more, stream=s)
    assert made == [(shape, s, returned) for shape, returned in own.values()] and len(calls) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["experts", "step", "prompt"])
def test_a_call_on_a_side_stream_with_its_own_buffers(name):
    """What the current stream's pending work reads is not what the call is handed."""
    g = torch.Generator(device="cuda").manual_seed(1)
    side = torch.cuda.Stream()
    if name == "experts":
        x = torch.randn((2, HIDDEN), generator=g, device="cuda").to(BF16)
        gu, dn = (torch.randn(s, generator=g, device="cuda").to(BF16) for s in ((4, 2 * WIDTH, HIDDEN), (4, HIDDEN, WIDTH)))
        args = (x, gu, dn, torch.tensor([[0, 3], [1, 2]], dtype=I32, device="cuda"), torch.rand((2, 2), generator=g, device="cuda"))
        call = sk.sgemm_bf16_moe_experts
    else:
        n = 3 if name == "step" else 200
        q, k = (torch.randn((n, 2, 64), generator=g, device="cuda").to(BF16) * 0.1 for _ in range(2))
        v = torch.randn((n, 4, 128), generator=g, device="cuda").to(BF16)
        d, state = -torch.rand((n, 4), generator=g, device="cuda"), torch.randn((3, 4, 64, 128), generator=g, device="cuda")
        if name == "step":
            args, call = (q, k, v, d, state, torch.arange(3, device="cuda")), sk.sgemm_bf16_linear_step
        else:
            args = (q, k, v, d, state, torch.zeros(1, dtype=I64, device="cuda"), torch.tensor([0, n], dtype=I32, device="cuda"))
            call = sk.sgemm_bf16_linear_attention
    copies = [a.clone() for a in args]
    want = call(*copies)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = call(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
