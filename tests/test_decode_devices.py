"""The decode operators' tensors are all on the current device, where the library launches: both ways
of the binding refuse any other before they call it."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import decode

BF16, F32, I32, I64, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn

# each operator's tensors by name, and the call
CASES = {
    "norm": (dict(x=((2, 64), BF16), weight=((64,), BF16), residual=((2, 64), BF16), y=((2, 64), BF16),
                  residual_out=((2, 64), BF16)), sk.sgemm_bf16_add_rmsnorm, {}),
    "norm_e4m3": (dict(x=((2, 64), BF16), weight=((64,), BF16), q=((2, 64), E4M3), scales=((2, 1), F32)),
                  sk.sgemm_bf16_add_rmsnorm_e4m3, {}),
    "append": (dict(kv=((3, 96), BF16), cache=((4, 16, 96), BF16), slots=((3,), I64), positions=((3,), I64),
                    cos_sin=((50, 32), F32), weight=((64,), BF16), q=((3, 5, 32), BF16), q_out=((3, 5, 32), BF16)),
               sk.sgemm_bf16_latent_append, {}),
    "attention": (dict(q=((2, 8, 192), BF16), cache=((6, 16, 192), BF16), block_table=((2, 3), I32), seq_lens=((2,), I32),
                       cu_q=((3,), I32), out=((2, 8, 128), BF16), lse=((2, 8), F32), workspace=((64 << 20,), torch.uint8)),
                  sk.sgemm_bf16_latent_attention, dict(rank=128, scale=0.1)),
}
EACH = [(name, t) for name, (tensors, _, _) in CASES.items() for t in tensors]


class Fake:
    """What the binding reads of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device, self.nbytes = f"cuda:{index}", self.shape.numel()

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True


@pytest.fixture
def calls(monkeypatch):
    calls = []
    monkeypatch.setattr(decode, "_call", lambda name, *args: calls.append(name))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return calls


@pytest.mark.parametrize("name,other", EACH)
def test_one_tensor_on_another_device(calls, name, other):
    tensors, function, more = CASES[name]
    with pytest.raises(ValueError, match=f"{other} is on cuda:0, the current device is cuda:1"):
        function(**{t: Fake(*a, 0 if t == other else 1) for t, a in tensors.items()}, **more)
    assert not calls


@pytest.mark.parametrize("name", CASES)
def test_all_on_a_device_that_is_not_the_current_one_and_all_on_it(calls, name):
    tensors, function, more = CASES[name]
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        function(**{t: Fake(*a, 0) for t, a in tensors.items()}, **more)
    assert not calls
    function(**{t: Fake(*a, 1) for t, a in tensors.items()}, **more)
    assert len(calls) == 1


class Elsewhere(torch.Tensor):
    """A tensor that says that it is on the second device, and has no memory."""

    @staticmethod
    def __new__(cls, shape, dtype):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:1")

    @classmethod
    def __torch_dispatch__(cls, function, types, args=(), kwargs=None):
        raise RuntimeError(f"{function} of a tensor without memory")


@pytest.mark.gpu
@pytest.mark.parametrize("name,other", EACH)
def test_the_short_way_leaves_a_tensor_on_another_device(name, other):
    tensors, function, more = CASES[name]
    args = {t: torch.zeros(shape, dtype=torch.float32, device="cuda").to(dtype) for t, (shape, dtype) in tensors.items()}
    args[other] = Elsewhere(*tensors[other])
    assert torch.cuda.current_device() == 0
    with pytest.raises(ValueError, match=f"{other} is on cuda:1, the current device is cuda:0"):
        function(**args, **more)
