"""Buffers that a call makes for itself (outputs and scratch that it is not given) belong to the
stream it runs on.

The allocator hands a free block of a stream out again at once, for work that is queued behind
whatever still uses it on that stream.  A kernel on another stream is not behind that.  On the CPU:
which stream each buffer comes from.  On the GPU: what is left in such a block by the current
stream's pending work, and what that work reads.
"""
from __future__ import annotations

import contextlib

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
from bf16_skinny_gemm_gb300 import decode

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
HERE, THERE = 0x700, 0x900  # stream handles


class Fake:
    """What the binding reads of a contiguous CUDA tensor."""

    is_cuda, device, nbytes = True, "cuda:0", 1 << 30

    def __init__(self, shape, dtype=BF16, log=None):
        self.shape, self.dtype, self.log = torch.Size(shape), dtype, log

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        self.log.append(("used on", tuple(self.shape), stream.cuda_stream))


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class External(Stream):
    def __init__(self, handle, device=None):
        super().__init__(handle or 0xB00)  # what torch does with 0: a stream from its pool


@pytest.fixture
def log(monkeypatch):
    """(shape, stream that it comes from) of each buffer made, and the streams recorded for it."""
    log, now = [], [HERE]

    @contextlib.contextmanager
    def stream(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    def empty(shape, dtype, device):
        log.append((tuple(shape), now[-1]))
        return Fake(shape, dtype, log)

    def call(name, args, t, stream):
        log.append(("call", stream))

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(decode, "_call", call)
    monkeypatch.setattr(decode, "sgemm_latent_attention_workspace", lambda *a: 4096)
    return log


def norm(stream):
    sk.sgemm_bf16_add_rmsnorm(Fake((2, 64)), Fake((64,)), Fake((2, 64)), stream=stream)
    return {(2, 64)}


def norm_e4m3(stream):
    sk.sgemm_bf16_add_rmsnorm_e4m3(Fake((2, 200)), Fake((200,)), stream=stream)
    return {(2, 200), (2, 2)}


def append(stream):
    sk.sgemm_bf16_latent_append(Fake((3, 96)), Fake((4, 16, 96)), Fake((3,), I64), Fake((3,), I64), Fake((50, 32), F32),
                                q=Fake((3, 5, 32)), stream=stream)
    return {(3, 5, 32)}


def attention(stream):
    sk.sgemm_bf16_latent_attention(Fake((2, 8, 192)), Fake((6, 16, 192)), Fake((2, 3), I32), Fake((2,), I32), 128, 0.1,
                                   stream=stream)
    return {(2, 8, 128), (4096,)}


@pytest.mark.parametrize("operator", [norm, norm_e4m3, append, attention])
@pytest.mark.parametrize("there", [THERE, 0])  # 0: the default stream
def test_buffers_come_from_the_calls_stream(log, operator, there):
    made = operator(there)
    assert ("call", there) in log
    assert {(shape, s) for shape, s, *_ in log if shape not in ("call", "used on")} == {(shape, there) for shape in made}
    # what is returned is used on the current stream, what is not returned is not
    assert {r[1:] for r in log if r[0] == "used on"} == {(shape, HERE) for shape in made if shape != (4096,)}


@pytest.mark.parametrize("operator", [norm, norm_e4m3, append, attention])
@pytest.mark.parametrize("stream", [None, HERE])
def test_buffers_of_a_call_on_the_current_stream(log, operator, stream):
    made = operator(stream)
    assert {r for r in log if r[0] != "call"} == {(shape, HERE) for shape in made}


class Library:
    """Takes every call and launches nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


def test_gemm_outputs_come_from_the_calls_stream(log, monkeypatch):
    monkeypatch.setattr(torch, "Tensor", Fake)  # (the checks ask for one)
    monkeypatch.setattr(sk, "load", Library)
    x, W = Fake((2, 64)), Fake((48, 64))
    for call in (sk.sgemm_bf16_skinny, sk.sgemm_bf16_skinny_ex, sk.sgemm_bf16_skinny_f32out_ex, sk.sgemm_bf16_skinny_splitk_noalloc,
                 lambda x, W, stream: sk.sgemm_bf16_skinny_batched([(x, W)], stream=stream),
                 lambda x, W, stream: sk.sgemm_bf16_skinny_batched_ex([(x, W)], stream=stream)):
        log.clear()
        call(x, W, stream=THERE)
        assert log == [((2, 48), THERE), ("used on", (2, 48), HERE)]


# --------------------------------------------------------------------------------- on the GPU
def late_use(shape, dtype):
    """A block of this size that the current stream still wants: a kernel that is far from its turn
    adds to it and keeps the sum.  Returns what that has to be, and where it will be."""
    block = torch.full(shape, 1, dtype=dtype, device="cuda")
    kept = torch.empty_like(block)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    block.add_(1)
    kept.copy_(block)
    return kept  # the block goes back to the allocator here


@pytest.mark.gpu
def test_a_block_the_current_stream_still_uses_is_left_alone():
    """The call on another stream is done long before the current stream's turn: neither its scratch
    and outputs nor that stream's data are touched by the other."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn((2, 32, 576), generator=g).to(BF16)
    cache = torch.randn((20, 64, 576), generator=g).to(BF16)
    table = torch.arange(20, dtype=I32).view(2, 10)
    lens = torch.tensor([640, 500], dtype=I32)
    dev = [t.to("cuda") for t in (q, cache, table, lens)]
    want, _, bound, _ = D.latent_attention(q, cache, table, lens, 512, 0.05, [0, 1, 2])
    need = sk.sgemm_latent_attention_workspace(2, 32, 512, 64, 64, 10)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = late_use((need,), torch.uint8)
    out, _ = sk.sgemm_bf16_latent_attention(*dev, 512, 0.05, stream=s)
    torch.cuda.synchronize()
    assert bool((kept == 2).all())
    D.check(out, want, bound, "out")

    x, w = torch.randn((64, 4096), generator=g).to(BF16), torch.ones(4096).to(BF16)
    xd, wd = x.to("cuda"), w.to("cuda")
    want, _ = D.add_rmsnorm(x, w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = late_use((64, 4096), BF16)
    y, _ = sk.sgemm_bf16_add_rmsnorm(xd, wd, stream=s)
    torch.cuda.synchronize()
    assert bool((kept == 2).all())
    D.check(y, want, D.norm_y_bound(want, 4096), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [True, False])
def test_a_call_on_the_default_stream_while_another_is_current(handle):
    """By its handle, which is 0, and by torch's object."""
    x, w = torch.randn((64, 4096), device="cuda").to(BF16), torch.ones(4096, device="cuda").to(BF16)
    want, _ = sk.sgemm_bf16_add_rmsnorm(x, w)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        y, _ = sk.sgemm_bf16_add_rmsnorm(x, w, stream=0 if handle else default)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.gpu
def test_an_output_dropped_early_is_not_handed_out_before_the_current_stream_has_read_it():
    x, w = torch.randn((64, 4096), device="cuda").to(BF16), torch.ones(4096, device="cuda").to(BF16)
    minus = -x
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    want, _ = sk.sgemm_bf16_add_rmsnorm(x, w)
    torch.cuda.synchronize()
    y, _ = sk.sgemm_bf16_add_rmsnorm(x, w, stream=s)
    here.wait_stream(s)
    torch.cuda._sleep(200_000_000)
    kept = y + 0
    del y  # its block may not serve the next call on s before the sum above is done
    sk.sgemm_bf16_add_rmsnorm(minus, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
