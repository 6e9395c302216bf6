"""GPU: while a call of the binding's short way is in the library, other threads of the program run.

A launch waits where the stream's queue is full; where the work in front of it waits in turn for
another Python thread (a host callback, a collective whose other rank is a thread), a call that
kept the interpreter's lock would wait for ever.  Here the library's functions are replaced by one
that waits, for three seconds at most, for another thread to set a flag.
"""
from __future__ import annotations

import ctypes
import subprocess
import threading

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import decode

pytestmark = pytest.mark.gpu
SOURCE = """
#include <unistd.h>
volatile int entered = 0, flag = 0;
int waits(const void *args, void *stream) {
    entered = 1;
    for (int i = 0; i < 3000; ++i) {
        if (flag) return 0;
        usleep(1000);
    }
    return 1;
}
"""


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def norm():
    x = bf(2, 64)
    sk.sgemm_bf16_add_rmsnorm(x, bf(64), y=bf(2, 64))


def append():
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    sk.sgemm_bf16_latent_append(bf(1, 96), bf(2, 8, 96), at, at, torch.zeros((4, 32), device="cuda"))


def attention():
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    sk.sgemm_bf16_latent_attention(bf(1, 8, 192), bf(2, 8, 192), one.view(1, 1), one, 128, 0.1, out=bf(1, 8, 128),
                                   workspace=bf(64))


@pytest.mark.parametrize("operator", [norm, append, attention])
def test_other_threads_run_during_a_call(tmp_path, monkeypatch, operator):
    decode._short.add_rmsnorm(None, None, None, 0.0, 0, None, None, None, 0, None)  # loads the module
    source, path = tmp_path / "waits.c", tmp_path / "waits.so"
    source.write_text(SOURCE)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(source), "-o", str(path)], check=True)
    stub, lib = ctypes.CDLL(str(path)), sk.load()
    entered, flag = ctypes.c_int.in_dll(stub, "entered"), ctypes.c_int.in_dll(stub, "flag")
    over = threading.Event()

    def other():
        while not entered.value and not over.wait(0.001):
            pass
        flag.value = 1

    def bind(*functions):
        decode._short.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in functions))

    # the long way is not to be taken
    monkeypatch.setattr(decode, "_call", lambda *a: pytest.fail("the call was left to the long way"))
    thread = threading.Thread(target=other)
    bind(stub.waits, stub.waits, stub.waits)
    try:
        thread.start()
        operator()  # raises where the flag was not set in time
    finally:
        over.set()
        thread.join()
        bind(lib.sgemm_bf16_add_rmsnorm, lib.sgemm_bf16_latent_append, lib.sgemm_bf16_latent_attention)
