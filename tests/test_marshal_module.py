"""The binding's native module is built for one Python and torch, is not loaded into another, and
the binding does without it."""
from __future__ import annotations

import os
import warnings

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import build as skbuild
from bf16_skinny_gemm_gb300 import decode


@pytest.fixture(scope="module", autouse=True)
def built():
    skbuild.build()


@pytest.mark.parametrize("what", ["version", "git", "abi", "python"])
def test_another_torch_or_python_is_another_file(monkeypatch, what):
    here = skbuild.build_marshal()
    assert os.path.exists(here)
    if what == "version":
        monkeypatch.setattr(torch, "__version__", "99.1")
    elif what == "git":
        monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        real = skbuild.sysconfig.get_config_var
        monkeypatch.setattr(skbuild.sysconfig, "get_config_var", lambda n: "cpython-99" if n == "SOABI" else real(n))
    ran = []

    class Done:
        returncode = 0

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(skbuild.subprocess, "run", run)
    path = skbuild.build_marshal()
    try:
        assert path != here and len(ran) == 1  # compiled again, beside the other
    finally:
        os.remove(path)


@pytest.mark.parametrize("there", ["nothing", "no library"])
def test_without_the_module_every_call_goes_the_long_way(monkeypatch, tmp_path, there):
    path = tmp_path / "_marshal.so"
    if there == "no library":
        path.write_bytes(b"not a library")
    monkeypatch.setattr(decode, "marshal_path", lambda: str(path))
    monkeypatch.setattr(decode, "_short", decode._Unbound())
    cpu = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="build the module"), pytest.raises(TypeError, match="x must be on a CUDA device"):
        sk.sgemm_bf16_add_rmsnorm(cpu, cpu[0])
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        with pytest.raises(TypeError, match="kv must be a 2-D"):
            sk.sgemm_bf16_latent_append(cpu[0], cpu, cpu, cpu, cpu)
        with pytest.raises(TypeError, match="q must be a 3-D"):
            sk.sgemm_bf16_latent_attention(cpu, cpu, cpu, cpu, 512, 1.0)


@pytest.mark.gpu
def test_a_call_without_the_module(monkeypatch, tmp_path):
    x = torch.randn((3, 256), device="cuda").to(torch.bfloat16)
    w = torch.ones(256, device="cuda").to(torch.bfloat16)
    want, y = torch.empty_like(x), torch.empty_like(x)
    sk.sgemm_bf16_add_rmsnorm(x, w, y=want)
    monkeypatch.setattr(decode, "marshal_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(decode, "_short", decode._Unbound())
    with pytest.warns(RuntimeWarning):
        sk.sgemm_bf16_add_rmsnorm(x, w, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
