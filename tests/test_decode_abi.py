"""The operators of sgemm_decode.h on a CPU-only machine: the library exports them, the binding's
argument structures are the header's, and bad arguments are refused on the host.  No kernel is
launched: every call returns before the library touches a CUDA device.
"""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import build as skbuild
from bf16_skinny_gemm_gb300 import decode

HEADER = os.path.join(skbuild.INCLUDE, "sgemm_decode.h")
NULL = 0
A = 0x10000  # pointers that are never dereferenced: far apart, 64 KiB aligned
OK_OR_DEVICE = (sk.SGEMM_OK, sk.SGEMM_ERR_UNSUPPORTED_DEVICE, sk.SGEMM_ERR_CUDA)


@pytest.fixture(scope="module")
def lib():
    skbuild.build()
    return sk.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sgemm_[a-z0-9_]+)\s*\(", text))
    assert names == {"sgemm_bf16_add_rmsnorm", "sgemm_bf16_latent_append", "sgemm_bf16_latent_attention",
                     "sgemm_latent_attention_workspace"}
    assert not [n for n in names if not hasattr(lib, n)]
    for n in sk.decode.__all__:
        assert hasattr(sk, n)


def test_argument_structures_are_the_headers(tmp_path):
    """Size and offset of every field, as a C compiler lays them out."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    formats = {"sgemm_add_rmsnorm_t": decode._NORM, "sgemm_latent_append_t": decode._APPEND,
               "sgemm_latent_attention_t": decode._ATTN}
    body = []
    for name in formats:
        fields = re.search(r"typedef struct \{([^}]*)\} " + name, text).group(1)
        names = [f.strip().split()[-1].lstrip("*") for d in fields.split(";") if d.strip()
                 for f in re.sub(r"^(.*?)(\w+\s*(,|$))", r"\2", d.strip()).split(",")]
        body.append(f'printf("%zu", sizeof({name}));')
        body += [f'printf(" %zu:%zu", offsetof({name}, {n}), sizeof((({name} *)0)->{n}));' for n in names]
        body.append('printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sgemm_decode.h"\nint main(void) {'
                   + "\n".join(body) + "return 0;}\n")
    subprocess.run(["gcc", "-I", skbuild.INCLUDE, str(src), "-o", str(tmp_path / "layout")], check=True)
    lines = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.splitlines()
    for (name, fmt), line in zip(formats.items(), lines):
        size, *fields = line.split()
        assert int(size) == fmt.size, name
        codes = [c for n, c in re.findall(r"(\d*)([a-zA-Z])", fmt.format) for _ in range(int(n or 1))]
        assert len(codes) == len(fields), name
        at = 0
        for code, field in zip(codes, fields):
            width = {"Q": 8, "q": 8, "i": 4, "f": 4, "I": 4}[code]
            assert field == f"{at}:{width}", (name, field)
            at += width


# ------------------------------------------------------------------------------------- RMS norm
def norm(lib, **kw):
    a = dict(x=A, residual=2 * A, weight=3 * A, residual_out=4 * A, y=5 * A, scales=NULL, ldx=64, ldr=64, ldro=64,
             ldy=64, lds=0, T=2, D=64, form=0, eps=1e-6, flags=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_add_rmsnorm")(decode._NORM.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), 1), (dict(weight=NULL), 1), (dict(y=NULL), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(D=0), 1),
    (dict(form=3), 1), (dict(form=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(ldx=63), 1), (dict(ldr=63), 1), (dict(ldro=63), 1), (dict(ldy=63), 1), (dict(flags=4), 1), (dict(flags=8), 1),
    (dict(form=1), 1),                                   # 8 bits without scales
    (dict(form=2, scales=6 * A, lds=0), 1),              # fewer than its groups
    (dict(x=A + 1), 3), (dict(residual=2 * A + 1), 3), (dict(weight=3 * A + 1), 3), (dict(y=5 * A + 1), 3),
    (dict(form=1, scales=6 * A + 2, lds=1), 3),
    (dict(y=A + 64), 1),                                 # inside x, not x itself
    (dict(y=4 * A), 1),                                  # the residual's copy
    (dict(y=3 * A), 1),                                  # the weight
    (dict(form=1, scales=6 * A, lds=1, y=A), 1),         # 8 bits over x
    (dict(residual_out=A, ldro=128), 1),                 # x itself with another stride
    (dict(form=1, scales=A, lds=1), 1),                  # scales over x
])
def test_norm_refusals(lib, change, status):
    assert norm(lib, **change) == status


def test_norm_accepts(lib):
    assert norm(lib, T=0) == sk.SGEMM_OK
    for change in (dict(), dict(residual=NULL, residual_out=NULL), dict(residual_out=2 * A), dict(residual_out=A),
                   dict(y=A), dict(y=A, residual_out=2 * A), dict(form=2, scales=6 * A, lds=1, y=5 * A + 1),
                   dict(ldx=128, ldy=128, y=A + 128)):  # two column ranges of one buffer
        assert norm(lib, **change) in OK_OR_DEVICE, change


# ---------------------------------------------------------------------------------------- append
def append(lib, **kw):
    a = dict(kv=A, weight=2 * A, cos_sin=3 * A, positions=4 * A, slots=5 * A, cache=16 * A, q=6 * A, q_out=8 * A,
             ldkv=576, ldcs=64, row_stride=576, page_stride=576 * 16, q_token=64 * 8, q_head=64, qo_token=64 * 8, qo_head=64,
             T=3, max_position=100, pages=4, page_size=16, R=512, E=64, H=8, interleaved=1, eps=1e-6, flags=0, reserved=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_latent_append")(decode._APPEND.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(kv=NULL), 1), (dict(cos_sin=NULL), 1), (dict(positions=NULL), 1), (dict(slots=NULL), 1), (dict(cache=NULL), 1),
    (dict(q=NULL), 1), (dict(q_out=NULL), 1), (dict(T=-1), 1), (dict(R=0), 1), (dict(R=8193), 1), (dict(E=0), 1),
    (dict(E=63), 1), (dict(E=514), 1), (dict(H=-1), 1), (dict(page_size=0), 1), (dict(pages=-1), 1),
    (dict(max_position=0), 1), (dict(interleaved=2), 1), (dict(eps=-1.0), 1), (dict(flags=4), 1),
    (dict(ldkv=575), 1), (dict(ldcs=63), 1), (dict(row_stride=575), 1), (dict(page_stride=576 * 16 - 1), 1),
    (dict(qo_head=63), 1), (dict(qo_token=64 * 7), 1), (dict(q_token=-1), 1),
    (dict(kv=A + 1), 3), (dict(cos_sin=3 * A + 2), 3), (dict(positions=4 * A + 4), 3), (dict(slots=5 * A + 4), 3),
    (dict(cache=16 * A + 1), 3), (dict(q=6 * A + 1), 3),
    (dict(cache=A), 1), (dict(q_out=A), 1), (dict(q_out=6 * A + 64), 1), (dict(q_out=16 * A), 1), (dict(q=16 * A), 1),
])
def test_append_refusals(lib, change, status):
    assert append(lib, **change) == status


def test_append_accepts(lib):
    assert append(lib, T=0) == sk.SGEMM_OK
    wide = dict(q_head=128, q_token=1024, qo_head=128, qo_token=1024)
    for change in (dict(), dict(weight=NULL), dict(H=0, q=NULL, q_out=NULL), dict(q_out=6 * A), dict(interleaved=0),
                   dict(q_out=6 * A + 128, **wide),  # the other half of each head's elements
                   dict(qo_head=64 * 3, qo_token=64)):  # heads outermost
        assert append(lib, **change) in OK_OR_DEVICE, change


# ------------------------------------------------------------------------------------- attention
def attention(lib, **kw):
    a = dict(q=A, cache=16 * A, block_table=2 * A, seq_lens=3 * A, cu_q=4 * A, out=8 * A, lse=5 * A, workspace=32 * A,
             q_token=576 * 8, q_head=576, row_stride=576, page_stride=576 * 64, ldt=10, out_token=512 * 8, out_head=512,
             lse_token=8, pages=40, workspace_bytes=64 << 20, total_q=3, page_size=64, table_width=10, B=3, H=8, R=512, E=64,
             max_q=2, scale=0.1, flags=0, reserved=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_latent_attention")(decode._ATTN.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=NULL), 1), (dict(cache=NULL), 1), (dict(block_table=NULL), 1), (dict(seq_lens=NULL), 1), (dict(out=NULL), 1),
    (dict(B=-1), 1), (dict(H=0), 1), (dict(H=1025), 1), (dict(max_q=0), 1), (dict(pages=0), 1), (dict(table_width=-1), 1),
    (dict(page_size=0), 1), (dict(total_q=-1), 1), (dict(flags=8), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(workspace_bytes=-1), 1),
    (dict(R=500), 2), (dict(R=640), 2), (dict(R=64), 2), (dict(E=12), 2), (dict(E=72), 2), (dict(page_size=4), 2),
    (dict(page_size=48), 2), (dict(page_size=96), 2), (dict(pages=1 << 30), 2), (dict(max_q=1 << 28), 2),
    (dict(table_width=1 << 27), 2),
    (dict(cu_q=NULL), 1),                      # 3 tokens are not 3 x 2
    (dict(ldt=9), 1), (dict(row_stride=568), 1), (dict(page_stride=576 * 64 - 8), 1), (dict(q_token=-8), 1),
    (dict(out_head=504), 1), (dict(out_token=512 * 7), 1), (dict(lse_token=7), 1),
    (dict(q=A + 8), 3), (dict(q_head=580), 3), (dict(cache=16 * A + 8), 3), (dict(row_stride=580, page_stride=580 * 64), 3),
    (dict(out=8 * A + 2), 3), (dict(out_head=513, out_token=513 * 8), 3), (dict(lse=5 * A + 2), 3),
    (dict(block_table=2 * A + 2), 3), (dict(workspace=32 * A + 8), 3),
])
def test_attention_refusals(lib, change, status):
    assert attention(lib, **change) == status


def test_attention_accepts(lib):
    assert attention(lib, B=0) == sk.SGEMM_OK and attention(lib, total_q=0) == sk.SGEMM_OK
    assert attention(lib, lse=NULL) in OK_OR_DEVICE
    assert attention(lib, cu_q=NULL, total_q=6) in OK_OR_DEVICE
    assert attention(lib, out_head=512 * 3, out_token=512) in OK_OR_DEVICE  # heads outermost


def test_workspace_query_checks_its_sizes():
    with pytest.raises(sk.SgemmError) as e:
        sk.sgemm_latent_attention_workspace(1, 8, 500, 64, 64, 4)
    assert e.value.status == sk.SGEMM_ERR_UNSUPPORTED_SHAPE
    assert sk.sgemm_latent_attention_workspace(0, 8, 512, 64, 64, 4) == 0


# ------------------------------------------------------------------------------ the binding itself
def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_what_is_no_cuda_tensor():
    with pytest.raises(TypeError, match="x must be a 2-D"):
        sk.sgemm_bf16_add_rmsnorm(None, bf(4))
    with pytest.raises(TypeError, match="x must be a 2-D"):
        sk.sgemm_bf16_add_rmsnorm(torch.zeros(2, 4), bf(4))
    with pytest.raises(TypeError, match="CUDA"):
        sk.sgemm_bf16_add_rmsnorm(bf(2, 4), bf(4))
    with pytest.raises(ValueError, match="group"):
        sk.sgemm_bf16_add_rmsnorm_e4m3(bf(2, 4), bf(4), group=64)
    with pytest.raises(TypeError, match="kv"):
        sk.sgemm_bf16_latent_append(bf(2, 3, 4), None, None, None, None)
    with pytest.raises(ValueError, match="cache rows"):
        sk.sgemm_bf16_latent_append(bf(2, 96), bf(2, 4, 64), None, None, torch.zeros(5, 32))
    with pytest.raises(ValueError, match="wider"):
        sk.sgemm_bf16_latent_append(bf(2, 32), bf(2, 4, 32), None, None, torch.zeros(5, 32))
    with pytest.raises(TypeError, match="q must be a 3-D"):
        sk.sgemm_bf16_latent_attention(bf(2, 4), None, None, None, 128, 1.0)
    with pytest.raises(ValueError, match="cache rows"):
        sk.sgemm_bf16_latent_attention(bf(2, 4, 192), bf(2, 16, 128), torch.zeros((2, 3), dtype=torch.int32), None, 128, 1.0)
