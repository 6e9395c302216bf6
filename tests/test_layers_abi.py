"""The operators of sgemm_layers.h on a CPU-only machine: the library exports them, the binding's
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
from bf16_skinny_gemm_gb300 import decode, layers

HEADER = os.path.join(skbuild.INCLUDE, "sgemm_layers.h")
NULL = 0
A = 0x100000  # pointers that are never dereferenced: far apart, 1 MiB aligned
OK_OR_DEVICE = (sk.SGEMM_OK, sk.SGEMM_ERR_UNSUPPORTED_DEVICE, sk.SGEMM_ERR_CUDA)
# made-up pointers that pass every check would be launched on where there is a GPU
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU: the pointers are made up")


@pytest.fixture(scope="module")
def lib():
    skbuild.build()
    return sk.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sgemm_[a-z0-9_]+)\s*\(", text))
    assert names == {"sgemm_bf16_moe_route", "sgemm_bf16_moe_experts", "sgemm_moe_experts_workspace",
                     "sgemm_bf16_latent_tree_attention", "sgemm_latent_tree_attention_workspace", "sgemm_bf16_linear_step",
                     "sgemm_bf16_linear_attention", "sgemm_linear_attention_workspace"}
    assert not [n for n in names if not hasattr(lib, n)]
    for n in layers.__all__:
        assert hasattr(sk, n) and n in sk.__all__


def test_argument_structures_are_the_headers(tmp_path):
    """Size and offset of every field, as a C compiler lays them out."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    formats = {"sgemm_moe_route_t": layers._ROUTE, "sgemm_moe_experts_t": layers._EXPERTS, "sgemm_linear_step_t": layers._STEP,
               "sgemm_linear_attention_t": layers._LINEAR}
    body = []
    for name in formats:
        fields = re.search(r"typedef struct \{([^}]*)\} " + name, text).group(1)
        names = []
        for d in fields.split(";"):
            if d.strip():
                first, *more = d.strip().split(",")
                names += [first.split()[-1].lstrip("*"), *[m.strip().lstrip("*") for m in more]]
        body.append(f'printf("%zu", sizeof({name}));')
        body += [f'printf(" %zu:%zu", offsetof({name}, {n}), sizeof((({name} *)0)->{n}));' for n in names]
        body.append('printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sgemm_layers.h"\nint main(void) {'
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


# ---------------------------------------------------------------------------------------- router
def route(lib, **kw):
    a = dict(x=A, w=2 * A, bias=3 * A, ids=4 * A, weights=5 * A, ldx=64, ldw=64, ldi=4, ldwt=4, T=3, D=64, E=16, k=4, scoring=0,
             renormalize=1, scale=1.0, flags=0, reserved=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_moe_route")(layers._ROUTE.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), 1), (dict(w=NULL), 1), (dict(ids=NULL), 1), (dict(weights=NULL), 1), (dict(T=-1), 1), (dict(T=(1 << 20) + 1), 1),
    (dict(E=0), 1), (dict(E=1025), 1), (dict(k=0), 1), (dict(k=17, E=32, ldi=17, ldwt=17), 1), (dict(E=3), 1), (dict(D=0), 1),
    (dict(scoring=2), 1), (dict(scoring=-1), 1), (dict(renormalize=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(flags=4), 1), (dict(flags=8), 1), (dict(ldx=56), 1), (dict(ldw=56), 1), (dict(ldi=3), 1), (dict(ldwt=3), 1),
    (dict(D=60), 2), (dict(x=A + 8), 3), (dict(w=2 * A + 2), 3), (dict(ldx=68), 3), (dict(ldw=68), 3), (dict(bias=3 * A + 2), 3),
    (dict(ids=4 * A + 2), 3), (dict(weights=5 * A + 1), 3),
    (dict(ids=A + 128), 1), (dict(weights=2 * A + 64), 1), (dict(ids=3 * A), 1), (dict(weights=4 * A), 1), (dict(weights=4 * A + 16), 1),
])
def test_route_refusals(lib, change, status):
    assert route(lib, **change) == status


def test_route_without_tokens(lib):
    assert route(lib, T=0, x=NULL, ids=NULL, weights=NULL) == sk.SGEMM_OK


@no_gpu
def test_route_accepts(lib):
    for change in (dict(), dict(bias=NULL), dict(E=4), dict(ldi=9, ldwt=9, weights=4 * A + 16), dict(ldx=128, ldw=72)):
        assert route(lib, **change) in OK_OR_DEVICE, change


# ---------------------------------------------------------------------------------------- experts
def experts(lib, **kw):
    a = dict(x=A, w_gate_up=2 * A, w_down=4 * A, ids=6 * A, weights=7 * A, y=8 * A, workspace=16 * A, ldx=64, gu_expert=2 * 40 * 64,
             gu_row=64, dn_expert=64 * 40, dn_row=40, ldi=2, ldwt=2, ldy=64, workspace_bytes=1 << 20, T=3, D=64, F=40, E=5, k=2, flags=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_moe_experts")(layers._EXPERTS.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), 1), (dict(w_gate_up=NULL), 1), (dict(w_down=NULL), 1), (dict(ids=NULL), 1), (dict(weights=NULL), 1), (dict(y=NULL), 1),
    (dict(workspace=NULL), 5), (dict(workspace_bytes=5 * 3 * 40 * 2 - 1), 5), (dict(workspace_bytes=-1), 1),
    (dict(T=-1), 1), (dict(T=129), 2), (dict(D=0), 1), (dict(F=0), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(k=0), 1), (dict(k=33), 1),
    (dict(D=60), 2), (dict(F=36), 2), (dict(flags=8), 1), (dict(ldx=56), 1), (dict(gu_row=56), 1), (dict(dn_row=32), 1), (dict(ldi=1), 1),
    (dict(ldwt=1), 1), (dict(ldy=63), 1), (dict(gu_expert=79 * 64), 1), (dict(dn_expert=63 * 40), 1),
    (dict(E=1, gu_expert=-8), 1), (dict(gu_row=1 << 39, gu_expert=1 << 50), 2),
    (dict(x=A + 8), 3), (dict(w_gate_up=2 * A + 8), 3), (dict(w_down=4 * A + 2), 3), (dict(ldx=68), 3), (dict(gu_row=68, gu_expert=80 * 68), 3),
    (dict(gu_expert=2 * 40 * 64 + 4), 3), (dict(dn_row=44, dn_expert=64 * 44), 3), (dict(y=8 * A + 1), 3), (dict(ids=6 * A + 2), 3),
    (dict(weights=7 * A + 2), 3), (dict(workspace=16 * A + 64), 3),
    (dict(y=A), 1), (dict(y=2 * A + 128), 1), (dict(y=4 * A), 1), (dict(y=6 * A), 1), (dict(y=7 * A), 1), (dict(workspace=8 * A), 1),
    (dict(workspace=A), 1), (dict(workspace=2 * A), 1), (dict(workspace=4 * A), 1), (dict(workspace=6 * A), 1), (dict(workspace=7 * A), 1),
])
def test_experts_refusals(lib, change, status):
    assert experts(lib, **change) == status


def test_experts_without_tokens(lib):
    assert experts(lib, T=0, workspace=NULL) == sk.SGEMM_OK


@no_gpu
def test_experts_accept(lib):
    for change in (dict(), dict(E=1, gu_expert=0, dn_expert=0), dict(ldx=128, ldy=128, y=A + 128), dict(flags=4), dict(ldi=5, ldwt=5, weights=6 * A + 8)):
        assert experts(lib, **change) in OK_OR_DEVICE, change


def test_experts_workspace():
    assert sk.sgemm_moe_experts_workspace(3, 5, 2, 64, 40) == 5 * 3 * 40 * 2
    assert sk.sgemm_moe_experts_workspace(1, 100, 8, 64, 40) == 8 * 40 * 2  # no more experts than entries
    assert sk.sgemm_moe_experts_workspace(0, 5, 2, 64, 40) == 0
    with pytest.raises(sk.SgemmError) as e:
        sk.sgemm_moe_experts_workspace(129, 5, 2, 64, 40)
    assert e.value.status == sk.SGEMM_ERR_UNSUPPORTED_SHAPE


# ------------------------------------------------------------------------------------------- tree
def tree(lib, masks=6 * A, ld=1, words=1, **kw):
    a = dict(q=A, cache=16 * A, block_table=2 * A, seq_lens=3 * A, cu_q=4 * A, out=8 * A, lse=5 * A, workspace=32 * A,
             q_token=576 * 8, q_head=576, row_stride=576, page_stride=576 * 64, ldt=10, out_token=512 * 8, out_head=512,
             lse_token=8, pages=40, workspace_bytes=64 << 20, total_q=3, page_size=64, table_width=10, B=3, H=8, R=512, E=64,
             max_q=2, scale=0.1, flags=0, reserved=0)
    a.update(kw)
    import ctypes
    f = decode._fn("sgemm_bf16_latent_tree_attention")
    return f(decode._ATTN.pack(*a.values()), masks, ctypes.c_longlong(ld), ctypes.c_int(words), ctypes.c_void_p(None))


@pytest.mark.parametrize("change,status", [
    (dict(masks=NULL), 1), (dict(words=0), 1), (dict(ld=0), 1), (dict(words=2), 1), (dict(max_q=65), 1), (dict(ld=1 << 28), 1),
    (dict(masks=6 * A + 4), 3), (dict(masks=8 * A), 1), (dict(masks=5 * A), 1), (dict(q=NULL), 1), (dict(R=500), 2), (dict(flags=8), 1),
    (dict(out=A), 1), (dict(table_width=1 << 22, ldt=1 << 22, total_q=1 << 12, B=1 << 12, max_q=1), 2),
])
def test_tree_refusals(lib, change, status):
    assert tree(lib, **change) == status


def test_tree_without_tokens(lib):
    assert tree(lib, total_q=0, masks=NULL) == sk.SGEMM_OK and tree(lib, B=0) == sk.SGEMM_OK


@no_gpu
def test_tree_accepts(lib):
    for change in (dict(), dict(lse=NULL), dict(words=2, ld=3, max_q=100), dict(cu_q=NULL, total_q=6)):
        assert tree(lib, **change) in OK_OR_DEVICE, change


def test_tree_workspace_checks_its_sizes():
    with pytest.raises(sk.SgemmError):
        sk.sgemm_latent_tree_attention_workspace(1, 8, 500, 64, 64, 4)
    assert sk.sgemm_latent_tree_attention_workspace(0, 8, 512, 64, 64, 4) == 0


# ---------------------------------------------------------------------------------- linear attention
STEP = dict(q=A, k=2 * A, v=3 * A, g=4 * A, state=64 * A, slots=5 * A, out=6 * A, q_token=256, q_head=64, k_token=256, k_head=64,
            v_token=512, v_head=64, g_token=8, g_head=1, s_slot=8 * 4096, s_head=4096, o_token=512, o_head=64, B=3, pool=5, Hk=4, Hv=8,
            Dk=64, Dv=64, scale=1.0, flags=0)


def step(lib, **kw):
    return decode._fn("sgemm_bf16_linear_step")(layers._STEP.pack(*(STEP | kw).values()), None)


BOTH = [
    (dict(q=NULL), 1), (dict(k=NULL), 1), (dict(v=NULL), 1), (dict(g=NULL), 1), (dict(state=NULL), 1), (dict(slots=NULL), 1),
    (dict(out=NULL), 1), (dict(B=-1), 1), (dict(pool=-1), 1), (dict(pool=1 << 31), 1), (dict(Hk=0), 1), (dict(Hv=6), 1), (dict(Hv=2), 1),
    (dict(Hk=4, Hv=1028), 1), (dict(Dk=32), 2), (dict(Dv=96), 2), (dict(scale=float("nan")), 1), (dict(flags=16), 1),
    (dict(q_token=-8), 1), (dict(g_head=-1), 1), (dict(s_head=4092), 1), (dict(s_slot=7 * 4096), 1), (dict(o_head=63), 1),
    (dict(o_token=448), 1), (dict(v_token=1 << 29), 1),
    (dict(q=A + 8), 3), (dict(k=2 * A + 2), 3), (dict(v=3 * A + 8), 3), (dict(q_token=260), 3), (dict(v_head=68), 3), (dict(g=4 * A + 2), 3),
    (dict(state=64 * A + 8), 3), (dict(s_head=4098, s_slot=8 * 4098), 3), (dict(out=6 * A + 2), 3), (dict(o_head=65, o_token=520), 3),
    (dict(slots=5 * A + 4), 3),
    (dict(out=A), 1), (dict(out=2 * A + 64), 1), (dict(out=3 * A), 1), (dict(out=4 * A), 1), (dict(out=5 * A), 1), (dict(state=A), 1),
    (dict(state=3 * A), 1), (dict(state=4 * A), 1), (dict(state=6 * A), 1), (dict(slots=64 * A), 1),
]


@pytest.mark.parametrize("change,status", [*BOTH, (dict(flags=4), 1)])
def test_step_refusals(lib, change, status):
    assert step(lib, **change) == status


@no_gpu
def test_step_accepts(lib):
    assert step(lib, B=0) == sk.SGEMM_OK
    for change in (dict(), dict(g_token=0, g_head=0), dict(q_token=0), dict(pool=0, state=NULL), dict(Hk=1, q_head=0, k_head=0),
                   dict(o_token=64, o_head=64 * 3), dict(v=A + 512, q_token=2048, v_token=2048, out=A + 2048, o_token=2048)):
        assert step(lib, **change) in OK_OR_DEVICE, change


PROMPT = dict(q=A, k=2 * A, v=3 * A, g=4 * A, state=64 * A, slots=5 * A, cu=7 * A, fresh=8 * A, out=6 * A, workspace=512 * A,
              **{n: STEP[n] for n in list(STEP)[7:19]}, N=100, B=3, pool=5, workspace_bytes=64 << 20,
              **{n: STEP[n] for n in list(STEP)[21:]})


def prompt(lib, **kw):
    return decode._fn("sgemm_bf16_linear_attention")(layers._LINEAR.pack(*(PROMPT | kw).values()), None)


@pytest.mark.parametrize("change,status", [
    *[c for c in BOTH if "B" not in c[0]], (dict(cu=NULL), 1), (dict(N=-1), 1), (dict(B=-1), 1), (dict(N=1 << 28), 2), (dict(B=1 << 25), 2),
    (dict(workspace_bytes=-1), 1), (dict(cu=7 * A + 2), 3), (dict(fresh=8 * A + 2), 3), (dict(workspace=512 * A + 8), 3),
    (dict(q_token=0), 1), (dict(k_head=0), 1), (dict(v_token=0), 1), (dict(cu=6 * A), 1), (dict(fresh=64 * A), 1),
])
def test_prompt_refusals(lib, change, status):
    assert prompt(lib, **change) == status


@no_gpu
def test_prompt_accepts(lib):
    assert prompt(lib, B=0) == sk.SGEMM_OK
    for change in (dict(), dict(fresh=NULL), dict(N=0, q=NULL, k=NULL, v=NULL, g=NULL, out=NULL), dict(g_token=0), dict(flags=4)):
        assert prompt(lib, **change) in OK_OR_DEVICE, change


def test_prompt_workspace_checks_its_sizes():
    with pytest.raises(sk.SgemmError):
        sk.sgemm_linear_attention_workspace(100, 1, 8, 32, 64)
    assert sk.sgemm_linear_attention_workspace(100, 0, 8, 64, 64) == 0


# ------------------------------------------------------------------------------ the binding itself
def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_what_is_no_cuda_tensor():
    i32 = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(TypeError, match="x must be a 2-D"):
        sk.sgemm_bf16_moe_route(None, bf(4, 8), 2)
    with pytest.raises(ValueError, match="scoring"):
        sk.sgemm_bf16_moe_route(bf(2, 8), bf(4, 8), 2, scoring="top")
    with pytest.raises(TypeError, match="CUDA"):
        sk.sgemm_bf16_moe_route(bf(2, 8), bf(4, 8), 2)
    with pytest.raises(ValueError, match="even number of rows"):
        sk.sgemm_bf16_moe_experts(bf(2, 8), bf(4, 7, 8), bf(4, 8, 3), i32, torch.zeros(2, 2))
    with pytest.raises(TypeError, match="w_gate_up must be a 3-D"):
        sk.sgemm_bf16_moe_experts(bf(2, 8), bf(8, 8), bf(4, 8, 3), i32, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="cache rows"):
        sk.sgemm_bf16_latent_tree_attention(bf(2, 4, 192), bf(2, 16, 128), i32, None, 128, 1.0, torch.zeros((2, 1), dtype=torch.int64))
    with pytest.raises(TypeError, match="tree must be a 2-D"):
        sk.sgemm_bf16_latent_tree_attention(bf(2, 4, 192), bf(2, 16, 192), i32, None, 128, 1.0, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="state must be a 4-D"):
        sk.sgemm_bf16_linear_step(bf(2, 4, 64), bf(2, 4, 64), bf(2, 4, 64), torch.zeros(2, 4), torch.zeros(4, 64, 64), None)
    with pytest.raises(TypeError, match="CUDA"):
        sk.sgemm_bf16_linear_attention(bf(2, 4, 64), bf(2, 4, 64), bf(2, 4, 64), torch.zeros(2, 4), torch.zeros(3, 4, 64, 64), None, None)
