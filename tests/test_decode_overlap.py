"""The latent attention refuses outputs and scratch that lie over what it reads, or over each other,
and takes those that only lie between it."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import build as skbuild
from bf16_skinny_gemm_gb300 import decode

M = 1 << 24  # pointers that are never dereferenced, 16 MiB apart
T, H, R, E, PAGE, PAGES, B, WIDTH = 6, 8, 512, 64, 64, 40, 3, 10
W = R + E


@pytest.fixture(scope="module", autouse=True)
def built():
    skbuild.build()


def attention(**kw):
    a = dict(q=M, cache=2 * M, block_table=3 * M, seq_lens=4 * M, cu_q=5 * M, out=6 * M, lse=7 * M, workspace=8 * M,
             q_token=W * H, q_head=W, row_stride=W, page_stride=W * PAGE, ldt=WIDTH, out_token=R * H, out_head=R, lse_token=H,
             pages=PAGES, workspace_bytes=64 << 20, total_q=T, page_size=PAGE, table_width=WIDTH, B=B, H=H, R=R, E=E, max_q=2,
             scale=0.1, flags=0, reserved=0)
    a.update(kw)
    return decode._fn("sgemm_bf16_latent_attention")(decode._ATTN.pack(*a.values()), None)


BOTH = H * (W + R)  # a token's queries, then its results
WIDE = dict(q_token=H * (W + R), q_head=W + R, out_token=H * (W + R), out_head=W + R)


@pytest.mark.parametrize("change", [
    dict(out=M), dict(out=M + 2 * W * H * (T - 1)),                       # the queries, the last token's
    dict(out=M - 2 * R * H * T + 4),                                      # ends inside them
    dict(out=M + 2 * R, **WIDE), dict(out=M + 2 * (W + R) - 4, **WIDE),   # inside a row of a common buffer, and into the next
    dict(out=M + 2 * W, q_head=W + R, q_token=BOTH, out_head=W + R - 2, out_token=BOTH),
    dict(out=2 * M), dict(out=2 * M + 2 * W * PAGE * PAGES - 4),          # the cache's first and last bytes
    dict(out=2 * M + 2 * W * PAGE - 4, page_stride=2 * W * PAGE + 8 * R), # a page's last bytes, and free ones
    dict(out=3 * M), dict(out=3 * M + 4 * (B - 1) * WIDTH + 36), dict(out=4 * M + 8), dict(out=5 * M + 12),
    dict(lse=M), dict(lse=2 * M + 64), dict(lse=3 * M + 4), dict(lse=4 * M), dict(lse=5 * M + 12),
    dict(lse=6 * M), dict(lse=6 * M + 2 * R * H * T - 4),                 # the results
])
def test_outputs_over_inputs_or_each_other_are_refused(change):
    assert attention(**change) == sk.SGEMM_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="these would be launched on pointers that are made up")
@pytest.mark.parametrize("change", [
    dict(), dict(lse=0), dict(out=M + 2 * W * H * T), dict(out=M - 2 * R * H * T), dict(out=2 * M + 2 * W * PAGE * PAGES),
    dict(out=M + 2 * W, **WIDE),                                          # columns of a common buffer
    dict(q=M + 2 * R, out=M, **WIDE),
    dict(out=M + 2 * W * H, q_token=BOTH, out_token=BOTH),                # a token's queries, then its results
    dict(out=M + 2 * W * T, q_head=(W + R) * T, q_token=W, out_head=(W + R) * T, out_token=R),  # heads outermost
    dict(out=2 * M + 2 * W * PAGE, out_token=R, out_head=R * T, page_stride=2 * W * PAGE + 2 * R * T * H),  # between pages
    dict(lse=M + 2 * W * H, q_token=W * H + 64, lse_token=(W * H + 64) // 2),
    dict(lse=6 * M + 2 * R * H * T), dict(out=3 * M + 4 * WIDTH * B), dict(out=5 * M + 16), dict(lse=4 * M + 12),
])
def test_outputs_beside_and_between_are_taken(change):
    assert attention(**change) in (sk.SGEMM_ERR_UNSUPPORTED_DEVICE, sk.SGEMM_ERR_CUDA)


@pytest.mark.gpu
def test_scratch_over_inputs_or_outputs_is_refused():
    dev = "cuda"
    pool = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    need = sk.sgemm_latent_attention_workspace(2, 8, 512, 64, 64, 20)
    assert 0 < need < 16 << 20

    def part(at, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        return pool[at : at + n].view(dtype).view(shape)

    at = dict(q=1 << 20, cache=2 << 20, table=12 << 20, lens=13 << 20, cu=14 << 20, out=15 << 20, lse=16 << 20, ws=20 << 20)

    def call(**kw):
        a = at | kw
        q, cache = part(a["q"], (2, 8, 576), torch.bfloat16), part(a["cache"], (41, 64, 576), torch.bfloat16)
        table, lens = part(a["table"], (2, 20), torch.int32), part(a["lens"], (2,), torch.int32)
        cu, out = part(a["cu"], (3,), torch.int32), part(a["out"], (2, 8, 512), torch.bfloat16)
        sk.sgemm_bf16_latent_attention(q, cache, table, lens, 512, 0.1, cu_q=cu, out=out,
                                       lse=part(a["lse"], (2, 8), torch.float32), workspace=pool[a["ws"] : a["ws"] + need])

    call()
    for name, start in at.items():
        if name != "ws":
            for ws in (start, start - need + 16):
                if ws >= 0 and not (name == "cache" and ws < 2 << 20):
                    with pytest.raises(sk.SgemmError) as e:
                        call(ws=ws)
                    assert e.value.status == sk.SGEMM_ERR_INVALID_ARG, name
    call(ws=(16 << 20) + 64)  # right behind lse
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
