"""GPU: offsets that fall and rise again, so often that the sequences between them come to more work than 32 bits
count: nothing is computed, and the error word says so.

Taken without the bits that do not fit, or as it is, each case's work would keep a GPU busy for seconds at least, on
rows that several sequences write."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def alternating(pairs, n, last):
    """0, n, 0, n, ... (every second sequence falls), then a sequence of the first `last`."""
    return torch.tensor([0, n] * pairs + [0, last], dtype=torch.int32)


def drafts(pairs, n, last, H, length, page, width):
    """(arguments, blocks of 64 rows x tiles of 64 keys of all sequences)"""
    cu = alternating(pairs, n, last)
    B = len(cu) - 1
    q = torch.ones((n, H, 136), dtype=torch.bfloat16, device=DEV)
    cache = torch.ones((1, page, 136), dtype=torch.bfloat16, device=DEV)
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    lens = torch.full((B,), length, dtype=torch.int32, device=DEV)
    tree = torch.full((n, -(-n // 64)), -1, dtype=torch.int64, device=DEV)
    blocks = [-(-int(m) * H // 64) for m in (cu[1:] - cu[:-1]) if m > 0]
    return (q, cache, table, lens, tree, cu.to(DEV)), sum(blocks) * -(-length // 64)


def untouched(args, n, H):
    q, cache, table, lens, tree, cu = args
    out = torch.full((n, H, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, H), 7.0, device=DEV)
    work = torch.full((sk.LATENT_WORKSPACE_MAX,), 1, dtype=torch.uint8, device=DEV)
    sk.sgemm_bf16_latent_tree_attention(q, cache, table, lens, 128, 0.1, tree, cu_q=cu, max_q=n, out=out, lse=lse, workspace=work)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    assert torch.all(out == 9) and torch.all(lse == 7)


def test_many_overlapping_drafts():
    n, H, page, width = 1024, 16, 4096, 256
    args, work = drafts(2048, n, 3, H, page * width, page, width)
    assert work >= 1 << 32
    untouched(args, n, H)


def test_a_few_overlapping_drafts_over_long_contexts():
    """Few enough for a descriptor each (fewer blocks of rows than SMs)."""
    n, H, page, width = 28, 16, 1 << 20, 1023
    args, work = drafts(9, n, 28, H, page * width, page, width)
    assert 1 << 30 <= work < 1 << 31
    untouched(args, n, H)
