"""GPU: offsets that fall and rise again, so often that the sequences between them come to more work than 32 bits
count: nothing is computed, and the error word says so.

Taken without the bits that do not fit, or as it is, each case's work would keep a GPU busy for seconds at least, on
rows that several sequences write."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L

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


def test_many_overlapping_prompts():
    """2^19 sequences of 2^13 chunks and one of two: 2 chunks if the sum wraps."""
    n, pairs, last = 1 << 19, 1 << 19, 100
    cu = alternating(pairs, n, last)
    B = len(cu) - 1
    assert pairs * (n // 64) + -(-last // 64) == (1 << 32) + 2
    q = torch.ones((n, 1, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full((n, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    state = torch.full((2, 1, 64, 64), 3.0, device=DEV)
    slots = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    slots[0], slots[B - 1] = 0, 1
    sk.sgemm_bf16_linear_attention(q, q, q, torch.zeros((n, 1), device=DEV), state, slots, cu.to(DEV), out=out)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    assert torch.all(out == 9) and torch.all(state == 3)


def test_a_few_overlapping_prompts_are_computed():
    """Below that limit each sequence is: the states of all, and the rows that no two share."""
    n, Hv = 700, 2
    g = torch.Generator().manual_seed(1)
    q, k = ((torch.randn((n, Hv, 64), generator=g) / 8).to(torch.bfloat16) for _ in range(2))
    v = torch.randn((n, Hv, 64), generator=g).to(torch.bfloat16)
    decay = -torch.rand((n, Hv), generator=g) / 50
    cu = [0, 300, 200, n]  # the second falls; the first and the third share 200 .. 299
    state = torch.randn((3, Hv, 64, 64), generator=g)
    s, out = state.to(DEV), torch.zeros_like(v, device=DEV)
    sk.sgemm_bf16_linear_attention(q.to(DEV), k.to(DEV), v.to(DEV), decay.to(DEV), s, torch.arange(3, device=DEV),
                                   torch.tensor(cu, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    assert torch.equal(s[1].cpu(), state[1])
    for b, rows, alone in ((0, slice(0, 300), slice(0, 200)), (2, slice(200, n), slice(300, n))):
        want, last, ob, sb = L.linear(q[rows], k[rows], v[rows], decay[rows], state[b], 1.0, True)
        part = slice(alone.start - rows.start, alone.stop - rows.start)
        D.check(out[alone], want[part], ob[part], "out")
        D.check(s[b], last, sb, "state")


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
def test_many_empty_prompts_beside_many_rows(Dk, Dv):
    """So many sequences and rows that they might come to 2^30 chunks, and do not: short ones among empty ones, then
    rows of no sequence."""
    B, n = 1 << 14, 1 << 22
    lens = torch.zeros(B, dtype=torch.int64)
    used = [5, 700, 701, 9000, B - 1]
    lens[used] = torch.tensor([300, 1, 64, 130, 900])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)
    m = int(cu[-1])
    assert B * -(-n // 64) >= 1 << 30
    g = torch.Generator().manual_seed(2)
    q, k = ((torch.randn((m, 1, Dk), generator=g) * Dk ** -0.5).to(torch.bfloat16) for _ in range(2))
    v, decay = torch.randn((m, 1, Dv), generator=g).to(torch.bfloat16), -torch.rand((m, 1), generator=g) / 50
    state = torch.randn((len(used), 1, Dk, Dv), generator=g)
    slots = torch.full((B,), -1, dtype=torch.int64)
    slots[used] = torch.arange(len(used))

    def rows(t):
        wide = torch.zeros((n, *t.shape[1:]), dtype=t.dtype, device=DEV)
        wide[:m] = t
        return wide

    s, out = state.to(DEV), torch.full((n, 1, Dv), 9.0, dtype=torch.bfloat16, device=DEV)
    sk.sgemm_bf16_linear_attention(rows(q), rows(k), rows(v), rows(decay), s, slots.to(DEV), cu.to(DEV), out=out)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    assert torch.all(out[m:] == 9)
    for i, b in enumerate(used):
        r = slice(int(cu[b]), int(cu[b + 1]))
        want, last, ob, sb = L.linear(q[r], k[r], v[r], decay[r], state[i], 1.0, True)
        D.check(out[r], want, ob, "out")
        D.check(s[i], last, sb, "state")
