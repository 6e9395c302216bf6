"""GPU: the latent attention where one sequence needs more CTAs for its query rows than half of the
GPU's SMs, or than there are: one group of CTAs walks all sequences then, without scratch or a
joining kernel.  Just below that two groups do."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"


def compare(lens, qs, H, R, page=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    width = max([1, *need])
    cache = torch.randn((sum(need) + 2, page, R + 64), generator=g).to(torch.bfloat16)
    order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    q = torch.randn((sum(qs), H, R + 64), generator=g).to(torch.bfloat16)
    cu = torch.tensor([sum(qs[:b]) for b in range(len(qs) + 1)], dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32)
    need = sk.sgemm_latent_attention_workspace(len(lens), H, R, 64, page, width, max(qs))
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out, _ = sk.sgemm_bf16_latent_attention(q.to(DEV), cache.to(DEV), table.to(DEV), ln.to(DEV), R, 0.07, cu_q=cu.to(DEV),
                                            max_q=max(qs), lse=lse)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, R, 0.07, cu)
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")
    return need


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("more", [0, 1, 2])
def test_one_group_for_one_long_and_several_short_pieces_of_work(more):
    """128 heads: two CTAs for each new token.  At half of the SMs, and past it."""
    n = sms() // 4 + more
    need = compare([150, 700, 0, 64, 257], [1, n, 2, 0, 3], 128, 128, seed=more)
    assert (need == 0) == (2 * n > sms() // 2)


def test_more_rows_than_the_gpu_has_sms():
    n = sms() // 2 + 5
    assert compare([130, n + 70, 333], [1, n, 1], 128, 128, page=16, seed=5) == 0


def test_a_sequence_of_many_tokens_alone():
    """A third of its first tokens see nothing: more new tokens than cached rows."""
    assert compare([200], [300], 64, 256, seed=6) == 0


def test_full_width():
    assert compare([90, 400], [sms() // 4 + 2, 2], 128, 512, page=32, seed=7) == 0
