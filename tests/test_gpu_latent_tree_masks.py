"""GPU: the masks of drafted tokens at their limits."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L
from test_gpu_latent_attention import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("words", [(1 << 25) - 1, 1 << 25])
def test_masks_of_many_words(words):
    """64 bits in each word are 2^31 of them: a limit of the masks' width, not of the tokens."""
    q, cache, table, ln, cu = make([100], [3], 16, seed=1)
    tree = torch.zeros((3, words), dtype=torch.int64, device=DEV)
    tree[:, 0] = torch.tensor([1, 3, 5])
    out, _ = sk.sgemm_bf16_latent_tree_attention(*(t.to(DEV) for t in (q, cache, table, ln)), 512, 0.05, tree, cu_q=cu.to(DEV), max_q=3)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    want, _, ob, _ = L.tree_attention(q, cache, table, ln, 512, 0.05, cu, [{0}, {0, 1}, {0, 2}])
    D.check(out, want, ob, "out")


def test_drafts_of_nan_reach_who_sees_them():
    q, cache, table, ln, cu = make([150], [4], 16, seed=2)
    masks = [{0}, {0, 1}, {0, 1, 2}, {0, 3}]
    at = 150 - 4 + 1
    cache[table[0, at // 64], at % 64, 7] = float("nan")
    tree = torch.tensor([[sum(1 << j for j in m)] for m in masks])
    out, _ = sk.sgemm_bf16_latent_tree_attention(*(t.to(DEV) for t in (q, cache, table, ln)), 512, 0.05, tree.to(DEV),
                                                 cu_q=cu.to(DEV), max_q=4)
    torch.cuda.synchronize()
    assert torch.isnan(out[[1, 2]]).all()
    cache[table[0, at // 64], at % 64, 7] = 0
    want, _, ob, _ = L.tree_attention(q, cache, table, ln, 512, 0.05, cu, masks)
    D.check(out[[0, 3]], want[[0, 3]], ob[[0, 3]], "out")
