"""GPU: latent attention for drafted tokens that see one another by a mask, against FP64."""
from __future__ import annotations

import math

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L
from test_gpu_latent_attention import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def words_of(masks, words):
    rows = []
    for m in masks:
        v = sum(1 << j for j in m)
        rows.append([(w - (1 << 64) if w >> 63 else w) for w in ((v >> (64 * i)) & (2 ** 64 - 1) for i in range(words))])
    return torch.tensor(rows, dtype=torch.int64).view(len(masks), words)


def trees(qs, seed):
    """Random trees: each token sees its ancestors and itself."""
    g = torch.Generator().manual_seed(seed)
    masks = []
    for n in qs:
        mine = []
        for i in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            mine.append((mine[parent] if parent >= 0 else set()) | {i})
        masks += mine
    return masks


def compare(lens, qs, H, masks=None, words=1, max_q=None, R=512, E=64, page=64, seed=0, scale=None, ld=None):
    q, cache, table, ln, cu = make(lens, qs, H, R, E, page, seed=seed)
    masks = trees(qs, seed) if masks is None else masks
    scale = (128 + E) ** -0.5 if scale is None else scale
    tree = words_of(masks, words).to(DEV)
    if ld:
        wide = torch.full((len(masks), ld), -1, dtype=torch.int64, device=DEV)
        wide[:, :words] = tree
        tree = wide[:, :words]
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    out, lse = sk.sgemm_bf16_latent_tree_attention(q.to(DEV), cache.to(DEV), table.to(DEV), ln.to(DEV), R, scale, tree,
                                                   cu_q=cu.to(DEV), max_q=max_q or max(1, max(qs)), lse=lse)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    want, wlse, ob, lb = L.tree_attention(q, cache, table, ln, R, scale, cu, masks)
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")
    return out, lse


@pytest.mark.parametrize("n", [1, 2, 5, 12, 16, 33, 64])
@pytest.mark.parametrize("H", [1, 8, 20, 32])
def test_trees(n, H):
    compare([200], [n], H, seed=n * 100 + H)


@pytest.mark.parametrize("length", [12, 13, 63, 64, 65, 75, 76, 77, 128, 139, 1000, 4099])
def test_lengths_and_where_the_drafts_begin_in_a_tile(length):
    compare([length], [12], 16, seed=length)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("R,E", [(512, 64), (128, 8), (384, 64)])
def test_pages_and_widths(page, R, E):
    compare([30, 170, 333], [7, 1, 20], 12, R=R, E=E, page=page, seed=page + R)


@pytest.mark.parametrize("n,words", [(65, 2), (100, 2), (130, 3), (64, 4)])
def test_more_drafts_than_a_word(n, words):
    compare([300, 160], [n, 3], 8, words=words, seed=n)


def test_masks_of_any_shape():
    """Not only trees: nothing, itself alone, later tokens, all; and bits of tokens that are not there."""
    qs = [6, 4]
    masks = [set(), {1}, {5, 0}, set(range(64)), {2, 63}, {0, 1, 2, 3, 4, 5}, {3}, {40, 41}, {0}, {1, 2}]
    compare([100, 70], qs, 16, masks=masks, seed=5)


def test_rows_that_see_nothing():
    out, lse = compare([4, 9], [4, 4], 16, masks=[set(), {0}, set(), {0, 3}] + [set()] * 4, seed=6)
    assert torch.all(out[[0, 2]] == 0) and torch.all(lse[[0, 2]] == -math.inf) and torch.isfinite(lse[4:]).all()


def test_fewer_rows_than_drafts():
    """The first drafts of a sequence have no row in the cache."""
    compare([3, 0, 20], [8, 2, 8], 12, seed=7)


def test_a_chain_is_the_causal_attention():
    qs, lens = [8, 3, 1], [500, 65, 1]
    q, cache, table, ln, cu = [t.to(DEV) for t in make(lens, qs, 32, seed=8)]
    masks = [set(range(i + 1)) for n in qs for i in range(n)]
    a, _ = sk.sgemm_bf16_latent_tree_attention(q, cache, table, ln, 512, 0.05, words_of(masks, 1).to(DEV), cu_q=cu, max_q=8)
    b, _ = sk.sgemm_bf16_latent_attention(q, cache, table, ln, 512, 0.05, cu_q=cu, max_q=8)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_hidden_drafts_of_nan_reach_nobody():
    q, cache, table, ln, cu = make([150], [6], 16, seed=9)
    masks = [{0}, {0, 1}, {2}, {0, 3}, {0, 1, 4}, {0, 1, 5}]
    for j in (2, 4):  # rows that only their own tokens see
        at = 150 - 6 + j
        cache[table[0, at // 64], at % 64] = float("nan") if j == 2 else float("inf")
    args = [t.to(DEV) for t in (q, cache, table, ln)]
    out, _ = sk.sgemm_bf16_latent_tree_attention(*args, 512, 0.05, words_of(masks, 1).to(DEV), cu_q=cu.to(DEV), max_q=6)
    torch.cuda.synchronize()
    rows = [0, 1, 3, 5]
    clean = cache.clone()
    for j in (2, 4):
        at = 150 - 6 + j
        clean[table[0, at // 64], at % 64] = 0
    want, _, ob, _ = L.tree_attention(q, clean, table, ln, 512, 0.05, cu, masks)
    D.check(out[rows], want[rows], ob[rows], "out")


def test_many_sequences_split_anywhere():
    qs = [1 + (7 * b) % 16 for b in range(40)]
    compare([q + (53 * b * b) % 300 for b, q in enumerate(qs)], qs, 8, R=128, page=16, seed=10)


def test_strided_masks_and_a_larger_max_q():
    compare([90, 120], [5, 9], 16, max_q=40, ld=3, seed=11)


def test_long_context():
    compare([20000], [16], 16, seed=12)


def test_captured():
    qs, lens = [5, 3], [300, 90]
    q, cache, table, ln, cu = make(lens, qs, 16, seed=13)
    d = [t.to(DEV) for t in (q, cache, table, ln, cu)]
    masks = trees(qs, 1)
    tree = words_of(masks, 1).to(DEV)
    out = torch.empty((8, 16, 512), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=DEV)

    def call():
        sk.sgemm_bf16_latent_tree_attention(d[0], d[1], d[2], d[3], 512, 0.07, tree, cu_q=d[4], max_q=5, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (2, 3):
        masks = trees(qs, seed)
        tree.copy_(words_of(masks, 1))
        graph.replay()
        torch.cuda.synchronize()
        want, _, ob, _ = L.tree_attention(q, cache, table, ln, 512, 0.07, cu, masks)
        D.check(out, want, ob, "out")
    assert sk.sgemm_device_errors() == 0
