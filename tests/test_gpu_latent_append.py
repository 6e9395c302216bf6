"""GPU: the append to the paged latent cache with the position rotation, against FP64."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"


def problem(T, H, R, E, page, seed=0, longest=500):
    g = torch.Generator().manual_seed(seed)
    pages = -(-T // page) + 3
    kv = torch.randn((T, R + E), generator=g).to(torch.bfloat16)
    q = torch.randn((T, H, E), generator=g).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(R, generator=g)).to(torch.bfloat16)
    cache = torch.randn((pages, page, R + E), generator=g).to(torch.bfloat16)
    slots = torch.randperm(pages * page, generator=g)[:T]
    angle = torch.rand((longest, E // 2), generator=g) * 6.28
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    pos = torch.randint(0, longest, (T,), generator=g)
    return kv, q, w, cache, slots, cs, pos


def expect(kv, q, w, cache, slots, cs, pos, inter, eps=1e-6):
    """(cache, bound, q, bound)"""
    E = cs.shape[1]
    R = kv.shape[1] - E
    cos, sin = cs[pos].double().chunk(2, 1)
    latent = kv[:, :R].double()
    lb = torch.zeros_like(latent)  # a plain copy
    if w is not None:
        latent, _ = D.add_rmsnorm(kv[:, :R], w, None, eps)
        lb = D.norm_y_bound(latent, R)
    k, km = D.rotate(kv[:, R:], cos, sin, inter)
    row, rb = torch.cat([latent, k], 1), torch.cat([lb, D.rotate_bound(k, km)], 1)
    want = cache.double().flatten(0, 1).clone()
    bound = torch.zeros_like(want)
    keep = slots >= 0
    want[slots[keep]] = row[keep]
    bound[slots[keep]] = rb[keep]
    qw, qm = D.rotate(q, cos[:, None], sin[:, None], inter)
    return want.view(cache.shape), bound.view(cache.shape), qw, D.rotate_bound(qw, qm)


def go(args, inter=True, norm=True, **kw):
    kv, q, w, cache, slots, cs, pos = args
    dev = [t.to(DEV) for t in args]
    H = q.shape[1]
    c, qo = sk.sgemm_bf16_latent_append(dev[0], dev[3], dev[4], dev[6], dev[5], dev[2] if norm else None,
                                        q=dev[1] if H else None, interleaved=inter, **kw)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    want, cb, qw, qb = expect(kv, q, w if norm else None, cache, slots, cs, pos, inter)
    D.check(c, want, cb, "cache")
    if H:
        D.check(qo, qw, qb, "q")
    return c, qo


@pytest.mark.parametrize("T,H", [(1, 0), (1, 1), (1, 32), (3, 20), (8, 128), (130, 5)])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_tokens_and_heads(T, H, inter, norm):
    go(problem(T, H, 512, 64, 16, seed=T + H), inter, norm)


@pytest.mark.parametrize("R,E", [(1, 2), (8, 8), (100, 16), (127, 6), (128, 32), (384, 64), (512, 128), (1024, 64), (1032, 64), (2000, 512)])
@pytest.mark.parametrize("inter", [True, False])
def test_widths(R, E, inter):
    go(problem(5, 3, R, E, 7, seed=R + E), inter)


@pytest.mark.parametrize("page", [1, 16, 64, 100])
def test_pages_and_padded_tokens(page):
    args = problem(40, 2, 512, 64, page, seed=page)
    args[4][::3] = -1
    args[4][5] = -(1 << 40)
    go(args)


def test_many_tokens():
    args = list(problem(3000, 4, 512, 64, 64, seed=1))
    args[4][100::17] = -1
    go(args)
    go(args, inter=False, norm=False)


@pytest.mark.parametrize("shift", [0, 1, 4])
def test_strided_views_and_gaps(shift):
    """Views that start on and off 16 bytes; what lies between them stays."""
    kv, q, w, cache, slots, cs, pos = problem(9, 6, 512, 64, 16, seed=2)
    want, cb, qw, qb = expect(kv, q, w, cache, slots, cs, pos, True)
    kvd = torch.zeros((9, 2, 640), dtype=torch.bfloat16, device=DEV)[:, 1, 8 + shift : 584 + shift]
    kvd.copy_(kv)
    pool = torch.full((cache.shape[0], 2, 16, 600), 3.0, dtype=torch.bfloat16, device=DEV)
    cd = pool[:, 1, :, 8 + shift : 584 + shift]
    cd.copy_(cache)
    qd = torch.zeros((9, 6, 192 + 2 * shift), dtype=torch.bfloat16, device=DEV)[..., 128 : 192]
    qd.copy_(q)
    full = torch.full((9, 6, 576 + 2 * shift), 3.0, dtype=torch.bfloat16, device=DEV)
    sk.sgemm_bf16_latent_append(kvd, cd, slots.to(DEV), pos.to(DEV), cs.to(DEV), w.to(DEV), q=qd, q_out=full[..., 512:576])
    torch.cuda.synchronize()
    D.check(cd, want, cb, "cache")
    D.check(full[..., 512:576], qw, qb, "q")
    assert torch.all(full[..., :512] == 3) and torch.all(pool[:, 0] == 3)
    assert torch.all(pool[..., : 8 + shift] == 3) and torch.all(pool[..., 584 + shift :] == 3)


@pytest.mark.parametrize("inter", [True, False])
def test_queries_in_place_and_beside(inter):
    kv, q, w, cache, slots, cs, pos = problem(7, 5, 512, 64, 16, seed=3)
    _, _, qw, qb = expect(kv, q, w, cache, slots, cs, pos, inter)
    dev = [t.to(DEV) for t in (kv, cache, slots, pos, cs, w)]
    qd = q.to(DEV)
    _, got = sk.sgemm_bf16_latent_append(*dev, q=qd, q_out=qd, interleaved=inter)
    assert got is qd
    D.check(qd, qw, qb, "q")
    two = torch.zeros((7, 5, 128), dtype=torch.bfloat16, device=DEV)
    two[..., :64] = q.to(DEV)
    sk.sgemm_bf16_latent_append(*dev, q=two[..., :64], q_out=two[..., 64:], interleaved=inter)
    D.check(two[..., 64:], qw, qb, "q")
    assert torch.equal(two[..., :64], q.to(DEV))
    with pytest.raises(sk.SgemmError):
        sk.sgemm_bf16_latent_append(*dev, q=two[..., :64], q_out=two[..., 32:96], interleaved=inter)


@pytest.mark.parametrize("R", [512, 100])
def test_out_of_range_is_skipped_and_reported(R):
    kv, q, w, cache, slots, cs, pos = problem(6, 2, R, 64, 16, seed=4)
    _ = sk.sgemm_device_errors()
    bad = slots.clone()
    bad[2] = cache.shape[0] * 16
    pos2 = pos.clone()
    pos2[4] = cs.shape[0]
    pos2[5] = -1
    bad[5] = -1  # padded: its position is of no account
    dev = [t.to(DEV) for t in (kv, cache, bad, pos2, cs, w)]
    got, qo = sk.sgemm_bf16_latent_append(*dev, q=q.to(DEV))
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    skipped = slots.clone()
    skipped[2] = skipped[5] = -1
    want, cb, qw, qb = expect(kv, q, w, cache, skipped, cs, pos, True)
    want.flatten(0, 1)[slots[4], R:] = float("nan")
    qw[4:] = float("nan")
    D.check(got, want, cb, "cache")
    D.check(qo, qw, qb, "q")


def test_offsets_past_32_bits():
    R, E, page = 128, 64, 4
    stride = (1 << 30) + 64
    flat = torch.zeros(3 * stride + page * (R + E), dtype=torch.bfloat16, device=DEV)
    cache = torch.as_strided(flat, (4, page, R + E), (stride, R + E, 1))
    kv, q, w, small, _, cs, pos = problem(4, 1, R, E, page, seed=5)
    small = small[:4]
    cache.copy_(small.to(DEV))
    slots = torch.tensor([3, 7, 14, 15])
    sk.sgemm_bf16_latent_append(kv.to(DEV), cache, slots.to(DEV), pos.to(DEV), cs.to(DEV), w.to(DEV))
    torch.cuda.synchronize()
    want, cb, _, _ = expect(kv, q, w, small, slots, cs, pos, True)
    D.check(cache, want, cb, "cache")


def test_graph_and_other_stream():
    args = problem(8, 32, 512, 64, 64, seed=6)
    kv, q, w, cache, slots, cs, pos = args
    dev = [t.to(DEV) for t in (kv, cache, slots, pos, cs, w)]
    qd, qo = q.to(DEV), torch.empty_like(q, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        for _ in range(2):
            sk.sgemm_bf16_latent_append(*dev, q=qd, q_out=qo, flags=sk.SGEMM_FLAG_PDL)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want, cb, qw, qb = expect(kv, q, w, cache, slots, cs, pos, True)
    D.check(dev[1], want, cb, "cache")
    D.check(qo, qw, qb, "q")
