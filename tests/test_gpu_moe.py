"""GPU: a router's choice and the experts' products for a few tokens, against FP64."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def done():
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0


# ------------------------------------------------------------------------------------------ router
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 64, 129])
@pytest.mark.parametrize("E,k", [(8, 8), (16, 2), (128, 8), (160, 6), (1, 1)])
def test_route(T, E, k):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x, w = normal(g, T, 512), normal(g, E, 512, std=512 ** -0.5)
    ids, weights = sk.sgemm_bf16_moe_route(x.to(DEV), w.to(DEV), k)
    done()
    L.check_route(ids, weights, x, w, k)


@pytest.mark.parametrize("width", [8, 24, 40, 1000, 4096, 7168])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_scores_and_widths(width, scoring, with_bias):
    g = torch.Generator().manual_seed(width)
    x, w = normal(g, 5, width), normal(g, 1024, width, std=width ** -0.5)
    bias = torch.randn(1024, generator=g) if with_bias else None
    ids, weights = sk.sgemm_bf16_moe_route(x.to(DEV), w.to(DEV), 16, bias.to(DEV) if with_bias else None, scoring,
                                           renormalize=width != 40, scale=2.5)
    done()
    L.check_route(ids, weights, x, w, 16, bias, scoring, width != 40, 2.5)


def test_route_ties_go_to_the_lower_index():
    """Whole numbers: logits are exact, and many are equal."""
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-2, 3, (40, 64), generator=g).to(torch.bfloat16)
    w = torch.randint(-1, 2, (100, 64), generator=g).to(torch.bfloat16)
    w[50:] = w[:50]
    x[7] = 0
    want = torch.sort(x.double() @ w.double().T, dim=1, descending=True, stable=True)[1][:, :9]
    ids, _ = sk.sgemm_bf16_moe_route(x.to(DEV), w.to(DEV), 9, scoring="sigmoid")
    done()
    assert torch.equal(ids.cpu().long(), want)
    # with a bias the scores are compared: all are 1/2 for a token of zeros
    ids, _ = sk.sgemm_bf16_moe_route(x.to(DEV), w.to(DEV), 9, torch.zeros(100, device=DEV), "sigmoid")
    done()
    assert ids[7].tolist() == list(range(9))


def test_route_strided_and_nan():
    g = torch.Generator().manual_seed(2)
    x, w = normal(g, 6, 80), normal(g, 20, 88)
    x[2, 5] = NAN
    wide_ids = torch.full((6, 7), -5, dtype=torch.int32, device=DEV)
    wide_w = torch.full((6, 9), 3.0, device=DEV)
    sk.sgemm_bf16_moe_route(x.to(DEV)[:, :72], w.to(DEV)[:, 16:], 4, ids=wide_ids[:, :4], weights=wide_w[:, 2:6])
    done()
    rows = [0, 1, 3, 4, 5]
    L.check_route(wide_ids[rows, :4], wide_w[rows, 2:6], x[rows, :72], w[:, 16:], 4)
    # a token of NaN takes the first experts with weights of NaN, and no other token's
    assert wide_ids[2, :4].tolist() == [0, 1, 2, 3] and torch.isnan(wide_w[2, 2:6]).all()
    assert torch.all(wide_ids[:, 4:] == -5) and torch.all(wide_w[:, :2] == 3) and torch.all(wide_w[:, 6:] == 3)
    with pytest.raises(ValueError, match="unit stride"):
        sk.sgemm_bf16_moe_route(x.to(DEV).T, w.to(DEV), 4)


def test_route_takes_nan_last():
    x = torch.ones((1, 8), dtype=torch.bfloat16)
    w = torch.tensor([-3.0, NAN, 1.0, -INF, 2.0])[:, None].expand(5, 8).to(torch.bfloat16).contiguous()
    ids, _ = sk.sgemm_bf16_moe_route(x.to(DEV), w.to(DEV), 5, scoring="sigmoid")
    done()
    assert ids[0].tolist() == [4, 2, 0, 3, 1]


# ----------------------------------------------------------------------------------------- experts
def problem(T, E, k, width, F, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = normal(g, T, width)
    gu, dn = normal(g, E, 2 * F, width, std=std * width ** -0.5), normal(g, E, width, F, std=F ** -0.5)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else torch.zeros((0, k), dtype=torch.int32)
    weights = torch.rand((T, k), generator=g) + 0.05
    return x, gu, dn, ids, weights


def compare(x, gu, dn, ids, weights, **kw):
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV), **kw)
    done()
    want, bound = L.experts(x, gu, dn, ids, weights)
    D.check(y, want, bound, "y")
    return y


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 127, 128])
def test_tokens(T):
    compare(*problem(T, 12, 3, 256, 192, T))


@pytest.mark.parametrize("width,F", [(8, 8), (8, 1000), (64, 8), (72, 56), (1000, 24), (1032, 520), (2048, 64), (4104, 264), (512, 2048)])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (5, 9, 4), (40, 3, 3)])
def test_widths(width, F, T, E, k):
    compare(*problem(T, E, k, width, F, width + F + T))


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (33, 1), (64, 8), (300, 8), (1024, 2)])
def test_experts(E, k):
    compare(*problem(11, E, k, 64, 40, E))


def test_entries_that_are_not_used():
    x, gu, dn, ids, weights = problem(9, 10, 4, 128, 64, 5)
    ids[0] = -1            # a padded token
    ids[3, 1:] = -7
    ids[5, 0] = -1
    x[0] = NAN             # what a padded token holds
    weights[3, 1:] = NAN   # and what an unused entry's weight is
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV))
    done()
    x[0] = 0
    weights[3, 1:] = 0
    want, bound = L.experts(x, gu, dn, ids, weights)
    D.check(y, want, bound, "y")
    assert torch.all(y[0] == 0)


def test_no_entry_is_used_at_all():
    x, gu, dn, ids, weights = problem(3, 5, 2, 128, 64, 6)
    ids[:] = -1
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV))
    done()
    assert torch.all(y == 0)
    assert sk.sgemm_bf16_moe_experts(x.to(DEV)[:0], gu.to(DEV), dn.to(DEV), ids.to(DEV)[:0], weights.to(DEV)[:0]).shape == (0, 128)


def test_an_expert_twice_counts_with_both_weights():
    x, gu, dn, ids, weights = problem(4, 6, 3, 96, 48, 7)
    ids[1] = torch.tensor([2, 5, 2])
    compare(x, gu, dn, ids, weights)


def test_an_index_past_the_experts():
    x, gu, dn, ids, weights = problem(4, 6, 3, 96, 48, 8)
    ids[2, 1] = 6
    ids[3, 0] = 2 ** 30
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV))
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    want, bound = L.experts(x, gu, dn, ids, weights)
    D.check(y, want, bound, "y")


def test_a_token_of_nan_reaches_no_other():
    x, gu, dn, ids, weights = problem(20, 8, 2, 128, 64, 9)
    clean = compare(x, gu, dn, ids, weights)
    x[4], x[11, 3] = NAN, INF
    y = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV))
    done()
    rest = [t for t in range(20) if t not in (4, 11)]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[4]).all() and not torch.isfinite(y[11]).any()


def test_strided_operands_and_what_lies_between():
    x, gu, dn, ids, weights = problem(6, 5, 2, 64, 40, 10)
    xs = torch.full((6, 200), NAN, dtype=torch.bfloat16, device=DEV)
    xs[:, 64:128] = x.to(DEV)
    gus = torch.full((5, 90, 72), NAN, dtype=torch.bfloat16, device=DEV)
    gus[:, :80, :64] = gu.to(DEV)
    dns = torch.full((5, 66, 48), NAN, dtype=torch.bfloat16, device=DEV)
    dns[:, :64, 8:] = dn.to(DEV)
    ws = torch.zeros((6, 5), device=DEV)
    ws[:, 1:3] = weights.to(DEV)
    i2 = torch.full((6, 3), 4, dtype=torch.int32, device=DEV)
    i2[:, 1:] = ids.to(DEV)
    ys = torch.full((7, 69), 9.0, dtype=torch.bfloat16, device=DEV)
    work = torch.full((sk.sgemm_moe_experts_workspace(6, 5, 2, 64, 40),), 255, dtype=torch.uint8, device=DEV)  # NaN
    sk.sgemm_bf16_moe_experts(xs[:, 64:128], gus[:, :80, :64], dns[:, :64, 8:], i2[:, 1:], ws[:, 1:3], y=ys[:6, 3:67], workspace=work)
    done()
    want, bound = L.experts(x, gu, dn, ids, weights)
    D.check(ys[:6, 3:67], want, bound, "y")
    assert torch.all(ys[6] == 9) and torch.all(ys[:, :3] == 9) and torch.all(ys[:, 67:] == 9)
    # the same numbers in dense buffers give the same bits
    dense = sk.sgemm_bf16_moe_experts(x.to(DEV), gu.to(DEV), dn.to(DEV), ids.to(DEV), weights.to(DEV))
    assert torch.equal(dense, ys[:6, 3:67])


def test_large_gates():
    """silu far out on both sides."""
    compare(*problem(5, 4, 2, 128, 64, 11, std=40.0))


def test_shared_experts_are_entries_with_weight_one():
    x, gu, dn, _, _ = problem(5, 9, 1, 128, 64, 12)
    router = normal(torch.Generator().manual_seed(3), 8, 128)
    ids = torch.full((5, 3), 8, dtype=torch.int32, device=DEV)
    weights = torch.ones((5, 3), device=DEV)
    sk.sgemm_bf16_moe_route(x.to(DEV), router.to(DEV), 2, ids=ids[:, :2], weights=weights[:, :2])
    compare(x, gu, dn, ids.cpu(), weights.cpu())


def test_a_captured_layer_follows_its_inputs():
    x, gu, dn, _, _ = problem(4, 16, 3, 256, 128, 13)
    g = torch.Generator().manual_seed(14)
    router = normal(g, 16, 256)
    xd, gd, dd, rd = x.to(DEV), gu.to(DEV), dn.to(DEV), router.to(DEV)
    ids = torch.empty((4, 3), dtype=torch.int32, device=DEV)
    weights = torch.empty((4, 3), device=DEV)
    y = torch.empty_like(xd)
    work = torch.empty(sk.sgemm_moe_experts_workspace(4, 16, 3, 256, 128), dtype=torch.uint8, device=DEV)

    def layer():
        for _ in range(2):  # two layers share the scratch
            sk.sgemm_bf16_moe_route(xd, rd, 3, ids=ids, weights=weights, flags=sk.SGEMM_FLAG_PDL)
            sk.sgemm_bf16_moe_experts(xd, gd, dd, ids, weights, y=y, workspace=work, flags=sk.SGEMM_FLAG_PDL)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in range(3):
        x = normal(torch.Generator().manual_seed(seed), 4, 256)
        xd.copy_(x)
        graph.replay()
        done()
        L.check_route(ids, weights, x, router, 3)
        want, bound = L.experts(x, gu, dn, ids.cpu(), weights.cpu())
        D.check(y, want, bound, "y")


def test_stalled_copies_end_in_nan_and_an_error():
    x, gu, dn, ids, weights = problem(3, 4, 2, 512, 256, 15)
    args = [t.to(DEV) for t in (x, gu, dn, ids, weights)]
    y = sk.sgemm_bf16_moe_experts(*args, flags=sk.SGEMM_FLAG_TEST_STALL)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 1
    assert torch.isnan(y).all()
    compare(x, gu, dn, ids, weights)


@pytest.mark.parametrize("T,E,k,width,F", [(1, 16, 2, 256, 64), (8, 32, 4, 512, 256), (70, 16, 4, 128, 128), (20, 8, 2, 64, 64)])
def test_chained_launches(T, E, k, width, F):
    """Router, experts and a GEMM one behind the other, each allowed to start while the one before runs, with one
    buffer of ids: as without that."""
    g = torch.Generator().manual_seed(T)
    x0 = normal(g, T, width).to(DEV)
    routers = [normal(g, E, width).to(DEV) for _ in range(4)]
    gu, dn = normal(g, E, 2 * F, width, std=width ** -0.5).to(DEV), normal(g, E, width, F, std=F ** -0.5).to(DEV)
    w = normal(g, width, width, std=width ** -0.5).to(DEV)
    n = min(T, 8)

    def chain(flags):
        x, y, z = x0.clone(), torch.zeros_like(x0), torch.zeros((n, width), dtype=torch.bfloat16, device=DEV)
        ids, weights = torch.zeros((T, k), dtype=torch.int32, device=DEV), torch.zeros((T, k), device=DEV)
        work = torch.empty(sk.sgemm_moe_experts_workspace(T, E, k, width, F), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for i in range(24):
            a, b = (x, y) if i % 2 == 0 else (y, x)
            sk.sgemm_bf16_moe_route(a, routers[i % 4], k, ids=ids, weights=weights, flags=flags)
            sk.sgemm_bf16_moe_experts(a, gu, dn, ids, weights, y=b, workspace=work, flags=flags)
            sk.sgemm_bf16_skinny_ex(b[:n], w, z, flags=flags)
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0
        return x, y, z, ids, weights

    for a, b in zip(chain(0), chain(sk.SGEMM_FLAG_PDL)):
        assert torch.equal(a, b)
