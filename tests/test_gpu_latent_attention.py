"""GPU: attention over a paged latent cache against its FP64 definition, at the sizes, masks and
layouts where it can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(lens, qs, H, R=512, E=64, page=64, seed=0, spare=3, std=1.0, width=None):
    """A problem on the host: queries, a cache whose unused rows are NaN, shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    cache = torch.full((pages, page, R + E), float("nan"), dtype=torch.bfloat16)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max([1, *need]) if width is None else width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
        for i in range(need[b]):
            rows = min(page, n - i * page)
            cache[table[b, i], :rows] = torch.randn((rows, R + E), generator=g).to(torch.bfloat16)
    q = (torch.randn((sum(qs), H, R + E), generator=g) * std).to(torch.bfloat16)
    cu = torch.tensor([sum(qs[:b]) for b in range(len(qs) + 1)], dtype=torch.int32)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32), cu


def run(q, cache, table, lens, cu, R, scale, max_q, **kw):
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    out, lse = sk.sgemm_bf16_latent_attention(q.to(DEV), cache.to(DEV), table.to(DEV), lens.to(DEV), R, scale,
                                              cu_q=None if cu is None else cu.to(DEV), max_q=max_q, lse=lse, **kw)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    return out, lse


def compare(lens, qs, H, R=512, E=64, page=64, scale=None, max_q=None, **kw):
    q, cache, table, ln, cu = make(lens, qs, H, R, E, page, **kw)
    scale = (128 + E) ** -0.5 if scale is None else scale
    out, lse = run(q, cache, table, ln, cu, R, scale, max_q or max(1, max(qs)))
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, R, scale, cu)
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")
    return out, lse


@pytest.mark.parametrize("H", [1, 8, 16, 20, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("n", [1, 64, 200])
def test_heads(H, n):
    compare([n], [1], H, seed=H * 1000 + n)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 63, 64, 65, 127, 128, 129, 640, 1000, 4097, 20000])
def test_lengths(n):
    compare([n], [1], 32, seed=n)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192])
@pytest.mark.parametrize("R,E", [(512, 64), (128, 8), (256, 32), (384, 64)])
def test_pages_and_widths(page, R, E):
    compare([1, 70, 333], [1, 1, 1], 24, R=R, E=E, page=page, seed=page + R)


@pytest.mark.parametrize("H,qs", [(32, [2, 2, 2]), (20, [1, 8, 3]), (8, [2, 1, 2]), (5, [3, 3, 3]), (128, [4, 1, 2]),
                                  (16, [70, 5, 130])])
def test_several_new_tokens_see_causally(H, qs):
    compare([200, 65, 131], qs, H, page=16, seed=H)


def test_sequences_without_keys_or_tokens():
    out, lse = compare([0, 5, 0, 70], [1, 0, 2, 3], 12, page=32, seed=3)
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -math.inf)


def test_more_new_tokens_than_keys():
    # tokens 0..4 of 8 see nothing when 3 rows are cached
    out, lse = compare([3, 64], [8, 8], 16, seed=4)
    assert torch.all(out[:5] == 0) and torch.all(lse[:5] == -math.inf)
    assert torch.all(torch.isfinite(lse[5:]))


@pytest.mark.parametrize("B", [1, 2, 7, 64, 151, 152, 153, 400])
def test_batches_split_anywhere(B):
    lens = [1 + (37 * b * b + 11 * b) % 300 for b in range(B)]
    compare(lens, [1] * B, 16, page=16, R=128, seed=B)


def test_large_scores_and_a_late_maximum():
    """The running maximum moves in the last tiles, by far more than the lazy threshold."""
    q, cache, table, ln, cu = make([1500], [1], 32, seed=9)
    flat_page, row = int(table[0, 1490 // 64]), 1490 % 64
    cache[flat_page, row] = (q[0, 3].float() * 4).to(torch.bfloat16)
    scale = 576 ** -0.5
    out, lse = run(q, cache, table, ln, cu, 512, scale, 1)
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, 512, scale, cu)
    assert wlse[0, 3] > wlse[0, 4] + 40
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(scale):
    compare([500, 90], [1, 2], 32, scale=scale, seed=11)


def test_all_scores_far_below_zero():
    q, cache, table, ln, cu = make([300], [1], 16, seed=12)
    q = q.abs()
    cache = torch.where(torch.isnan(cache), cache, -cache.abs())
    out, lse = run(q, cache, table, ln, cu, 512, 4.0, 1)
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, 512, 4.0, cu)
    assert wlse.max() < -500
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")


def test_what_a_token_does_not_see_does_not_reach_it():
    """NaN and infinities in later tokens' rows, in rows past the end and in unused pages."""
    q, cache, table, ln, cu = make([130, 67], [3, 2], 24, page=16, seed=13)
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, 512, 0.1, cu)
    bad = cache.clone()
    for b, n in ((0, 130), (1, 67)):
        bad[table[b, (n - 1) // 16], (n - 1) % 16] = float("nan")
    bad[table[0, 128 // 16], 128 % 16, ::3] = float("inf")
    out, lse = run(q, bad, table, ln, cu, 512, 0.1, 3)
    for t in (0, 3):  # the first tokens see neither
        D.check(out[t], want[t], ob[t], "out")
        D.check(lse[t], wlse[t], lb[t], "lse")
    assert torch.all(torch.isnan(out[2])) and torch.all(torch.isnan(out[4]))


def test_strided_views():
    q, cache, table, ln, cu = make([100, 3], [1, 1], 12, page=16, seed=14)
    want, wlse, ob, lb = D.latent_attention(q, cache, table, ln, 512, 0.07, cu)
    qd = torch.zeros((2, 12, 2, 600), dtype=torch.bfloat16, device=DEV)[:, :, 1, 8:584]
    qd.copy_(q)
    layers = torch.zeros((cache.shape[0], 3, 16, 640), dtype=torch.bfloat16, device=DEV)
    cd = layers[:, 1, :, :576]
    cd.copy_(cache)
    wide = torch.full((2, 5 + table.shape[1]), 1 << 20, dtype=torch.int32, device=DEV)
    td = wide[:, 2 : 2 + table.shape[1]]
    td.copy_(table)
    big = torch.full((12, 2, 600), 5.0, dtype=torch.bfloat16, device=DEV)
    od = big.transpose(0, 1)[:, :, 6:518]  # heads outermost
    ld = torch.full((2, 20), 5.0, device=DEV)
    out, lse = sk.sgemm_bf16_latent_attention(qd, cd, td, ln.to(DEV), 512, 0.07, out=od, lse=ld[:, :12])
    torch.cuda.synchronize()
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")
    assert torch.all(big[..., :6] == 5) and torch.all(big[..., 518:] == 5) and torch.all(ld[:, 12:] == 5)


@pytest.mark.parametrize("H", [7, 20, 100])
def test_queries_whose_rows_are_not_evenly_spaced(H):
    """Some heads of each token: no one stride leads from row to row."""
    qs, lens = [1, 4, 2], [300, 77, 64]
    q, cache, table, ln, cu = make(lens, qs, H + 3, page=32, seed=21)
    out, lse = run(q[:, 2 : 2 + H], cache, table, ln, cu, 512, 0.06, 4)
    qd = q.to(DEV)
    got, _ = sk.sgemm_bf16_latent_attention(qd[:, 2 : 2 + H], cache.to(DEV), table.to(DEV), ln.to(DEV), 512, 0.06,
                                            cu_q=cu.to(DEV), max_q=4)
    torch.cuda.synchronize()
    want, wlse, ob, lb = D.latent_attention(q[:, 2 : 2 + H], cache, table, ln, 512, 0.06, cu)
    D.check(got, want, ob, "out")
    D.check(lse, wlse, lb, "lse")
    assert torch.equal(got.view(torch.int16), out.view(torch.int16))


def test_one_long_sequence_among_short_ones():
    """Most shares are pieces of one sequence, more than its joining warps take in one turn."""
    lens = [1 + 13 * b % 90 for b in range(40)]
    lens[17] = 30000
    compare(lens, [1] * 40, 16, R=128, seed=22)


@pytest.mark.parametrize("lens,H", [([1500, 0, 2900, 1, 700], 128), ([3000, 80], 512), ([40] * 20 + [9000], 64)])
def test_many_pieces_of_many_rows(lens, H):
    """Rows enough for one joining warp a sequence, and more pieces than it takes in one turn."""
    compare(lens, [1] * len(lens), H, seed=23)


def test_no_lse_no_cu_q_own_workspace_and_stream():
    q, cache, table, ln, cu = make([700, 300], [2, 2], 32, seed=15)
    want, _, ob, _ = D.latent_attention(q, cache, table, ln, 512, 0.05, cu)
    args = [t.to(DEV) for t in (q, cache, table, ln)]
    need = sk.sgemm_latent_attention_workspace(2, 32, 512, 64, 64, table.shape[1], 2)
    assert 0 < need <= sk.LATENT_WORKSPACE_MAX
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, none = sk.sgemm_bf16_latent_attention(*args, 512, 0.05, max_q=2, stream=s)
    b, _ = sk.sgemm_bf16_latent_attention(*args, 512, 0.05, max_q=2, stream=s,
                                          workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert none is None and torch.equal(a.view(torch.int16), b.view(torch.int16))
    D.check(a, want, ob, "out")
    with pytest.raises(sk.SgemmError) as err:
        sk.sgemm_bf16_latent_attention(*args, 512, 0.05, max_q=2,
                                       workspace=torch.empty(need - 4, dtype=torch.uint8, device=DEV))
    assert err.value.status == sk.SGEMM_ERR_NO_WORKSPACE


def test_same_bits_every_time_and_in_a_graph():
    q, cache, table, ln, cu = [t.to(DEV) for t in make([3000, 10, 700], [1, 1, 1], 32, seed=16)]
    out = torch.empty((3, 32, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3, 32), device=DEV)
    ws = torch.empty(sk.LATENT_WORKSPACE_MAX, dtype=torch.uint8, device=DEV)

    def call(flags=0):
        sk.sgemm_bf16_latent_attention(q, cache, table, ln, 512, 0.06, cu_q=cu, out=out, lse=lse, workspace=ws, flags=flags)

    call()
    torch.cuda.synchronize()
    first, first_lse = out.clone(), lse.clone()
    for _ in range(20):
        out.fill_(3)
        ws.fill_(255)  # NaN everywhere: nothing is read that this call did not write
        call()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and torch.equal(lse, first_lse)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        for _ in range(3):
            call(sk.SGEMM_FLAG_PDL)
    torch.cuda.current_stream().wait_stream(s)
    out.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and torch.equal(lse, first_lse)
    # a replay reads the lengths that are on the device then
    ln.copy_(torch.tensor([64, 9, 699], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want, wlse, ob, lb = D.latent_attention(*[t.cpu() for t in (q, cache, table, ln)], 512, 0.06, cu.cpu())
    D.check(out, want, ob, "out")
    D.check(lse, wlse, lb, "lse")


def test_a_row_does_not_depend_on_its_neighbours():
    """Heads are independent: a call with 32 heads and one with the first 7 of them agree."""
    q, cache, table, ln, cu = [t.to(DEV) for t in make([900], [1], 32, seed=17)]
    a, _ = sk.sgemm_bf16_latent_attention(q, cache, table, ln, 512, 0.06)
    b, _ = sk.sgemm_bf16_latent_attention(q[:, :7], cache, table, ln, 512, 0.06)
    torch.cuda.synchronize()
    assert (a[:, :7].float() - b.float()).abs().max() <= 2.0 ** -8 * a.float().abs().max()


def test_indices_out_of_range_are_skipped_and_reported():
    q, cache, table, ln, cu = make([100, 40], [1, 1], 16, page=16, seed=18)
    _ = sk.sgemm_device_errors()
    args = [t.to(DEV) for t in (q, cache)]
    table2 = table.clone()
    table2[0, 2] = cache.shape[0] + 5  # reads as zeros
    out, _ = sk.sgemm_bf16_latent_attention(*args, table2.to(DEV), ln.to(DEV), 512, 0.05)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    zeroed = torch.cat([cache, torch.zeros_like(cache[:1])])
    table2[0, 2] = cache.shape[0]
    want, _, ob, _ = D.latent_attention(q, zeroed, table2, ln, 512, 0.05, cu)
    D.check(out, want, ob, "out")
    # a length past the table is cut there
    long = torch.tensor([table.shape[1] * 16 + 9, 40], dtype=torch.int32)
    filled = torch.where(torch.isnan(cache), torch.zeros_like(cache), cache)
    out, _ = sk.sgemm_bf16_latent_attention(q.to(DEV), filled.to(DEV), table.to(DEV), long.to(DEV), 512, 0.05)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 2
    cut = torch.tensor([table.shape[1] * 16, 40], dtype=torch.int32)
    want, _, ob, _ = D.latent_attention(q, filled, table, cut, 512, 0.05, cu)
    D.check(out, want, ob, "out")


def test_offsets_past_32_bits():
    """Rows of a cache whose pages lie 4 GiB and more apart."""
    R, E, page = 128, 64, 16
    stride = (1 << 31) // 2 + 64  # elements from page to page: 2 GiB
    flat = torch.empty(3 * stride + page * (R + E), dtype=torch.bfloat16, device=DEV)
    cache = torch.as_strided(flat, (4, page, R + E), (stride, R + E, 1))
    q, small, table, ln, cu = make([60], [1], 8, R=R, E=E, page=page, seed=19, spare=0)
    cache.copy_(small.to(DEV))
    out, _ = sk.sgemm_bf16_latent_attention(q.to(DEV), cache, table.to(DEV), ln.to(DEV), R, 0.1)
    torch.cuda.synchronize()
    want, _, ob, _ = D.latent_attention(q, small, table, ln, R, 0.1, cu)
    D.check(out, want, ob, "out")


def test_a_stalled_copy_ends_in_nan_and_an_error_bit():
    q, cache, table, ln, cu = [t.to(DEV) for t in make([900, 30], [1, 1], 16, seed=20)]
    _ = sk.sgemm_device_errors()
    lse = torch.zeros((2, 16), device=DEV)
    out, _ = sk.sgemm_bf16_latent_attention(q, cache, table, ln, 512, 0.06, lse=lse, flags=sk.SGEMM_FLAG_TEST_STALL)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() & 1
    assert torch.all(torch.isnan(out)) and torch.all(torch.isnan(lse))
    out, _ = sk.sgemm_bf16_latent_attention(q, cache, table, ln, 512, 0.06)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0
    want, _, ob, _ = D.latent_attention(*[t.cpu() for t in (q, cache, table, ln)], 512, 0.06, cu.cpu())
    D.check(out, want, ob, "out")
