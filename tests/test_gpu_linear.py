"""GPU: linear attention with a decay for each head, single tokens and whole prompts, against the
recurrence in FP64."""
from __future__ import annotations

import math

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_oracle as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def problem(lens, Hk, Hv, Dk, Dv, seed, slowest=1000.0, pool=None):
    g = torch.Generator().manual_seed(seed)
    N, B = sum(lens), len(lens)
    q = (torch.randn((N, Hk, Dk), generator=g) * Dk ** -0.5).to(torch.bfloat16)
    k = (torch.randn((N, Hk, Dk), generator=g) * Dk ** -0.5).to(torch.bfloat16)
    v = torch.randn((N, Hv, Dv), generator=g).to(torch.bfloat16)
    decay = -torch.exp(-torch.rand((N, Hv), generator=g) * math.log(slowest))
    pool = pool or B + 2
    state = torch.randn((pool, Hv, Dk, Dv), generator=g)
    slots = torch.randperm(pool, generator=g)[:B]
    return q, k, v, decay, state, slots


def expect(q, k, v, g, state, slots, lens, scale, chunked, fresh=None):
    """(out, states, their bounds); a sequence without a slot starts from zeros and is not kept."""
    outs, last, sb = [], state.double().clone(), torch.full_like(state, 0.0).double()
    bounds, at = [], 0
    for b, n in enumerate(lens):
        slot = int(slots[b])
        used = 0 <= slot < state.shape[0]
        first = state[slot] if used and not (fresh is not None and fresh[b]) else torch.zeros_like(state[0])
        r = slice(at, at + n)
        o, S, ob, s_b = L.linear(q[r], k[r], v[r], g[r], first, scale, chunked)
        outs.append(o)
        bounds.append(ob)
        if used:
            last[slot], sb[slot] = S, s_b
        at += n
    return torch.cat(outs), last, torch.cat(bounds), sb


# ----------------------------------------------------------------------------------- single tokens
def step(q, k, v, g, state, slots, scale=1.0, **kw):
    s = state.to(DEV)
    out = sk.sgemm_bf16_linear_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), s, slots.to(DEV), scale, **kw)
    torch.cuda.synchronize()
    return out, s


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("B,Hk,Hv", [(1, 1, 1), (1, 4, 32), (3, 5, 5), (70, 2, 8), (10, 16, 32)])
def test_step(Dk, Dv, B, Hk, Hv):
    p = problem([1] * B, Hk, Hv, Dk, Dv, B + Hv)
    out, s = step(*p, scale=0.7)
    assert sk.sgemm_device_errors() == 0
    want, last, ob, sb = expect(*p, [1] * B, 0.7, False)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


@pytest.mark.parametrize("B", [5, 100])
def test_step_padded_and_bad_slots(B):
    q, k, v, g, state, slots = problem([1] * B, 4, 8, 128, 128, B)
    slots[::3] = -1
    q[0], k[0], v[0], g[0] = NAN, INF, NAN, NAN  # what a padded token holds
    out, s = step(q, k, v, g, state, slots)
    assert sk.sgemm_device_errors() == 0
    for t in (q, k, v, g):
        t[0] = 0
    want, last, ob, sb = expect(q, k, v, g, state, slots, [1] * B, 1.0, False)
    want[::3], ob[::3] = 0, 1e-300
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")
    slots[1] = B + 2
    out, _ = step(q, k, v, g, state, slots)
    assert sk.sgemm_device_errors() == 2 and torch.all(out[1] == 0)


def test_step_decays():
    q, k, v, g, state, slots = problem([1] * 4, 2, 4, 64, 128, 3)
    g[0], g[1], g[2], g[3] = 0.0, -INF, -200.0, 0.5
    out, s = step(q, k, v, g, state, slots)
    want, last, ob, sb = expect(q, k, v, g, state, slots, [1] * 4, 1.0, False)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def strided(q, k, v, g, state):
    """The same numbers inside wider buffers: one projection's output, heads outermost, and so on."""
    N, Hk, Dk = q.shape
    Hv, Dv = v.shape[1:]
    qkv = torch.full((N, 2 * Hk * Dk + Hv * Dv + 24), NAN, dtype=torch.bfloat16, device=DEV)
    views = []
    at = 8
    for t in (q, k, v):
        w = t.shape[1] * t.shape[2]
        views.append(qkv[:, at : at + w].unflatten(1, t.shape[1:]))
        views[-1].copy_(t)
        at += w
    views[1] = k.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    gs = torch.full((Hv, 3, N), NAN, device=DEV)
    gs[:, 1] = g.T.to(DEV)
    states = torch.full((state.shape[0], Hv, Dk + 1, Dv), 5.0, device=DEV)
    states[:, :, :Dk] = state.to(DEV)
    out = torch.full((Hv, N + 1, Dv + 2), 9.0, dtype=torch.bfloat16, device=DEV)
    return (*views, gs[:, 1].T, states, out)


def test_step_strided():
    p = problem([1] * 7, 3, 6, 128, 64, 4)
    q, k, v, g, states, out = strided(*p[:5])
    o = out.transpose(0, 1)[:7, :, :64]
    sk.sgemm_bf16_linear_step(q, k, v, g, states[:, :, :128], p[5].to(DEV), 1.5, out=o)
    torch.cuda.synchronize()
    want, last, ob, sb = expect(*p, [1] * 7, 1.5, False)
    D.check(o, want, ob, "out")
    D.check(states[:, :, :128], last, sb + 1e-300, "state")
    assert torch.all(states[:, :, 128] == 5) and torch.all(out[:, 7] == 9) and torch.all(out[:, :, 64:] == 9)


def test_step_one_decay_a_head_for_all_tokens():
    q, k, v, _, state, slots = problem([1] * 9, 4, 4, 128, 128, 5)
    slopes = -torch.tensor([0.5, 0.25, 0.125, 0.0625])
    g = slopes.to(DEV).expand(9, 4)
    assert g.stride() == (0, 1)
    s = state.to(DEV)
    out = sk.sgemm_bf16_linear_step(q.to(DEV), k.to(DEV), v.to(DEV), g, s, slots.to(DEV))
    torch.cuda.synchronize()
    want, last, ob, sb = expect(q, k, v, slopes.expand(9, 4), state, slots, [1] * 9, 1.0, False)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_step_captured():
    q, k, v, g, state, slots = problem([1] * 3, 4, 4, 128, 128, 6)
    d = [t.to(DEV) for t in (q, k, v, g, state, slots)]
    out = torch.empty_like(d[2])
    sk.sgemm_bf16_linear_step(*d, out=out)
    d[4].copy_(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # three tokens alike
            sk.sgemm_bf16_linear_step(*d, out=out, flags=sk.SGEMM_FLAG_PDL)
    graph.replay()
    torch.cuda.synchronize()
    three = [t.repeat_interleave(3, 0) for t in (q, k, v, g)]
    want, last, ob, sb = expect(*three, state, slots, [3] * 3, 1.0, False)
    D.check(out, want[2::3], ob[2::3], "out")
    D.check(d[4], last, sb + 1e-300, "state")


# ----------------------------------------------------------------------------------------- prompts
def prompt(q, k, v, g, state, slots, lens, scale=1.0, fresh=None, errors=0, cu=None, **kw):
    s = state.to(DEV)
    if cu is None:
        cu = [sum(lens[:b]) for b in range(len(lens) + 1)]
    out = sk.sgemm_bf16_linear_attention(
        q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), s, slots.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), scale,
        fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.int32, device=DEV), **kw)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == errors
    return out, s


def compare(lens, Hk, Hv, Dk=128, Dv=128, seed=0, scale=1.0, fresh=None, slowest=1000.0):
    p = problem(lens, Hk, Hv, Dk, Dv, seed, slowest)
    out, s = prompt(*p, lens, scale, fresh)
    want, last, ob, sb = expect(*p, lens, scale, True, fresh)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")
    return out, s


@pytest.mark.parametrize("n", [1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 191, 256, 300, 511, 1000])
def test_lengths(n):
    compare([n], 2, 2, seed=n)


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("n", [1, 64, 100, 400])
def test_widths(Dk, Dv, n):
    compare([n], 3, 6, Dk, Dv, seed=n + Dk, scale=0.3)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 8), (2, 4), (5, 5), (16, 16), (4, 64)])
def test_heads(Hk, Hv):
    compare([150, 70], Hk, Hv, 64, 64, seed=Hk * 10 + Hv)


@pytest.mark.parametrize("lens", [[1, 1, 1], [64, 64], [5, 700, 1, 128, 63], [0, 10, 0], [0, 0], [300] * 7, [2000, 3, 1]])
def test_ragged(lens):
    compare(lens, 2, 2, seed=sum(lens) + len(lens), fresh=[b % 2 for b in range(len(lens))])


def test_many_sequences():
    compare([1 + (37 * b * b) % 150 for b in range(90)], 1, 2, 64, 64, seed=3, fresh=[b % 3 == 0 for b in range(90)])


@pytest.mark.parametrize("Hv", [1, 3])
def test_long(Hv):
    compare([9000], 1, Hv, 64, 64, seed=Hv, slowest=1e4)


def test_decays():
    """Fast and slow ones, none, all, and what passes single precision's range."""
    p = problem([400], 1, 6, 128, 128, 4)
    g = p[3]
    g[:, 0] = 0.0
    g[:, 1] = -100.0
    g[::37, 2] = -INF
    g[:, 3] = -1e-6
    g[:, 4] = -3e38
    g[150:250, 5] = 0.01
    out, s = prompt(*p, [400])
    want, last, ob, sb = expect(*p, [400], 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_slots():
    """No slot: from zeros and not kept; fresh: from zeros whatever the slot holds."""
    lens = [70, 200, 5, 64]
    p = problem(lens, 2, 4, 128, 128, 5)
    p[5][1] = -1
    p[4][p[5][2]] = NAN
    out, s = prompt(*p, lens, fresh=[0, 0, 1, 0])
    state = p[4].clone()
    state[p[5][2]] = 0
    want, last, ob, sb = expect(*p[:4], state, p[5], lens, 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")
    p[5][3] = 99
    prompt(*p, lens, errors=2)


def test_sequences_without_tokens_keep_their_slots():
    q, k, v, g, state, slots = problem([50, 60], 2, 2, 64, 128, 6, pool=6)
    slots = torch.tensor([3, 0, 5, 1])
    cu = [0, 50, 50, 50, 110]
    out, s = prompt(q, k, v, g, state, slots, None, cu=cu, fresh=[0, 0, 1, 1])
    assert torch.equal(s[0].cpu(), state[0]) and torch.all(s[5] == 0)
    assert torch.equal(s[[2, 4]].cpu(), state[[2, 4]])
    want, last, ob, sb = expect(q, k, v, g, state, torch.tensor([3, 1]), [50, 60], 1.0, True, [0, 1])
    D.check(out, want, ob, "out")
    D.check(s[[1, 3]], last[[1, 3]], sb[[1, 3]], "state")


def test_offsets_that_fall_are_skipped():
    q, k, v, g, state, slots = problem([50, 60], 2, 2, 64, 64, 7, pool=6)
    for cu in ([0, 50, 40, 110], [0, 50, 111, 110], [-1, 50, 50, 110]):
        out = torch.full((110, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        _, s = prompt(q, k, v, g, state, torch.tensor([2, 4, 1]), None, cu=cu, errors=2, out=out)
        bad = [b for b in range(3) if not 0 <= cu[b] <= cu[b + 1] <= 110]
        for b in bad:
            assert torch.equal(s[[2, 4, 1][b]].cpu(), state[[2, 4, 1][b]])


def test_rows_outside_the_sequences_are_left_alone():
    q, k, v, g, state, slots = problem([30, 100, 40], 2, 2, 128, 128, 8)
    for t in (q, k, v, g):
        t[:30], t[130:] = NAN, NAN
    out = torch.full((170, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    _, s = prompt(q, k, v, g, state, slots[1:2], None, cu=[30, 130], out=out)
    assert torch.all(out[:30] == 9) and torch.all(out[130:] == 9)
    r = slice(30, 130)
    want, last, ob, sb = expect(q[r], k[r], v[r], g[r], state, slots[1:2], [100], 1.0, True)
    D.check(out[r], want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_a_neighbour_of_nan_reaches_no_other_sequence():
    lens = [100, 77, 200]
    p = problem(lens, 2, 4, 128, 128, 9)
    clean, cs = prompt(*p, lens)
    for t in p[:4]:
        t[100:177] = NAN
    out, s = prompt(*p, lens)
    rows = [*range(100), *range(177, 377)]
    assert torch.equal(out[rows], clean[rows]) and torch.equal(s[p[5][[0, 2]]], cs[p[5][[0, 2]]])


def test_strided():
    lens = [90, 75]
    p = problem(lens, 3, 6, 128, 64, 10)
    q, k, v, g, states, out = strided(*p[:5])
    o = out.transpose(0, 1)[:165, :, :64]
    cu = torch.tensor([0, 90, 165], dtype=torch.int32, device=DEV)
    work = torch.full((sk.sgemm_linear_attention_workspace(165, 2, 6, 128, 64),), 255, dtype=torch.uint8, device=DEV)
    sk.sgemm_bf16_linear_attention(q, k, v, g, states[:, :, :128], p[5].to(DEV), cu, 1.5, out=o, workspace=work)
    torch.cuda.synchronize()
    want, last, ob, sb = expect(*p, lens, 1.5, True)
    D.check(o, want, ob, "out")
    D.check(states[:, :, :128], last, sb + 1e-300, "state")
    assert torch.all(states[:, :, 128] == 5) and torch.all(out[:, 165] == 9) and torch.all(out[:, :, 64:] == 9)


def test_a_prompt_in_parts_and_then_tokens():
    """A prompt in two calls, then single tokens, is the recurrence over all of it."""
    n, cut = 203, 200
    p = problem([n], 2, 4, 128, 128, 11)
    q, k, v, g, state, slots = [t.to(DEV) for t in p]
    outs = []
    for a, b in ((0, 77), (77, cut)):
        outs.append(sk.sgemm_bf16_linear_attention(q[a:b], k[a:b], v[a:b], g[a:b], state, slots,
                                                   torch.tensor([0, b - a], dtype=torch.int32, device=DEV)))
    for t in range(cut, n):
        r = slice(t, t + 1)
        outs.append(sk.sgemm_bf16_linear_step(q[r], k[r], v[r], g[r], state, slots))
    torch.cuda.synchronize()
    want, last, ob, sb = expect(*p, [n], 1.0, True)
    D.check(torch.cat(outs), want, ob, "out")
    D.check(state, last, sb + 1e-300, "state")


def test_captured():
    lens = [100, 300]
    p = problem(lens, 2, 2, 128, 128, 12)
    d = [t.to(DEV) for t in p]
    cu = torch.tensor([0, 100, 400], dtype=torch.int32, device=DEV)
    out = torch.empty_like(d[2])
    work = torch.empty(sk.sgemm_linear_attention_workspace(400, 2, 2, 128, 128), dtype=torch.uint8, device=DEV)

    def call():
        sk.sgemm_bf16_linear_attention(*d, cu, out=out, workspace=work, flags=sk.SGEMM_FLAG_PDL)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([100, 300], [250, 150], [0, 400]):
        cu.copy_(torch.tensor([0, lens[0], 400]))
        d[4].copy_(p[4])
        graph.replay()
        torch.cuda.synchronize()
        want, last, ob, sb = expect(*p, lens, 1.0, True)
        D.check(out, want, ob, "out")
        D.check(d[4], last, sb + 1e-300, "state")
    assert sk.sgemm_device_errors() == 0


def test_stalled_copies_end_in_nan_and_an_error():
    lens = [300]
    p = problem(lens, 2, 2, 128, 128, 13)
    out, _ = prompt(*p, lens, errors=1, flags=sk.SGEMM_FLAG_TEST_STALL)
    assert torch.isnan(out).all()
    compare(lens, 2, 2, seed=13)


def test_what_is_not_finite_reaches_later_tokens_only():
    """In q its token, in k and g its head from its token on (of the states, k the element's row), in v its
    element from its token on."""
    n = 400
    p = problem([n], 4, 4, 128, 128, 14)
    clean, _ = prompt(*p, [n])
    q, k, v, g = p[:4]
    q[100, 0] = NAN
    k[150, 1, 7] = INF
    v[77, 2, 5], v[200, 2, 100], v[201, 2, 100], v[333, 2, 64] = NAN, -INF, NAN, INF
    g[390, 3] = NAN
    out, s = prompt(*p, [n])
    hit = torch.zeros((n, 4, 128), dtype=torch.bool)
    hit[100, 0] = True
    hit[150:, 1] = True
    hit[77:, 2, 5], hit[200:, 2, 100], hit[333:, 2, 64] = True, True, True
    hit[390:, 3] = True
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])
    assert not torch.isfinite(out.cpu()[hit]).any()
    last = s[p[5][0]].cpu()
    assert torch.isfinite(last[0]).all() and not torch.isfinite(last[3]).any()
    assert not torch.isfinite(last[1][7]).any()  # a key element's row of the state
    assert torch.isfinite(last[1][torch.arange(128) != 7]).all()
    gone = torch.zeros(128, dtype=torch.bool)
    gone[[5, 64, 100]] = True
    assert not torch.isfinite(last[2][:, gone]).any() and torch.isfinite(last[2][:, ~gone]).all()


def test_rows_of_out_that_start_on_four_bytes():
    n = 130
    p = problem([n], 2, 2, 128, 128, 15)
    wide = torch.full((n, 2, 134), 9.0, dtype=torch.bfloat16, device=DEV)
    out, _ = prompt(*p, [n], out=wide[:, :, 2:130])
    dense, _ = prompt(*p, [n])
    assert torch.equal(out, dense) and torch.all(wide[:, :, :2] == 9) and torch.all(wide[:, :, 130:] == 9)


@pytest.mark.parametrize("B", [255, 256, 257, 600])
def test_batches_that_take_several_passes_over_their_offsets(B):
    lens = [(b * b * 7) % 5 if b % 3 else 0 for b in range(B)]
    lens[B - 1] = 130
    compare(lens, 1, 1, 64, 64, seed=B, fresh=[b % 2 for b in range(B)])


@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv,top", [(40, 2, 8, 128, 128, 200), (24, 16, 16, 128, 64, 350), (200, 1, 8, 64, 64, 130),
                                                (256, 4, 4, 64, 128, 100), (9, 3, 18, 128, 128, 129)])
def test_more_sequences_and_heads_than_sms(B, Hk, Hv, Dk, Dv, top):
    """Whole sequences in several rounds, the longest first: lengths in no order, some of them 0."""
    lens = [(b * b * 31 + 17 * b) % (top + 1) if b % 7 else 0 for b in range(B)]
    lens[B // 2] = top
    compare(lens, Hk, Hv, Dk, Dv, seed=B, fresh=[b % 2 for b in range(B)])


def test_more_sequences_than_sms_with_bad_ones():
    B, Hv = 60, 8
    lens = [1 + (37 * b * b) % 150 for b in range(B)]
    q, k, v, g, state, slots = problem(lens, 2, Hv, 64, 64, 21, pool=70)
    want, last, ob, sb = expect(q, k, v, g, state, slots, lens, 1.0, True)
    at = [sum(lens[:b]) for b in range(B + 1)]
    # one sequence more, which runs backwards, a slot outside the pool, and one that is none
    spare = [s for s in range(70) if s not in slots.tolist()]
    cu = at[:31] + [at[30] - 5] + [at[30]] + at[31:]
    cu[31] = at[30] - 5  # sequence 30 falls; 31 repeats rows of the one before
    slots2 = torch.cat([slots[:30], torch.tensor([spare[0], -1]), slots[30:]])
    out = torch.full((sum(lens), Hv, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    out, s = prompt(q, k, v, g, state, slots2, None, cu=cu, errors=2, out=out)
    # sequence 31 writes rows that another one has too: those are left out
    rows = torch.ones(sum(lens), dtype=torch.bool)
    rows[at[30] - 5:at[30]] = False
    D.check(out[rows], want[rows], ob[rows], "out")
    assert torch.equal(s[spare[0]].cpu(), state[spare[0]])
    used = torch.tensor(slots.tolist())
    D.check(s[used], last[used], sb[used] + 1e-300, "state")
    slots3 = slots.clone()
    slots3[13] = 70
    out, s = prompt(q, k, v, g, state, slots3, lens, errors=2)
    others = torch.cat([slots[:13], slots[14:]])
    D.check(s[others], last[others], sb[others] + 1e-300, "state")
    assert torch.equal(s[slots[13]].cpu(), state[slots[13]])


def test_stalled_copies_of_many_sequences():
    lens = [1 + (37 * b * b) % 150 for b in range(40)]
    p = problem(lens, 2, 8, 128, 128, 22)
    out, s = prompt(*p, lens, errors=1, flags=sk.SGEMM_FLAG_TEST_STALL)
    assert torch.isnan(out).all() and torch.isnan(s[p[5]]).all()
    compare(lens, 2, 8, seed=22)


def test_chained_launches():
    """Calls and GEMMs one behind the other, each allowed to start while the one before runs: as without that."""
    lens = [400, 30, 700]
    q, k, v, g, state, slots = (t.to(DEV) for t in problem(lens, 2, 4, 128, 128, 31))
    cu = torch.tensor([0, 400, 430, 1130], dtype=torch.int32, device=DEV)
    w = torch.randn((1024, 512), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    work = torch.empty(sk.sgemm_linear_attention_workspace(1130, 3, 4, 128, 128), dtype=torch.uint8, device=DEV)

    def chain(flags):
        s, out, y = state.clone(), torch.zeros_like(v), torch.zeros((8, 1024), dtype=torch.bfloat16, device=DEV)
        token = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        for _ in range(20):
            sk.sgemm_bf16_linear_attention(q, k, v, g, s, slots, cu, 0.1, out=out, workspace=work, flags=flags)
            sk.sgemm_bf16_skinny_ex(out.view(-1, 512)[:8], w, y, flags=flags)
            sk.sgemm_bf16_linear_step(q[:3], k[:3], v[:3], g[:3], s, slots, 0.1, out=token, flags=flags)
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0
        return s, out, y, token

    for a, b in zip(chain(0), chain(sk.SGEMM_FLAG_PDL)):
        assert torch.equal(a, b)
