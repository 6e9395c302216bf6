"""GPU: prompts that are cut into parts, whose states the first two kernels make: what test_gpu_linear.py holds of
prompts in general, at lengths that are cut whatever the rule on their costs, and the states' accuracy.

That a call has cut something is seen in its scratch, where the parts' states lie behind 3 KB of other things."""
from __future__ import annotations

import pytest
import torch

import bf16_skinny_gemm_gb300 as sk
import decode_oracle as D
import layers_tight as R
from test_gpu_linear import expect, problem, strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")
RAGGED = [3000, 5, 1500, 64, 700]


def scratch(p):
    q, v, slots = p[0], p[2], p[5]
    n = sk.sgemm_linear_attention_workspace(v.shape[0], len(slots), v.shape[1], q.shape[2], v.shape[2])
    return torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)


def cut(work):
    return bool((work[4096:] != 0x5A).any())


def prompt(p, lens, scale=1.0, fresh=None, errors=0, out=None, flags=0):
    q, k, v, g, state, slots = p
    s, work = state.to(DEV), scratch(p)
    cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    out = sk.sgemm_bf16_linear_attention(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), s, slots.to(DEV), cu, scale,
                                         fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.int32, device=DEV),
                                         out=out, workspace=work, flags=flags)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == errors
    assert cut(work)
    return out, s


def compare(p, lens, scale=1.0, fresh=None, **kw):
    out, s = prompt(p, lens, scale, fresh, **kw)
    want, last, ob, sb = expect(*p, lens, scale, True, fresh)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")
    return out, s, want, last


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("lens", [[1000], [2000, 2000], RAGGED], ids=["one", "alike", "ragged"])
def test_widths(Dk, Dv, lens):
    """With the errors over many elements: of the outputs, and of the states."""
    p = problem(lens, 2, 4, Dk, Dv, len(lens) + Dk + Dv)
    out, s, want, last = compare(p, lens, 0.3, [b % 2 for b in range(len(lens))])
    assert R.rms(out, want) <= R.OUTPUTS
    for b, slot in enumerate(p[5]):
        assert R.rms(s[slot], last[slot]) <= R.STATES, b


@pytest.mark.parametrize("lens,Hk,Hv", [([63], 2, 2), ([64], 2, 2), ([300], 4, 4), ([500, 130], 2, 8), ([200] * 40, 4, 8)])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64)])
def test_states_of_whole_prompts(lens, Hk, Hv, Dk, Dv):
    """The same of prompts that are not cut."""
    p = problem(lens, Hk, Hv, Dk, Dv, sum(lens))
    s = p[4].to(DEV)
    cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    work = scratch(p)
    out = sk.sgemm_bf16_linear_attention(*(t.to(DEV) for t in p[:4]), s, p[5].to(DEV), cu, workspace=work)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0 and not cut(work)
    want, last, _, _ = expect(*p, lens, 1.0, True)
    assert R.rms(out, want) <= R.OUTPUTS
    assert R.rms(s[p[5]], last[p[5]]) <= R.STATES


def test_states_of_a_long_prompt():
    p = problem([9000], 1, 2, 128, 128, 1)
    _, s, _, last = compare(p, [9000])
    assert R.rms(s[p[5]], last[p[5]]) <= R.STATES


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 8), (5, 5), (4, 16)])
def test_heads(Hk, Hv):
    p = problem([1500, 900], Hk, Hv, 64, 64, Hk * 10 + Hv)
    compare(p, [1500, 900])


def test_strided():
    lens = [1500, 700]
    n = sum(lens)
    p = problem(lens, 3, 6, 128, 64, 10)
    q, k, v, g, states, out = strided(*p[:5])
    o = out.transpose(0, 1)[:n, :, :64]
    cu = torch.tensor([0, 1500, n], dtype=torch.int32, device=DEV)
    work = scratch(p)
    sk.sgemm_bf16_linear_attention(q, k, v, g, states[:, :, :128], p[5].to(DEV), cu, 1.5, out=o, workspace=work)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0 and cut(work)
    want, last, ob, sb = expect(*p, lens, 1.5, True)
    D.check(o, want, ob, "out")
    D.check(states[:, :, :128], last, sb + 1e-300, "state")
    assert torch.all(states[:, :, 128] == 5) and torch.all(out[:, n] == 9) and torch.all(out[:, :, 64:] == 9)


def test_rows_of_out_that_start_on_four_bytes():
    p = problem([1000], 2, 2, 128, 128, 15)
    wide = torch.full((1000, 2, 134), 9.0, dtype=torch.bfloat16, device=DEV)
    out, s = prompt(p, [1000], out=wide[:, :, 2:130])
    dense, t = prompt(p, [1000])
    assert torch.equal(out, dense) and torch.equal(s, t)
    assert torch.all(wide[:, :, :2] == 9) and torch.all(wide[:, :, 130:] == 9)


def test_one_decay_a_head_for_all_tokens():
    q, k, v, _, state, slots = problem([1200], 4, 4, 128, 128, 5)
    g = -torch.tensor([0.5, 0.25, 0.125, 0.0625])
    s, cu = state.to(DEV), torch.tensor([0, 1200], dtype=torch.int32, device=DEV)
    work = scratch((q, k, v, g, state, slots))
    out = sk.sgemm_bf16_linear_attention(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV).expand(1200, 4), s, slots.to(DEV), cu, workspace=work)
    torch.cuda.synchronize()
    assert sk.sgemm_device_errors() == 0 and cut(work)
    want, last, ob, sb = expect(q, k, v, g.expand(1200, 4), state, slots, [1200], 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_decays():
    """Fast and slow ones, none, all, and what passes single precision's range."""
    p = problem([1600], 1, 6, 128, 128, 4)
    g = p[3]
    g[:, 0] = 0.0
    g[:, 1] = -100.0
    g[::37, 2] = -INF
    g[:, 3] = -1e-6
    g[:, 4] = -3e38
    g[600:700, 5] = 0.01
    compare(p, [1600])


def test_slots():
    """No slot: from zeros and not kept; fresh: from zeros whatever the slot holds; a slot past the pool."""
    lens = [1500, 1200, 900, 64]
    p = problem(lens, 2, 4, 128, 128, 5)
    p[5][1] = -1
    p[4][p[5][2]] = NAN
    out, s = prompt(p, lens, fresh=[0, 0, 1, 0])
    clean = list(p)
    clean[4] = p[4].clone()
    clean[4][p[5][2]] = 0
    want, last, ob, sb = expect(*clean, lens, 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")
    bad = list(clean)
    bad[5] = p[5].clone()
    bad[5][0] = 99
    out, s = prompt(bad, lens, errors=2)
    want, last, ob, sb = expect(*bad, lens, 1.0, True)
    D.check(out, want, ob, "out")
    D.check(s, last, sb + 1e-300, "state")


def test_a_neighbour_of_nan_reaches_no_other_sequence():
    lens = [1000, 777, 1400]
    p = problem(lens, 2, 4, 128, 128, 9)
    clean, cs = prompt(p, lens)
    for t in p[:4]:
        t[1000:1777] = NAN
    out, s = prompt(p, lens)
    rows = [*range(1000), *range(1777, sum(lens))]
    assert torch.equal(out[rows], clean[rows]) and torch.equal(s[p[5][[0, 2]]], cs[p[5][[0, 2]]])


def test_what_is_not_finite_reaches_later_tokens_only():
    """In q its token, in k and g its head from its token on (of the states, k the element's row), in v its
    element from its token on."""
    n = 1600
    p = problem([n], 4, 4, 128, 128, 14)
    clean, _ = prompt(p, [n])
    q, k, v, g = p[:4]
    q[100, 0] = NAN
    k[650, 1, 7] = INF
    v[277, 2, 5], v[800, 2, 100], v[801, 2, 100], v[1333, 2, 64] = NAN, -INF, NAN, INF
    g[1190, 3] = NAN
    out, s = prompt(p, [n])
    hit = torch.zeros((n, 4, 128), dtype=torch.bool)
    hit[100, 0] = True
    hit[650:, 1] = True
    hit[277:, 2, 5], hit[800:, 2, 100], hit[1333:, 2, 64] = True, True, True
    hit[1190:, 3] = True
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])
    assert not torch.isfinite(out.cpu()[hit]).any()
    last = s[p[5][0]].cpu()
    assert torch.isfinite(last[0]).all() and not torch.isfinite(last[3]).any()
    assert not torch.isfinite(last[1][7]).any()  # a key element's row of the state
    assert torch.isfinite(last[1][torch.arange(128) != 7]).all()
    gone = torch.zeros(128, dtype=torch.bool)
    gone[[5, 64, 100]] = True
    assert not torch.isfinite(last[2][:, gone]).any() and torch.isfinite(last[2][:, ~gone]).all()


def test_a_prompt_in_parts_and_then_tokens():
    n, at = 2203, 2200
    p = problem([n], 2, 4, 128, 128, 11)
    q, k, v, g, state, slots = [t.to(DEV) for t in p]
    outs = []
    for a, b in ((0, 1077), (1077, at)):
        outs.append(sk.sgemm_bf16_linear_attention(q[a:b], k[a:b], v[a:b], g[a:b], state, slots,
                                                   torch.tensor([0, b - a], dtype=torch.int32, device=DEV)))
    for t in range(at, n):
        r = slice(t, t + 1)
        outs.append(sk.sgemm_bf16_linear_step(q[r], k[r], v[r], g[r], state, slots))
    torch.cuda.synchronize()
    want, last, ob, sb = expect(*p, [n], 1.0, True)
    D.check(torch.cat(outs), want, ob, "out")
    D.check(state, last, sb + 1e-300, "state")


def test_captured():
    """One graph, offsets that change: cut in other places, and not at all."""
    n = 4000
    p = problem([1000, 3000], 2, 2, 128, 128, 12)
    d = [t.to(DEV) for t in p]
    cu = torch.tensor([0, 1000, n], dtype=torch.int32, device=DEV)
    out, work = torch.empty_like(d[2]), scratch(p)

    def call():
        sk.sgemm_bf16_linear_attention(*d, cu, out=out, workspace=work, flags=sk.SGEMM_FLAG_PDL)

    call()
    torch.cuda.synchronize()
    assert cut(work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1000, 3000], [2500, 1500], [0, n], [100, 300]):
        cu.copy_(torch.tensor([0, lens[0], sum(lens)]))
        d[4].copy_(p[4])
        graph.replay()
        torch.cuda.synchronize()
        r = slice(0, sum(lens))
        want, last, ob, sb = expect(*(t[r] for t in p[:4]), *p[4:], lens, 1.0, True)
        D.check(out[r], want, ob, "out")
        D.check(d[4], last, sb + 1e-300, "state")
    assert sk.sgemm_device_errors() == 0


def test_two_streams_at_once():
    """Each with scratch of its own, and calls that overlap: as one after the other."""
    lens = [1800, 600]
    problems = [[t.to(DEV) for t in problem(lens, 2, 4, 128, 128, seed)] for seed in (1, 2)]
    cu = torch.tensor([0, 1800, 2400], dtype=torch.int32, device=DEV)

    def calls(streams):
        got = []
        for p in problems:
            got.append(([t.clone() if i == 4 else t for i, t in enumerate(p)], torch.empty_like(p[2]), scratch(p)))
        torch.cuda.synchronize()
        for _ in range(20):
            for (p, out, work), stream in zip(got, streams):
                sk.sgemm_bf16_linear_attention(*p, cu, 0.5, out=out, workspace=work, stream=stream)
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0 and all(cut(work) for _, _, work in got)
        return [t for p, out, _ in got for t in (p[4], out)]

    main = torch.cuda.current_stream()
    for a, b in zip(calls([main, main]), calls([torch.cuda.Stream(), torch.cuda.Stream()])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[2000, 30, 1700], [1500]])
def test_chained_launches(lens):
    """Calls and GEMMs one behind the other, each allowed to start while the one before runs: as without that."""
    p = problem(lens, 2, 4, 128, 128, 31)
    n, B = sum(lens), len(lens)
    q, k, v, g, state, slots = (t.to(DEV) for t in p)
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    w = torch.randn((1024, 512), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    work = scratch(p)

    def chain(flags):
        s, out, y = state.clone(), torch.zeros_like(v), torch.zeros((8, 1024), dtype=torch.bfloat16, device=DEV)
        token = torch.zeros((B, 4, 128), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        for _ in range(20):
            sk.sgemm_bf16_linear_attention(q, k, v, g, s, slots, cu, 0.1, out=out, workspace=work, flags=flags)
            sk.sgemm_bf16_skinny_ex(out.view(-1, 512)[:8], w, y, flags=flags)
            sk.sgemm_bf16_linear_step(q[:B], k[:B], v[:B], g[:B], s, slots, 0.1, out=token, flags=flags)
        torch.cuda.synchronize()
        assert sk.sgemm_device_errors() == 0 and cut(work)
        return s, out, y, token

    for a, b in zip(chain(0), chain(sk.SGEMM_FLAG_PDL)):
        assert torch.equal(a, b)


def test_stalled_copies_end_in_nan_and_an_error():
    lens = [1500, 900]
    p = problem(lens, 2, 2, 128, 128, 13)
    out, s = prompt(p, lens, errors=1, flags=sk.SGEMM_FLAG_TEST_STALL)
    assert torch.isnan(out).all() and torch.isnan(s[p[5]]).all()
    compare(p, lens)
