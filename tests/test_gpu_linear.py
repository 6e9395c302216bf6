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
