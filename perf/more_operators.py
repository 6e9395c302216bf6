"""Cases for the operators that make whole layers of a decode or verification step: a mixture of
experts for a few tokens (router and experts), latent attention for a tree of drafted tokens, and
linear attention with a decay for each head (chunks of a prompt, and single tokens).

``run`` computes them in plain torch (FP32, rounded once at the end), or, where ``own`` is set,
with this package's kernels.  ``exact`` computes them in FP64 from their definitions.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # two sequences' tokens through a small model's experts: latency
        {"name": "moe_small", "op": "moe", "T": 2, "E": 16, "k": 2, "D": 1024, "F": 512, "score": "softmax", "bias": False},
        # one decode token: eight experts of a wide layer
        {"name": "moe_token", "op": "moe", "T": 1, "E": 128, "k": 8, "D": 4096, "F": 1024, "score": "softmax", "bias": False},
        # verification of eight drafted tokens; selection bias, an expert width that is no power of two
        {"name": "moe_verify", "op": "moe", "T": 8, "E": 64, "k": 6, "D": 2048, "F": 1408, "score": "sigmoid", "bias": True},
        # a serving batch: nearly every expert has tokens
        {"name": "moe_batch", "op": "moe", "T": 64, "E": 128, "k": 8, "D": 4096, "F": 1024, "score": "softmax", "bias": False},
        # one sequence's small tree of drafts over a short context: latency
        {"name": "tree_token", "op": "tree", "B": 1, "n": 12, "H": 32, "len": 1000, "R": 512, "E": 64, "page": 64, "ragged": False},
        # a batch of trees of 1 to 24 tokens, an odd head count, pages that end inside a tile
        {"name": "tree_batch", "op": "tree", "B": 8, "n": 24, "H": 20, "len": 4099, "R": 512, "E": 64, "page": 16, "ragged": True},
        # full trees of 64 drafts over long contexts
        {"name": "tree_wide", "op": "tree", "B": 2, "n": 64, "H": 64, "len": 16384, "R": 512, "E": 64, "page": 64, "ragged": False},
        # one decode token: latency
        {"name": "step_token", "op": "step", "B": 1, "Hk": 32, "Hv": 32, "Dk": 128, "Dv": 128, "pad": 0},
        # a padded serving batch, two value heads a key head
        {"name": "step_batch", "op": "step", "B": 128, "Hk": 16, "Hv": 32, "Dk": 128, "Dv": 128, "pad": 9},
        # a short prompt, no multiple of any chunk
        {"name": "prompt_short", "op": "prompt", "B": 1, "Hk": 16, "Hv": 16, "Dk": 128, "Dv": 128, "len": 500, "ragged": False},
        # ragged prompts in one call, some of them going on from a state, narrow keys
        {"name": "prompt_ragged", "op": "prompt", "B": 8, "Hk": 8, "Hv": 32, "Dk": 64, "Dv": 128, "len": 2049, "ragged": True},
        # a long prompt's chunk
        {"name": "prompt_long", "op": "prompt", "B": 1, "Hk": 32, "Hv": 32, "Dk": 128, "Dv": 128, "len": 16384, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["moe", "moe", "tree", "step", "prompt"])
    if op == "moe":
        E = rng.choice([8, 16, 32, 64, 96, 128, 160, 256])
        k = rng.randint(1, 8)
        D = max(512, _log_int(rng, 512, 8192) // 8 * 8)
        # at most the weights of the largest listed case
        F = max(64, _log_int(rng, 64, max(64, min(4096, 128 * 1024 * 4096 // (E * D)))) // 8 * 8)
        return {"op": "moe", "T": _log_int(rng, 1, 64), "E": E, "k": k, "D": D, "F": F, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5}
    if op == "tree":
        B, n, H = _log_int(rng, 1, 32), _log_int(rng, 1, 64), _log_int(rng, 8, 128)
        # at most the largest listed case's keys x rows
        most = min(65536, max(1, 2 * 64 * 64 * 16384 // (B * n * H)), 262144 // B)
        return {"op": "tree", "B": B, "n": n, "H": H, "len": max(n, _log_int(rng, 1, most)) if rng.random() < 0.9 else n,
                "R": rng.choice([512, 512, 384, 256, 128]), "E": rng.choice([64, 64, 32]), "page": rng.choice([16, 32, 64, 128]),
                "ragged": rng.random() < 0.6}
    Hk = rng.choice([1, 2, 4, 8, 16, 20, 32])
    Hv = Hk * rng.choice([1, 1, 2, 4]) if Hk <= 8 else Hk
    heads = {"Hk": Hk, "Hv": Hv, "Dk": rng.choice([64, 128, 128]), "Dv": rng.choice([64, 128, 128])}
    if op == "step":
        return {"op": "step", "B": _log_int(rng, 1, 128), **heads, "pad": rng.choice([0, 0, 5])}
    B = _log_int(rng, 1, 32)
    return {"op": "prompt", "B": B, **heads, "len": _log_int(rng, 1, 16384 // B), "ragged": rng.random() < 0.6}


# ------------------------------------------------------------------------------------ the inputs
def _lengths(case):
    """Lengths of a case's sequences (of the case alone, so that its work is known)."""
    B, L = case["B"], case["len"]
    if not case["ragged"]:
        return [L] * B
    lens = [max(1, round(L * (0.25 + 0.75 * ((0.7548776662 * (b + 1)) % 1.0)))) for b in range(B)]
    lens[0] = L
    return lens


def _trees(case):
    """Cached rows and drafted tokens of each sequence."""
    lens = _lengths(case)
    n = [case["n"]] * case["B"]
    if case["ragged"]:
        n = [1 + int(((0.6180339887 * (b + 1)) % 1.0) * case["n"]) for b in range(case["B"])]
    return [max(a, b) for a, b in zip(lens, n)], n


def _parents(count, seed):
    """A tree of drafted tokens: a chain of likely ones whose nodes have other children."""
    state, parents = seed * 2654435761 % 2**32, [-1]
    for i in range(1, count):
        state = (state * 1664525 + 1013904223) % 2**32
        parents.append(i - 1 if state / 2**32 < 0.4 else (state >> 8) % i)
    return parents


def _bf16(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(torch.bfloat16)


def _weight(gen, *shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in out:
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * shape[-1] ** -0.5)
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "moe":
        T, E, k, D, F = case["T"], case["E"], case["k"], case["D"], case["F"]
        s["x"] = _bf16(gen, T, D)
        s["w_router"] = (torch.randn((E, D), generator=gen, device=DEV) * D**-0.5).to(torch.bfloat16)
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None
        s["w_gate_up"], s["w_down"] = _weight(gen, E, 2 * F, D), _weight(gen, E, D, F)
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["y"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
        if own:
            import bf16_skinny_gemm_gb300 as sk
            # scratch between the two products; a decode loop keeps one for all layers
            s["workspace"] = torch.empty(sk.sgemm_moe_experts_workspace(T, E, k, D, F), dtype=torch.uint8, device=DEV)
        return s
    if case["op"] == "tree":
        R, E, page, H, B = case["R"], case["E"], case["page"], case["H"], case["B"]
        lens, ns = _trees(case)
        need = [-(-m // page) for m in lens]
        order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros((B, max(need)), dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            table[b, : need[b]] = order[at : at + need[b]]
            at += need[b]
        s["cache"] = torch.empty((at, page, R + E), dtype=torch.bfloat16, device=DEV)
        for i in range(0, at, 1 << 14):
            s["cache"][i : i + (1 << 14)] = torch.randn(s["cache"][i : i + (1 << 14)].shape, generator=gen, device=DEV)
        s["q"] = _bf16(gen, sum(ns), H, R + E)
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu_q"] = torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
        masks = []
        for b in range(B):
            rows = []
            for i, parent in enumerate(_parents(ns[b], seed + b)):
                rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
            masks += [m - (1 << 64) if m >> 63 else m for m in rows]
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device=DEV)[:, None]
        s["scale"], s["max_q"] = (128 + E) ** -0.5, max(ns)
        # each drafted token's sequence and place in it, for the plain form
        s["seq"] = torch.tensor([b for b in range(B) for _ in range(ns[b])], device=DEV)
        s["place"] = torch.tensor([i for b in range(B) for i in range(ns[b])], device=DEV)
        s["out"] = torch.empty((sum(ns), H, R), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((sum(ns), H), dtype=torch.float32, device=DEV)
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        return s
    B, Hk, Hv, Dk, Dv = case["B"], case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    lens = [1] * B if case["op"] == "step" else _lengths(case)
    N = sum(lens)
    # queries, keys and values as one projection's output, the keys of unit length
    qkv = torch.randn((N, 2 * Hk * Dk + Hv * Dv), generator=gen, device=DEV)
    qkv[:, : 2 * Hk * Dk] *= Dk**-0.5
    qkv = qkv.to(torch.bfloat16)
    s["q"], s["k"], s["v"] = (a.unflatten(1, h) for a, h in zip(
        qkv.split([Hk * Dk, Hk * Dk, Hv * Dv], 1), ((Hk, Dk), (Hk, Dk), (Hv, Dv))))
    # logarithms of the decays: memories of one to a thousand tokens
    s["g"] = -torch.exp(torch.rand((N, Hv), generator=gen, device=DEV) * math.log(1000.0) - math.log(1000.0))
    # slot 0 is kept out of use
    s["state"] = torch.randn((B + 1, Hv, Dk, Dv), generator=gen, device=DEV) * 0.1
    s["slots"] = 1 + torch.randperm(B, generator=gen, device=DEV)
    s["scale"] = 1.0
    s["out"] = torch.zeros((N, Hv, Dv), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "step":
        if case["pad"]:
            s["slots"][:: case["pad"]] = -1
        return s
    cu = [sum(lens[:b]) for b in range(B + 1)]
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s["fresh"] = (torch.arange(B, device=DEV) % 2 == 0).to(torch.int32)  # every other prompt goes on from its state
    # each row's place in a batch of padded sequences, for the plain form
    s["longest"] = max(lens)
    s["at"] = torch.cat([torch.arange(m, device=DEV) + b * s["longest"] for b, m in enumerate(lens)])
    if own:
        import bf16_skinny_gemm_gb300 as sk
        s["workspace"] = torch.empty(sk.sgemm_linear_attention_workspace(N, B, Hv, Dk, Dv), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------- the passes
def run(s):
    return {"moe": _moe, "tree": _tree, "step": _step, "prompt": _prompt}[s["case"]["op"]](s)


def _moe(s):
    case = s["case"]
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_moe_route(s["x"], s["w_router"], case["k"], s["bias"], case["score"], ids=s["ids"], weights=s["weights"])
        sk.sgemm_bf16_moe_experts(s["x"], s["w_gate_up"], s["w_down"], s["ids"], s["weights"], y=s["y"], workspace=s["workspace"])
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    T, E, k, F = case["T"], case["E"], case["k"], case["F"]
    logits = s["x"].double() @ s["w_router"].double().T
    if case["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    key = score if s["bias"] is None else score + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    weights = score.gather(1, ids)
    weights = (weights / weights.sum(1, keepdim=True)).float()
    x = s["x"].float()
    y = torch.zeros_like(x)

    def expert(xs, gate_up, down):
        a = xs @ gate_up.float().transpose(-1, -2)
        gate, up = a[..., :F], a[..., F:]
        return (gate / (1.0 + torch.exp(-gate)) * up) @ down.float().transpose(-1, -2)

    if T * k < E:
        for t in range(T):
            for j in range(k):
                e = ids[t, j : j + 1]
                y[t] += weights[t, j] * expert(x[t : t + 1], s["w_gate_up"].index_select(0, e)[0], s["w_down"].index_select(0, e)[0])[0]
    else:
        for e in range(E):
            w = (weights * (ids == e)).sum(1, keepdim=True)
            y += w * expert(x, s["w_gate_up"][e], s["w_down"][e])
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": weights}


def _tree(s):
    case = s["case"]
    R, H, B, Q = case["R"], case["H"], case["B"], s["max_q"]
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_latent_tree_attention(s["q"], s["cache"], s["table"], s["lens"], R, s["scale"], s["tree"], cu_q=s["cu_q"],
                                            max_q=Q, out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    keys = s["cache"][s["table"].long()].flatten(1, 2).float()  # [B, padded length, R + E]
    cu = s["cu_q"].long()
    at = (cu[:-1, None] + torch.arange(Q, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    scores = s["q"][at].flatten(1, 2).float() @ keys.transpose(1, 2) * s["scale"]
    scores = scores.view(B, Q, H, -1)
    # rows before the drafted tokens' are seen by all of them, a drafted token's where its bit is set
    before = (s["lens"] - (cu[1:] - cu[:-1]))[:, None, None]
    row = torch.arange(keys.shape[1], device=DEV)
    draft = row - before  # [B, 1, padded length]
    bit = (s["tree"][at, 0][..., None] >> draft.clamp(0, 63)) & 1
    sees = (draft < 0) | ((bit == 1) & (row < s["lens"][:, None, None]))
    scores.masked_fill_(~sees[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(1, 2) @ keys[..., :R]).view(B, Q, H, R) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    return {"out": out[s["seq"], s["place"]].to(torch.bfloat16), "lse": lse[s["seq"], s["place"]]}


def _step(s):
    case = s["case"]
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_linear_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"], s["scale"], out=s["out"])
        return {"out": s["out"], "state": s["state"]}
    r = case["Hv"] // case["Hk"]
    q, k = (a.float().repeat_interleave(r, 1) for a in (s["q"], s["k"]))
    keep = (s["slots"] >= 0)[:, None, None]
    at = s["slots"].clamp(min=0)  # a padded sequence rewrites the slot out of use
    old = s["state"][at]
    new = old * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    s["state"][at] = torch.where(keep[..., None], new, old)
    out = (q[..., None] * new).sum(2) * s["scale"]
    return {"out": torch.where(keep, out, torch.zeros_like(out)).to(torch.bfloat16), "state": s["state"]}


def _prompt(s):
    case = s["case"]
    B, Hk, Hv, Dk, Dv, L = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv", "len"))
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_linear_attention(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"], s["cu"], s["scale"],
                                       fresh=s["fresh"], out=s["out"], workspace=s["workspace"])
        return {"out": s["out"], "state": s["state"]}
    L, C = s["longest"], 128
    full = -(-L // C) * C

    def padded(x, width):  # [B, heads, padded length, width]; padded tokens add nothing and decay nothing
        flat = torch.zeros((B * L, *x.shape[1:]), device=DEV)
        flat[s["at"]] = x.float()
        flat = torch.nn.functional.pad(flat.view(B, L, -1, width), (0, 0, 0, 0, 0, full - L))
        return flat.repeat_interleave(Hv // flat.shape[2], 2).transpose(1, 2)

    q, k, v = padded(s["q"], Dk), padded(s["k"], Dk), padded(s["v"], Dv)
    g = padded(s["g"][..., None], 1)[..., 0].double()
    state = torch.where(s["fresh"].bool()[:, None, None, None], torch.zeros((), device=DEV), s["state"][s["slots"]])
    out = torch.empty_like(v)
    hidden = torch.ones((C, C), dtype=torch.bool, device=DEV).triu(1)
    for i in range(0, full, C):
        qc, kc, vc = q[:, :, i : i + C], k[:, :, i : i + C], v[:, :, i : i + C]
        sums = g[:, :, i : i + C].cumsum(-1)
        decay = torch.exp((sums[..., :, None] - sums[..., None, :]).masked_fill(hidden, -math.inf)).float()
        out[:, :, i : i + C] = (qc @ kc.transpose(-1, -2) * decay) @ vc + torch.exp(sums).float()[..., None] * (qc @ state)
        left = torch.exp(sums[..., -1:] - sums).float()[..., None]
        state = torch.exp(sums[..., -1]).float()[..., None, None] * state + (kc * left).transpose(-1, -2) @ vc
    s["state"][s["slots"]] = state
    out = out.transpose(1, 2)[:, :L].reshape(B * L, Hv, Dv)[s["at"]] * s["scale"]
    return {"out": out.to(torch.bfloat16), "state": s["state"]}


# ----------------------------------------------------------------------------------- their work
def work(case):
    if case["op"] == "moe":
        T, E, k, D, F = case["T"], case["E"], case["k"], case["D"], case["F"]
        # experts that have tokens, as many as independent choices leave
        active = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(2 * E * D + 6 * active * F * D + 4 * T * D + 8 * T * k), "flops": 2 * T * (E * D + 3 * k * F * D)}
    if case["op"] == "tree":
        R, E, H = case["R"], case["E"], case["H"]
        lens, ns = _trees(case)
        rows = sum(ns) * H
        seen = sum(n * (m - n) + n * (n + 1) // 2 for m, n in zip(lens, ns))
        return {"bytes": sum(lens) * (R + E) * 2 + rows * ((R + E) * 2 + R * 2 + 4) + 4 * sum(-(-m // case["page"]) for m in lens)
                + 8 * sum(ns), "flops": 2 * seen * H * (2 * R + E)}
    B, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
    N = sum([1] * B if case["op"] == "step" else _lengths(case))
    kept, read = B, B
    if case["op"] == "step":
        kept = read = B - (-(-B // case["pad"]) if case["pad"] else 0)
    else:
        read = B // 2
    return {"bytes": 4 * N * Hk * Dk + 4 * N * Hv * Dv + 4 * N * Hv + 4 * (read + kept) * Hv * Dk * Dv,
            "flops": 4 * (kept if case["op"] == "step" else N) * Hv * Dk * Dv}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        T, k, F = case["T"], case["k"], case["F"]
        x = s["x"].double()
        logits = torch.stack([(s["w_router"].double() * row).sum(1) for row in x])
        score = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
        rank = (score if s["bias"] is None else score + s["bias"].double()).tolist()
        ids = [sorted(range(case["E"]), key=lambda e: (-row[e], e))[:k] for row in rank]
        chosen = torch.tensor(ids, device=DEV)
        weights = torch.stack([score[t, chosen[t]] / score[t, chosen[t]].sum() for t in range(T)])
        y = torch.zeros_like(x)
        for e in sorted({e for row in ids for e in row}):
            tokens = [t for t in range(T) if e in ids[t]]
            a = x[tokens] @ s["w_gate_up"][e].double().T
            h = torch.nn.functional.silu(a[:, :F]) * a[:, F:]
            w = torch.stack([weights[t, ids[t].index(e)] for t in tokens])
            y[tokens] += w[:, None] * (h @ s["w_down"][e].double().T)
        return {"y": y, "ids": chosen.to(torch.int32), "weights": weights}
    if case["op"] == "tree":
        R, E, H = case["R"], case["E"], case["H"]
        lens, ns = _trees(case)
        out = torch.zeros((sum(ns), H, R), dtype=torch.float64, device=DEV)
        lse = torch.full((sum(ns), H), -math.inf, dtype=torch.float64, device=DEV)
        t = 0
        for b, (m, n) in enumerate(zip(lens, ns)):
            pages = s["table"][b, : -(-m // case["page"])].long()
            keys = s["cache"][pages].reshape(-1, R + E)[:m].double()
            parents = _parents(n, seed + b)
            for i in range(n):
                path, at = [], i
                while at >= 0:
                    path.append(m - n + at)
                    at = parents[at]
                sees = torch.cat([torch.arange(m - n, device=DEV), torch.tensor(path[::-1], device=DEV)])
                mine = keys[sees]
                score = (s["q"][t].double() @ mine.T) * s["scale"]
                lse[t] = torch.logsumexp(score, 1)
                out[t] = torch.exp(score - lse[t][:, None]) @ mine[:, :R]
                t += 1
        return {"out": out, "lse": lse}
    B, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
    lens = [1] * B if case["op"] == "step" else _lengths(case)
    if max(lens) > 20000:
        return None
    state = s["state"].double()
    out = torch.zeros((sum(lens), Hv, Dv), dtype=torch.float64, device=DEV)
    head = torch.arange(Hv, device=DEV) // (Hv // Hk)
    slots, first = s["slots"].tolist(), [sum(lens[:b]) for b in range(B)]
    fresh = s["fresh"].tolist() if "fresh" in s else [0] * B
    # token by token, all sequences that have one at a time
    live = [b for b in range(B) if slots[b] >= 0]
    now = torch.stack([torch.zeros_like(state[0]) if fresh[b] else state[slots[b]] for b in live]) if live else None
    for i in range(max(lens)):
        on = [j for j, b in enumerate(live) if lens[b] > i]
        if not on:
            break
        rows = torch.tensor([first[live[j]] + i for j in on], device=DEV)
        q, k, v = s["q"][rows].double()[:, head], s["k"][rows].double()[:, head], s["v"][rows].double()
        part = now if len(on) == len(live) else now[on]
        part = torch.exp(s["g"][rows].double())[..., None, None] * part + k[..., :, None] * v[..., None, :]
        out[rows] = s["scale"] * torch.einsum("bhk,bhkv->bhv", q, part)
        if len(on) == len(live):
            now = part
        else:
            now[on] = part
    for j, b in enumerate(live):
        state[slots[b]] = now[j]
    return {"out": out, "state": state}
