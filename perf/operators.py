"""Cases for the operators that stand between a decode step's projections: the residual add with
its RMS norm, the append to a paged latent cache with the position rotation, and the latent
attention (absorbed form) that reads that cache.

``run`` computes them in plain torch (FP32, rounded once at the end), or, where ``own`` is set,
with this package's kernels.  ``exact`` computes them in FP64 from their definitions.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode token's norm before a layer's projections: latency
        {"name": "norm_token", "op": "norm", "T": 1, "D": 4096, "form": "bf16", "add": True},
        # eight tokens of a speculative verification, in 8 bits for a quantised projection
        {"name": "norm_verify_e4m3", "op": "norm", "T": 8, "D": 8192, "form": "e4m3", "group": 128, "add": True},
        # an odd width (no row but the first starts on 16 bytes) and no residual
        {"name": "norm_odd", "op": "norm", "T": 1003, "D": 1537, "form": "bf16", "add": False},
        # a prompt's chunk, one scale a row
        {"name": "norm_prompt_e4m3", "op": "norm", "T": 16384, "D": 4096, "form": "e4m3", "group": 0, "add": True},
        # one decode token into the cache, and the rotation of its 32 query heads: latency
        {"name": "append_token", "op": "append", "T": 1, "H": 32, "R": 512, "E": 64, "page": 64, "inter": True, "norm": True, "pad": 0},
        # a padded batch of ragged sequences, pages of 16, half-split rotation
        {"name": "append_padded", "op": "append", "T": 777, "H": 20, "R": 512, "E": 64, "page": 16, "inter": False, "norm": True, "pad": 5},
        # a prompt's chunk into the cache
        {"name": "append_prompt", "op": "append", "T": 16384, "H": 32, "R": 512, "E": 64, "page": 64, "inter": True, "norm": True, "pad": 0},
        # one sequence, one token, a short context: latency
        {"name": "attn_token", "op": "attn", "B": 1, "q": 1, "H": 32, "len": 1000, "R": 512, "E": 64, "page": 64, "ragged": False},
        # one sequence with a long context: the key axis is all there is to split
        {"name": "attn_long", "op": "attn", "B": 1, "q": 1, "H": 32, "len": 131072, "R": 512, "E": 64, "page": 64, "ragged": False},
        # verification of 1 to 8 drafted tokens, an odd head count, pages that end inside a tile
        {"name": "attn_verify", "op": "attn", "B": 8, "q": 8, "H": 20, "len": 4099, "R": 512, "E": 64, "page": 16, "ragged": True},
        # a serving batch of ragged contexts
        {"name": "attn_batch", "op": "attn", "B": 64, "q": 1, "H": 32, "len": 8192, "R": 512, "E": 64, "page": 64, "ragged": True},
        # all heads of a wide model on one GPU
        {"name": "attn_wide", "op": "attn", "B": 32, "q": 1, "H": 128, "len": 8192, "R": 512, "E": 64, "page": 32, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn"])
    if op == "norm":
        D = _log_int(rng, 64, 8192)
        D = rng.choice([D, max(64, D // 8 * 8), max(64, D // 128 * 128)])
        T = _log_int(rng, 1, min(16384, 16384 * 4096 // D))
        form = rng.choice(["bf16", "e4m3"])
        case = {"op": "norm", "T": T, "D": D, "form": form, "add": rng.random() < 0.75}
        if form == "e4m3":
            case["group"] = rng.choice([0, 128])
        return case
    R, E = rng.choice([512, 512, 512, 384, 256, 128]), rng.choice([64, 64, 32])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = _log_int(rng, 1, 16384)
        return {"op": "append", "T": T, "H": _log_int(rng, 1, 32), "R": R, "E": E, "page": page, "inter": rng.random() < 0.5,
                "norm": rng.random() < 0.75, "pad": rng.choice([0, 0, 7])}
    B, q, H = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 8]), _log_int(rng, 8, 128)
    # at most the largest listed case's keys, and its keys x rows
    most = min(131072, 262144 // B, 32 * 8192 * 128 // (B * q * H))
    return {"op": "attn", "B": B, "q": q, "H": H, "len": _log_int(rng, 1, most), "R": R, "E": E, "page": page,
            "ragged": rng.random() < 0.6}


# ------------------------------------------------------------------------------------ the inputs
def _shape(case):
    """Context lengths and new tokens of an attention case's sequences (of the case alone, so that
    its work is known)."""
    B, L, Q = case["B"], case["len"], case["q"]
    if not case["ragged"]:
        return [L] * B, [Q] * B
    part = [(0.7548776662 * (b + 1)) % 1.0 for b in range(B)]
    lens = [max(1, round(L * (0.25 + 0.75 * p))) for p in part]
    lens[0] = L
    return lens, [1 + int(((0.6180339887 * (b + 1)) % 1.0) * Q) for b in range(B)]


def _bf16(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        # activations of a residual stream: a few columns are much larger than the others
        s["x"] = _bf16(gen, T, D)
        s["residual"] = (_bf16(gen, T, D).float() * (1.0 + 15.0 * (torch.rand(D, generator=gen, device=DEV) < 0.01))).to(torch.bfloat16)
        s["weight"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16)
        s["residual_out"] = torch.empty_like(s["x"])
        if case["form"] == "bf16":
            s["y"] = torch.empty_like(s["x"])
        else:
            groups = -(-D // case["group"]) if case["group"] else 1
            s["y"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV)
            s["scales"] = torch.empty((T, groups), dtype=torch.float32, device=DEV)
        return s
    R, E, page, H = case["R"], case["E"], case["page"], case["H"]
    if case["op"] == "append":
        T = case["T"]
        pages = 1 + -(-T // page) + 8  # page 0 is kept out of use
        s["kv"] = _bf16(gen, T, R + E)
        s["cache"] = _bf16(gen, pages, page, R + E)
        s["slots"] = page + torch.randperm((pages - 1) * page, generator=gen, device=DEV)[:T]
        if case["pad"]:
            s["slots"][:: case["pad"]] = -1
        longest = 32768
        angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, E, 2, device=DEV, dtype=torch.float64) / E))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, longest, (T,), generator=gen, device=DEV)
        s["weight"] = (1.0 + 0.1 * torch.randn(R, generator=gen, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        # the rotated part of each head's query, inside the query projection's output, and its
        # place behind the absorbed part in the attention's query
        s["q"] = _bf16(gen, T, H, 128 + E)[..., 128:]
        s["q_out"] = torch.zeros((T, H, R + E), dtype=torch.bfloat16, device=DEV)[..., R:]
        return s
    lens, qs = _shape(case)
    B, total = case["B"], sum(qs)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
    s["cache"] = torch.empty((at, page, R + E), dtype=torch.bfloat16, device=DEV)
    for i in range(0, at, 1 << 14):
        s["cache"][i : i + (1 << 14)] = torch.randn(s["cache"][i : i + (1 << 14)].shape, generator=gen, device=DEV)
    s["q"] = _bf16(gen, total, H, R + E)
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu_q"] = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    s["scale"], s["max_q"] = (128 + E) ** -0.5, max(qs)
    # each query token's sequence and place in it, for the plain form
    s["seq"] = torch.tensor([b for b in range(B) for _ in range(qs[b])], device=DEV)
    s["place"] = torch.tensor([i for b in range(B) for i in range(qs[b])], device=DEV)
    s["out"] = torch.empty((total, H, R), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((total, H), dtype=torch.float32, device=DEV)
    # scratch for the partial results of split contexts; a decode loop keeps one for all layers
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------- the passes
def run(s):
    return {"norm": _norm, "append": _append, "attn": _attn}[s["case"]["op"]](s)


def _norm(s):
    case = s["case"]
    residual = s["residual"] if case["add"] else None
    if own:
        import bf16_skinny_gemm_gb300 as sk
        kept = s["residual_out"] if case["add"] else None
        if case["form"] == "bf16":
            y, kept = sk.sgemm_bf16_add_rmsnorm(s["x"], s["weight"], residual, EPS, y=s["y"], residual_out=kept)
            return {"y": y, "residual": kept}
        q, scales, kept = sk.sgemm_bf16_add_rmsnorm_e4m3(s["x"], s["weight"], residual, EPS, group=case["group"], q=s["y"],
                                                         scales=s["scales"], residual_out=kept)
        return {"q": q, "scales": scales, "residual": kept}
    h = s["x"].float()
    if residual is not None:
        h = h + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    kept = h.to(torch.bfloat16) if residual is not None else None
    if case["form"] == "bf16":
        return {"y": y.to(torch.bfloat16), "residual": kept}
    T, D = y.shape
    group = case["group"] or D
    parts = torch.nn.functional.pad(y, (0, -D % group)).view(T, -1, group)
    top = parts.abs().amax(-1)
    scales = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (parts / scales[..., None]).view(T, -1)[:, :D].clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"q": q, "scales": scales, "residual": kept}


def _rotate(x, cos, sin, inter):
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    case = s["case"]
    R, E = case["R"], case["E"]
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_latent_append(s["kv"], s["cache"], s["slots"], s["positions"], s["cos_sin"], s["weight"], EPS, q=s["q"],
                                    q_out=s["q_out"], interleaved=case["inter"])
        return {"cache": s["cache"], "q": s["q_out"]}
    kv, table = s["kv"].float(), s["cos_sin"][s["positions"]]
    cos, sin = table[:, : E // 2], table[:, E // 2 :]
    latent = kv[:, :R]
    if case["norm"]:
        latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat([latent, _rotate(kv[:, R:], cos, sin, case["inter"])], 1).to(torch.bfloat16)
    flat = s["cache"].view(-1, R + E)
    keep = s["slots"] >= 0  # a padded token rewrites row 0 of the page out of use
    flat[torch.where(keep, s["slots"], 0)] = torch.where(keep[:, None], row, flat[0])
    s["q_out"].copy_(_rotate(s["q"].float(), cos[:, None], sin[:, None], case["inter"]))
    return {"cache": s["cache"], "q": s["q_out"]}


def _attn(s):
    case = s["case"]
    R, H, B, Q = case["R"], case["H"], case["B"], s["max_q"]
    if own:
        import bf16_skinny_gemm_gb300 as sk
        sk.sgemm_bf16_latent_attention(s["q"], s["cache"], s["table"], s["lens"], R, s["scale"], cu_q=s["cu_q"], max_q=Q,
                                       out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    keys = s["cache"][s["table"].long()].flatten(1, 2).float()  # [B, padded length, R + E]
    cu = s["cu_q"].long()
    at = (cu[:-1, None] + torch.arange(Q, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    scores = s["q"][at].flatten(1, 2).float() @ keys.transpose(1, 2) * s["scale"]
    scores = scores.view(B, Q, H, -1)
    # token i of a sequence's n new ones sees the keys up to its own
    sees = s["lens"][:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(1, Q + 1, device=DEV)
    hidden = torch.arange(keys.shape[1], device=DEV) >= sees[..., None]
    scores.masked_fill_(hidden[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(1, 2) @ keys[..., :R]).view(B, Q, H, R) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    return {"out": out[s["seq"], s["place"]].to(torch.bfloat16), "lse": lse[s["seq"], s["place"]]}


# ----------------------------------------------------------------------------------- their work
def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["D"]
        out = 2 * n if case["form"] == "bf16" else n + 4 * case["T"] * (-(-case["D"] // case["group"]) if case["group"] else 1)
        return {"bytes": 2 * n + (4 * n if case["add"] else 0) + out + 2 * case["D"], "flops": 6 * n}
    R, E, H = case["R"], case["E"], case["H"]
    if case["op"] == "append":
        T, kept = case["T"], case["T"] - (-(-case["T"] // case["pad"]) if case["pad"] else 0)
        rows = 2 * (R + E) * 2 * kept + T * H * E * 2 * 2
        return {"bytes": rows + T * (16 + 4 * E) + (2 * R if case["norm"] else 0), "flops": kept * (4 * R + 3 * E) + 3 * T * H * E}
    lens, qs = _shape(case)
    seen = sum(max(0, n - q + i + 1) for n, q in zip(lens, qs) for i in range(q))
    rows = sum(qs) * H
    return {"bytes": sum(lens) * (R + E) * 2 + rows * ((R + E) * 2 + R * 2 + 4) + 4 * sum(-(-n // case["page"]) for n in lens),
            "flops": 2 * seen * H * (2 * R + E)}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["add"]:
            h += s["residual"].double()
        y = h / torch.sqrt((h * h).sum(1) / case["D"] + EPS)[:, None] * s["weight"].double()
        kept = h if case["add"] else None
        if case["form"] == "bf16":
            return {"y": y, "residual": kept}
        group = case["group"] or case["D"]
        q, scales = [], []
        for part in y.split(group, 1):
            top = part.abs().max(1, keepdim=True).values / E4M3_MAX
            top[top == 0] = 1.0
            scales.append(top)
            q.append(part / top)
        return {"q": torch.cat(q, 1), "scales": torch.cat(scales, 1), "residual": kept}
    R, E, H = case["R"], case["E"], case["H"]
    if case["op"] == "append":
        def turned(x, c, d):
            # a pair as one complex number, turned by its angle
            if case["inter"]:
                z = torch.view_as_complex(x.unflatten(-1, (E // 2, 2)).contiguous())
            else:
                z = torch.complex(x[..., : E // 2].contiguous(), x[..., E // 2 :].contiguous())
            z = z * torch.complex(c, d)
            return torch.view_as_real(z).flatten(-2) if case["inter"] else torch.cat([z.real, z.imag], -1)

        turn = s["cos_sin"].double()[s["positions"]]
        c, d = turn[:, : E // 2].contiguous(), turn[:, E // 2 :].contiguous()
        kv = s["kv"].double()
        if case["norm"]:
            kv[:, :R] *= s["weight"].double() / torch.sqrt((kv[:, :R] ** 2).sum(1, keepdim=True) / R + EPS)
        kv[:, R:] = turned(kv[:, R:], c, d)
        cache = s["cache"].double()
        used = torch.nonzero(s["slots"] >= 0)[:, 0]
        page = case["page"]
        at = s["slots"][used]
        cache[at // page, at % page] = kv[used]
        return {"cache": cache, "q": turned(s["q"].double(), c[:, None], d[:, None])}
    lens, qs = _shape(case)
    out = torch.zeros((sum(qs), H, R), dtype=torch.float64, device=DEV)
    lse = torch.full((sum(qs), H), -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, nq) in enumerate(zip(lens, qs)):
        pages = s["table"][b, : -(-n // case["page"])].long()
        keys = s["cache"][pages].reshape(-1, R + E)[:n].double()
        for i in range(nq):
            m = n - nq + i + 1
            if m > 0:
                score = (s["q"][t].double() @ keys[:m].T) * s["scale"]
                lse[t] = torch.logsumexp(score, 1)
                out[t] = torch.exp(score - lse[t][:, None]) @ keys[:m, :R]
            t += 1
    return {"out": out, "lse": lse}
