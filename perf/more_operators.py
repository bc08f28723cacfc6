"""The other half of a decoder layer, as its users call it: cases, inputs and plain forms.

Kinds of cases:

* ``norm``    the residual stream's addition and RMS norm; with ``fp8`` also the FP8 rows that FP8 experts
  take, read back as the values they stand for
* ``route``   a router's scores to the chosen experts and their weights
* ``experts`` the chosen experts' gated products and their weighted sum, with bf16 or FP8 weights

FP8 rows: value = E4M3 code * 2^k, one k per row and 128 channels. The experts' hidden values are held in
bf16, or with FP8 weights as E4M3 codes with one 2^k per 32 channels.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # Between attention and router, a decode batch of 8: latency alone.
        {"name": "norm_decode_8", "op": "norm", "rows": 8, "width": 4096, "residual": True, "fp8": False},
        # Rows of a width that is no multiple of 16, without a residual (a first norm).
        {"name": "norm_ragged_1021x1000", "op": "norm", "rows": 1021, "width": 1000, "residual": False, "fp8": False},
        # A prefill chunk before FP8 experts: bf16 for the router, FP8 for the experts.
        {"name": "norm_prefill_4096_fp8", "op": "norm", "rows": 4096, "width": 4096, "residual": True, "fp8": True},
        # The router of a decode batch: sigmoid scores, a bias for balance, the best 4 of 8 groups.
        {"name": "route_decode_8", "op": "route", "rows": 8, "experts": 256, "score": "sigmoid", "bias": True, "groups": 8,
         "topk_group": 4, "group_top": 2, "topk": 8, "renorm": True},
        # A prefill chunk through a softmax router without groups.
        {"name": "route_prefill_4096", "op": "route", "rows": 4096, "experts": 128, "score": "softmax", "bias": False, "groups": 1,
         "topk_group": 1, "group_top": 1, "topk": 8, "renorm": True},
        # A long prompt's rows at once (an odd count).
        {"name": "route_long_32749", "op": "route", "rows": 32749, "experts": 256, "score": "sigmoid", "bias": True, "groups": 8,
         "topk_group": 4, "group_top": 2, "topk": 8, "renorm": True},
        # One token: eight experts' weights are read.
        {"name": "experts_1", "op": "experts", "rows": 1, "experts": 64, "topk": 8, "hidden": 4096, "inter": 1024, "fp8": False,
         "skew": 0.3, "pad": 0},
        # A decode batch of 8, few rows share an expert.
        {"name": "experts_8", "op": "experts", "rows": 8, "experts": 128, "topk": 8, "hidden": 4096, "inter": 1024, "fp8": False,
         "skew": 0.3, "pad": 0},
        # A paged decode batch of 64 with FP8 experts.
        {"name": "experts_64_fp8", "op": "experts", "rows": 64, "experts": 128, "topk": 8, "hidden": 4096, "inter": 1024, "fp8": True,
         "skew": 0.3, "pad": 0},
        # An odd chunk with padding rows, uneven experts, another width.
        {"name": "experts_517_fp8", "op": "experts", "rows": 517, "experts": 32, "topk": 6, "hidden": 2048, "inter": 1408, "fp8": True,
         "skew": 0.8, "pad": 21},
        # A prefill chunk of 4,096 rows, bf16 and FP8.
        {"name": "experts_4096", "op": "experts", "rows": 4096, "experts": 64, "topk": 8, "hidden": 4096, "inter": 1024, "fp8": False,
         "skew": 0.3, "pad": 0},
        {"name": "experts_4096_fp8", "op": "experts", "rows": 4096, "experts": 64, "topk": 8, "hidden": 4096, "inter": 1024, "fp8": True,
         "skew": 0.3, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts", "experts"])
    if op == "norm":
        fp8 = rng.random() < 0.5
        width = _log(rng, 2, 64) * 128 if fp8 else _log(rng, 16, 8192)
        return {"op": op, "rows": _log(rng, 1, min(8192, (1 << 24) // width)), "width": width, "residual": rng.random() < 0.7, "fp8": fp8}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = rng.randint(4, 512 // groups)
        topk_group = rng.randint(1, groups)
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": groups * size, "score": rng.choice(["sigmoid", "softmax"]),
                "bias": rng.random() < 0.6, "groups": groups, "topk_group": topk_group, "group_top": rng.choice([1, 2]),
                "topk": rng.randint(1, min(16, topk_group * size)), "renorm": rng.random() < 0.7}
    hidden, inter = rng.choice([512, 1024, 2048, 2560, 4096]), rng.choice([256, 512, 768, 1024, 1408, 2048])
    experts = rng.choice([n for n in (8, 16, 32, 64, 96) if n * hidden * inter <= 1 << 28])
    topk = rng.choice([1, 2, 4, 6, 8])
    rows = _log(rng, 1, min(4096, max(64, (1 << 37) // (topk * hidden * inter))))
    return {"op": op, "rows": rows, "experts": experts, "topk": topk, "hidden": hidden, "inter": inter, "fp8": rng.random() < 0.5,
            "skew": rng.choice([0.0, 0.3, 0.8]), "pad": rng.choice([0, 0, rows // 7])}


# ---- FP8 rows in elementary operations ----------------------------------------------------------


def _encode(x, group):
    """f32 rows [.., n] -> E4M3 values [.., n] and the groups' scales [.., n / group]."""
    a = x.view(*x.shape[:-1], -1, group)
    m, e = torch.frexp(a.abs().amax(-1, keepdim=True))
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)  # the least k with amax <= 448 * 2^k
    k = torch.where(m > 0, k, torch.zeros_like(k))
    codes = torch.ldexp(a, -k).to(torch.float8_e4m3fn)
    return codes.view(x.shape), torch.ldexp(torch.ones_like(m), k).squeeze(-1)


def _decode(codes, scales, group):
    v = codes.float().view(*codes.shape[:-1], -1, group) * scales.unsqueeze(-1)
    return v.view(codes.shape)


# ---- inputs ---------------------------------------------------------------------------------------


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 9241 + 31)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std


def _weights(g, experts, n, width, fp8):
    """Expert weights [experts, n, width] in bf16, or as codes (bytes) and scales."""
    w = torch.empty(experts, n, width, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    s = torch.empty(experts, n, width // 128, device="cuda") if fp8 else None
    step = max(1, (1 << 28) // (n * width))
    for i in range(0, experts, step):
        x = _randn(g, min(step, experts - i), n, width, std=width ** -0.5)
        if fp8:
            c, s[i:i + step] = _encode(x, 128)
            w[i:i + step] = c.view(torch.uint8)
        else:
            w[i:i + step] = x.to(torch.bfloat16)
    return w, s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    rows = case["rows"]
    if case["op"] == "norm":
        # a sublayer's output onto a residual stream with a few channels that stand out
        gain = torch.exp(0.5 * _randn(g, case["width"]))
        s["x"] = (_randn(g, rows, case["width"]) * gain).to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * _randn(g, case["width"])).to(torch.bfloat16)
        s["stream"] = (_randn(g, rows, case["width"], std=3.0) * gain).to(torch.bfloat16) if case["residual"] else None
        s["stream_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        if case["fp8"]:
            s["codes"] = torch.empty(rows, case["width"], dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(rows, case["width"] // 128, device="cuda")
            s["back"] = torch.empty_like(s["x"])
        return s
    if case["op"] == "route":
        n = case["experts"]
        s["logits"] = _randn(g, rows, n)
        # a few experts are out of service for a part of the rows
        s["logits"][: rows // 4, torch.randperm(n, generator=g, device="cuda")[: n // 16]] = -math.inf
        s["balance"] = _randn(g, n, std=0.05) if case["bias"] else None
        s["ids"] = torch.empty(rows, case["topk"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(rows, case["topk"], device="cuda")
        return s
    n, k, hidden, inter = case["experts"], case["topk"], case["hidden"], case["inter"]
    x = _randn(g, rows, hidden).to(torch.bfloat16)
    if case["fp8"]:
        c, s["x_scales"] = _encode(x.float(), 128)
        s["x"] = c.view(torch.uint8)
    else:
        s["x"], s["x_scales"] = x, None
    s["w13"], s["w13_scales"] = _weights(g, n, 2 * inter, hidden, case["fp8"])
    s["w2"], s["w2_scales"] = _weights(g, n, hidden, inter, case["fp8"])
    # distinct experts per row, some more popular than others, ids ascending; padding rows at the end
    gumbel = -torch.log(-torch.log(torch.rand(rows, n, generator=g, device="cuda").clamp(1e-7, 1 - 1e-6)))
    s["ids"] = (_randn(g, n, std=case["skew"]) + gumbel).topk(k, 1).indices.sort(1).values.int()
    s["weights"] = torch.softmax(_randn(g, rows, k), 1)
    if case["pad"]:
        s["ids"][rows - case["pad"]:] = -1
    s["y"] = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ---- the plain forms ------------------------------------------------------------------------------


def _norm(s):
    v = s["x"].float()
    out = {}
    if s["residual"]:
        v = v + s["stream"].float()
        out["stream"] = v.to(torch.bfloat16)
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["weight"].float()
    out["out"] = y.to(torch.bfloat16)
    if s["fp8"]:
        out["fp8"] = _decode(*_encode(out["out"].float(), 128), 128).to(torch.bfloat16)
    return out


def _route(s):
    rows, n, k = s["rows"], s["experts"], s["topk"]
    z = s["logits"].double()
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    choice = score if s["balance"] is None else score + s["balance"].double()
    choice = torch.where(z > -math.inf, choice, torch.full_like(choice, -math.inf))
    if s["groups"] > 1:
        c = choice.view(rows, s["groups"], -1)
        best = torch.sort(c, dim=2, descending=True).values[:, :, : s["group_top"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        total = torch.where(some, total, torch.full_like(total, -math.inf))
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, : s["topk_group"]]
        kept = torch.zeros_like(some).scatter_(1, order, True)
        choice = torch.where(kept[:, :, None], c, torch.full_like(c, -math.inf)).view(rows, n)
    top = torch.sort(choice, dim=1, descending=True, stable=True)
    ids = torch.where(top.values[:, :k] > -math.inf, top.indices[:, :k], n).sort(1).values
    w = torch.where(ids < n, score.gather(1, ids.clamp(max=n - 1)), 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"ids": torch.where(ids < n, ids, -1).int(), "weights": w.float()}


def _experts(s):
    rows, n, k, hidden = s["rows"], s["experts"], s["topk"], s["hidden"]
    wide = lambda w, c: w.float() if c is None else _decode(w.view(torch.float8_e4m3fn), c, 128)  # noqa: E731
    x = wide(s["x"], s["x_scales"])
    # the (row, expert) pairs sorted by expert, each expert's padded to the largest count
    ids = s["ids"].long().view(-1)
    key = torch.where(ids >= 0, ids, n)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=n + 1)
    start = counts.cumsum(0) - counts
    expert = key[order]
    rank = torch.arange(rows * k, device=ids.device) - start[expert]
    live = torch.nonzero(expert < n)[:, 0]
    order, expert, rank = order[live], expert[live], rank[live]
    active = torch.nonzero(counts[:n])[:, 0]
    slot = ((counts[:n] > 0).cumsum(0) - 1)[expert]
    most = int(counts[:n].max())
    xp = torch.zeros(active.numel(), most, hidden, device=x.device)
    xp[slot, rank] = x[order // k]
    pick = lambda w, c: wide(w[active], None if c is None else c[active]).transpose(1, 2)  # noqa: E731
    gate, up = torch.bmm(xp, pick(s["w13"], s["w13_scales"])).chunk(2, -1)
    h = gate / (1 + torch.exp(-gate)) * up
    h = _decode(*_encode(h.contiguous(), 32), 32) if s["fp8"] else h.to(torch.bfloat16).float()
    o = torch.bmm(h, pick(s["w2"], s["w2_scales"]))
    part = torch.zeros(rows * k, hidden, device=x.device)
    part[order] = o[slot, rank]
    return (part.view(rows, k, hidden) * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)


# ---- one pass -------------------------------------------------------------------------------------


def _own(s):
    """The framework's calls. A state's workspace is made on its first pass and kept."""
    from sparse_attention_decode_kpool_gb300 import api

    if s["op"] == "norm":
        out = {"out": s["out"]}
        if s["fp8"]:
            api.dsa_rmsnorm(s["x"], s["weight"], EPS, s["out"], residual=s["stream"], residual_out=s["stream_out"], codes=s["codes"],
                            scales=s["scales"])
            api.dsa_dequantize_latent(s["codes"], s["scales"], s["back"])
            out["fp8"] = s["back"]
        else:
            api.dsa_rmsnorm(s["x"], s["weight"], EPS, s["out"], residual=s["stream"], residual_out=s["stream_out"])
        if s["residual"]:
            out["stream"] = s["stream_out"]
        return out
    if s["op"] == "route":
        api.dsa_route(s["logits"], s["topk"], s["ids"], s["weights"], score=s["score"], bias=s["balance"], n_group=s["groups"],
                      topk_group=s["topk_group"], group_top=s["group_top"], renorm=s["renorm"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if "ws" not in s:
        need = api.dsa_experts_workspace(s["rows"], s["topk"], s["experts"], s["hidden"], s["inter"], s["fp8"])
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    api.dsa_experts(s["x"], s["ids"], s["weights"], s["w13"], s["w2"], s["y"], x_scales=s["x_scales"], w13_scales=s["w13_scales"],
                    w2_scales=s["w2_scales"], status=s["status"], workspace=s["ws"])
    return s["y"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "route": _route, "experts": _experts}[state["op"]](state)


def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        per = 2 + 2 + (4 if case["residual"] else 0)
        if case["fp8"]:  # codes and scales out and in again, bf16 rows out
            per += 2 * (1 + 4 / 128) + 2
        return {"bytes": int(rows * case["width"] * per + 2 * case["width"]), "flops": 4 * rows * case["width"]}
    if case["op"] == "route":
        return {"bytes": rows * (4 * case["experts"] + 8 * case["topk"]) + (4 * case["experts"] if case["bias"] else 0), "flops": 0}
    n, k, hidden, inter = case["experts"], case["topk"], case["hidden"], case["inter"]
    live = rows - case["pad"]
    size = 1 + 4 / 128 if case["fp8"] else 2
    chosen = n * (1 - (1 - k / n) ** live)  # experts that any row chose, were they all as popular
    return {"bytes": int(chosen * 3 * hidden * inter * size + live * hidden * size + rows * hidden * 2 + rows * k * 8),
            "flops": 6 * live * k * hidden * inter}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def _fp8_64(v, group):
    """What FP8 rows hold of v (64 bits): the nearest of E4M3's values times 2^k, ties to even."""
    a = v.reshape(*v.shape[:-1], -1, group)
    top = a.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448))
    k = torch.where(top > 448 * torch.exp2(k), k + 1, k)
    k = torch.where((top > 0) & (top <= 448 * torch.exp2(k - 1)), k - 1, k).clamp(min=-126)
    b = a / torch.exp2(k)
    _, e = torch.frexp(b)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(b / step) * step * torch.exp2(k)).reshape(v.shape)


def _e4m3_64(codes):
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
    return torch.where(c >= 128, -v, v)


def _rows64(w, scales):
    return w.double() if scales is None else _e4m3_64(w) * scales.double().repeat_interleave(128, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = {}
        v = s["x"].double()
        if case["residual"]:
            v = v + s["stream"].double()
            out["stream"] = v
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * s["weight"].double()
        out["out"] = y
        if case["fp8"]:
            out["fp8"] = _fp8_64(y.to(torch.bfloat16).double(), 128)
        return out
    if case["op"] == "route":
        # the chosen experts are decided one after the other, by the definition
        rows, n = case["rows"], case["experts"]
        z = s["logits"].double()
        score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        choice = score + (0 if s["balance"] is None else s["balance"].double())
        choice = choice.masked_fill(z == -math.inf, -math.inf)
        if case["groups"] > 1:
            c = choice.reshape(rows, case["groups"], -1)
            best = c.topk(case["group_top"], 2).values
            total = best.masked_fill(best == -math.inf, 0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
            for _ in range(case["groups"] - case["topk_group"]):
                # the last of the worst groups goes
                worst = case["groups"] - 1 - total.flip(1).argmin(1)
                c[torch.arange(rows, device=z.device), worst] = -math.inf
                total[torch.arange(rows, device=z.device), worst] = math.inf
            choice = c.reshape(rows, n)
        taken = torch.zeros(rows, n, dtype=torch.bool, device=z.device)
        for _ in range(case["topk"]):
            at = choice.argmax(1, keepdim=True)
            taken |= torch.zeros_like(taken).scatter_(1, at, True) & (choice > -math.inf)
            choice = choice.scatter(1, at, -math.inf)
        w = torch.where(taken, score, 0.0)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        at = torch.where(taken, torch.arange(n, device=z.device), n).sort(1).values[:, : case["topk"]]
        return {"ids": None, "weights": torch.where(at < n, w.gather(1, at.clamp(max=n - 1)), 0.0)}
    x = _rows64(s["x"], s["x_scales"])
    y = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        row, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not row.numel():
            continue
        part = lambda w, c: _rows64(w[e], None if c is None else c[e])  # noqa: E731
        z = x[row] @ part(s["w13"], s["w13_scales"]).T
        gate, up = z[:, : case["inter"]], z[:, case["inter"]:]
        h = gate * torch.sigmoid(gate) * up
        h = _fp8_64(h, 32) if case["fp8"] else h.to(torch.bfloat16).double()
        y[row] += s["weights"][row, j, None].double() * (h @ part(s["w2"], s["w2_scales"]).T)
    return y
