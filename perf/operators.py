"""The 4-bit latent cache and the page operators, as their users call them: cases, inputs and plain forms.

Kinds of cases:

* ``store``   a chunk of latent rows encoded into the 4-bit cache and read back
* ``append``  one token per sequence appended to paged caches whose latent cache is 4-bit
* ``attend``  sparse latent attention over the selected tokens of a 4-bit cache
* ``turn``    a scheduler's turn between two decode steps: ended sequences freed, others forked over
  them, and room made for each sequence's next token (new pages, copies of shared ones)
* ``compact`` the live pages of a pool moved to its front

The cache: value = 2^cache_exp * E4M3 scale of a 16-channel block * E2M1 code, channel 2i in the low
nibble of byte i.
"""
import math

import torch

own = False

KVL = 512
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
EPS = 1e-6


def listed():
    return [
        # A prefill chunk's latent rows go into the cache.
        {"name": "store_chunk_4096", "op": "store", "rows": 4096, "cache_exp": -8},
        # A long prompt's rows, 4 sequences of 131,072 tokens, re-encoded at once (an odd count).
        {"name": "store_context_524283", "op": "store", "rows": 524283, "cache_exp": -8},
        # The append of a decode batch of 8 and of a large serving batch, pages of 64 tokens.
        {"name": "append_8", "op": "append", "batch": 8, "block": 64, "max_len": 4096, "kpool": 4, "cache_exp": -8},
        {"name": "append_253", "op": "append", "batch": 253, "block": 64, "max_len": 2048, "kpool": 4, "cache_exp": -8},
        # The tiny single-query layer: latency alone.
        {"name": "attend_tiny", "op": "attend", "rows": 1, "batch": 1, "heads": 4, "max_len": 2048, "min_len": 2045, "topk": 256,
         "block": 0, "cache_exp": -8},
        # A long-context decode batch: 8 sequences of 262,144 tokens.
        {"name": "attend_8x262144", "op": "attend", "rows": 8, "batch": 8, "heads": 64, "max_len": 262144, "min_len": 262144,
         "topk": 2048, "block": 0, "cache_exp": -8},
        # Paged decode: 64 sequences of 4,096 to 65,536 tokens, pages of 64 tokens.
        {"name": "attend_paged_64", "op": "attend", "rows": 64, "batch": 64, "heads": 64, "max_len": 65536, "min_len": 4096,
         "topk": 2048, "block": 64, "cache_exp": -8},
        # A chunked prefill: 4,096 query rows of one sequence of 131,072 tokens.
        {"name": "attend_prefill_4096", "op": "attend", "rows": 4096, "batch": 1, "heads": 64, "max_len": 131072,
         "min_len": 131072, "topk": 2048, "block": 0, "cache_exp": -8},
        # A turn of one layer's pool: 64 sequences, half of them forked anew.
        {"name": "turn_64", "op": "turn", "batch": 64, "layers": 1, "block": 64, "max_len": 8192, "kpool": 4},
        # A turn of a larger pool and batch, the caches of four layers under one table.
        {"name": "turn_251", "op": "turn", "batch": 251, "layers": 4, "block": 64, "max_len": 16384, "kpool": 4},
        # Compaction of a small pool and of a large one after most sequences ended.
        {"name": "compact_16", "op": "compact", "batch": 16, "layers": 1, "block": 64, "max_len": 8192, "kpool": 4, "keep": 0.3},
        {"name": "compact_64", "op": "compact", "batch": 64, "layers": 1, "block": 64, "max_len": 65536, "kpool": 4, "keep": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "append", "attend", "attend", "turn", "compact"])
    exp = rng.choice([-9, -8, -6, 0])
    if op == "store":
        return {"op": op, "rows": _log(rng, 1, 400000), "cache_exp": exp}
    if op == "append":
        return {"op": op, "batch": _log(rng, 1, 250), "block": rng.choice([16, 32, 64, 128]), "max_len": _log(rng, 256, 2048) // 128 * 128,
                "kpool": rng.choice([2, 4, 8]), "cache_exp": exp}
    if op == "attend":
        heads = rng.choice([1, 4, 16, 24, 64, 64, 64, 96, 128])
        topk = rng.choice([64, 256, 512, 1000, 2048])
        rows = _log(rng, 1, min(4000, max(2, 4096 * 64 * 2048 // (max(heads, 16) * topk) // 4)))
        batch = 1 if rows > 128 else rows
        hi = 131072 if batch <= 8 else 16384
        max_len = _log(rng, 64, hi)
        return {"op": op, "rows": rows, "batch": batch, "heads": heads, "max_len": max_len, "min_len": max(1, max_len // 3), "topk": topk,
                "block": rng.choice([0, 16, 64]), "cache_exp": exp}
    if op == "turn":
        return {"op": op, "batch": _log(rng, 2, 240), "layers": rng.choice([1, 2, 3]), "block": rng.choice([16, 32, 64]),
                "max_len": _log(rng, 128, 16000) // 64 * 64, "kpool": 4}
    return {"op": op, "batch": _log(rng, 2, 64), "layers": rng.choice([1, 2]), "block": rng.choice([16, 32, 64]),
            "max_len": _log(rng, 128, 20000) // 64 * 64, "kpool": 4, "keep": round(rng.uniform(0.1, 0.9), 2)}


# ---- the codec in elementary operations ---------------------------------------------------------


def _encode(x, cache_exp):
    """bf16 rows [n, 512] -> codes [n, 256] u8, scales [n, 32] u8 (E4M3 bytes)."""
    a = x.float().view(-1, KVL // 16, 16) * 2.0 ** -cache_exp
    s = (a.abs().amax(2, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    m = torch.where(sf > 0, a.abs() / sf, torch.zeros_like(a))
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = torch.where((a < 0) & (sf > 0), code + 8, code).view(-1, KVL)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(-1, KVL // 16).view(torch.uint8)


def _decode(codes, scales, cache_exp):
    """f32 values [..., 512] of the packed codes [..., 256] and scales [..., 32]."""
    lut = torch.tensor(LUT, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1)
    s = scales.view(torch.float8_e4m3fn).float() * 2.0 ** cache_exp
    return (v.view(*codes.shape[:-1], KVL // 16, 16) * s.unsqueeze(-1)).view(*codes.shape[:-1], KVL)


# ---- inputs ---------------------------------------------------------------------------------------


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _latent(g, rows):
    """Latent rows after their RMS norm: unit variance, a few channels that stand out."""
    gain = torch.exp(0.4 * torch.randn(KVL, generator=g, device="cuda"))
    return (torch.randn(rows, KVL, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _latent_cache(g, rows, cache_exp):
    codes = torch.empty(rows, KVL // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, KVL // 16, dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.4 * torch.randn(KVL, generator=g, device="cuda"))
    for i in range(0, rows, 1 << 18):
        n = min(1 << 18, rows - i)
        x = (torch.randn(n, KVL, generator=g, device="cuda") * gain).to(torch.bfloat16)
        codes[i:i + n], scales[i:i + n] = _encode(x, cache_exp)
    return codes, scales


def _lengths(g, batch, lo, hi):
    """Lengths spread evenly from hi down to lo, in a shuffled order: their pages add up to the same number
    whatever the seed."""
    at = torch.randperm(batch, generator=g, device="cuda")
    return (hi - at * (hi - lo) // max(1, batch - 1)).int()


def _table(g, lens, block, max_blocks, spare):
    """Block table [batch, max_blocks] (-1 past a sequence's last page) over shuffled pages."""
    need = (lens.long() + block - 1) // block
    total = int(need.sum())
    num = total + spare
    perm = torch.randperm(num, generator=g, device="cuda").int()
    start = need.cumsum(0) - need
    j = torch.arange(max_blocks, device="cuda")
    at = (start[:, None] + j[None]).clamp(max=num - 1)
    return torch.where(j[None] < need[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous(), num


def _caches(g, layers, num, block, kpool):
    """The paged caches of `layers` layers, [layers, pages, bytes of a page]: indexer keys and gates,
    validity, latent codes and scales, pooled keys and their flags."""
    byte = lambda w: torch.randint(0, 256, (layers, num, w), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    flag = lambda w: torch.ones(layers, num, w, device="cuda", dtype=torch.uint8)  # noqa: E731
    return {"k_raw": byte(block * 256), "gate": byte(block * 256), "valid": flag(block), "codes": byte(block * 256),
            "scales": byte(block * 32), "kpool": byte(block // kpool * 256), "pool_valid": flag(block // kpool)}


def _refs(table, num):
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    return refs.index_add_(0, table.view(-1).clamp(min=0).long(), (table.view(-1) >= 0).int())


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "store":
        s["x"] = _latent(g, case["rows"])
        s["codes"] = torch.empty(case["rows"], KVL // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(case["rows"], KVL // 16, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["x"])
        return s
    if case["op"] == "attend":
        rows, batch, block = case["rows"], case["batch"], case["block"]
        lens = _lengths(g, batch, case["min_len"], case["max_len"])
        s["seq_lens"] = lens
        s["row_seq"] = (torch.arange(rows, device="cuda") % batch).int()
        if block:
            s["max_blocks"] = -(-case["max_len"] // block)
            s["table"], s["num"] = _table(g, lens, block, s["max_blocks"], 8)
            cache_rows = s["num"] * block
        else:
            s["table"], s["num"] = None, 0
            cache_rows = batch * case["max_len"]
        s["codes"], s["scales"] = _latent_cache(g, cache_rows, case["cache_exp"])
        s["qlat"] = _normal(g, rows, case["heads"], KVL)
        # Selected pools of four tokens, ascending, -1 after them: a decode row chooses among its whole
        # sequence, the rows of a prefill chunk are its last positions.
        ctx = lens[s["row_seq"].long()].long()
        if rows > batch:
            ctx = (ctx - rows + 1 + torch.arange(rows, device="cuda")).clamp(min=0)
        s["token_ids"] = torch.full((rows, case["topk"]), -1, dtype=torch.int32, device="cuda")
        pools = max(1, case["max_len"] // 4)
        sk = min(case["topk"] // 4, pools)
        for i in range(0, rows, 1024):
            n = ctx[i:i + 1024] // 4
            u = torch.rand(n.numel(), pools, generator=g, device="cuda")
            u.masked_fill_(torch.arange(pools, device="cuda")[None] >= n[:, None], -1.0)
            v, p = u.topk(sk, 1)
            p = torch.where(v >= 0, p, torch.full_like(p, pools)).sort(1).values
            t = (p[:, :, None] * 4 + torch.arange(4, device="cuda")).view(n.numel(), -1)
            s["token_ids"][i:i + 1024, :sk * 4] = torch.where(t < 4 * n[:, None], t, torch.full_like(t, -1)).int()
        s["scale"] = 256 ** -0.5
        s["olat"] = torch.empty(rows, case["heads"], KVL, dtype=torch.bfloat16, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    # paged caches
    batch, block, kpool = case["batch"], case["block"], case["kpool"]
    s["max_blocks"] = -(-case["max_len"] // block) + 1
    lens = _lengths(g, batch, max(1, case["max_len"] // 8), case["max_len"] - 1)
    s["seq_lens"], s["lens0"] = lens.clone(), lens
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        s["table"], s["num"] = _table(g, lens + 1, block, s["max_blocks"], 4)
        n, cap = s["num"] * block, s["num"]
        s["codes"], s["scales"] = _latent_cache(g, n, case["cache_exp"])
        s["k_raw"], s["gate"] = _normal(g, cap, block, 128), _normal(g, cap, block, 128)
        s["valid"] = (torch.rand(cap, block, generator=g, device="cuda") < 0.99).to(torch.uint8)
        s["kpool"] = _normal(g, cap, block // kpool, 128)
        s["pool_valid"] = torch.ones(cap, block // kpool, dtype=torch.uint8, device="cuda")
        s["k_new"], s["gate_new"] = _normal(g, batch, 128), _normal(g, batch, 128)
        s["ckv_new"] = _latent(g, batch)
        s["ape"] = _normal(g, kpool, 128, std=0.1, dtype=torch.float32)
        s["ln_w"], s["ln_b"] = (_normal(g, 128, std=0.1).float() + 1).to(torch.bfloat16), _normal(g, 128, std=0.1)
        s["row_ctx"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        at = s["table"].gather(1, (lens.long() // block)[:, None])[:, 0].long() * block + lens.long() % block
        s["new_rows"] = at.int()
        s["out"] = torch.empty(batch, KVL, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "turn":
        s["table"], s["num"] = _table(g, lens, block, s["max_blocks"], 4 * batch + 16)
        s["refs"] = _refs(s["table"], s["num"])
        order = torch.randperm(batch, generator=g, device="cuda").int()
        half = batch // 2
        s["parents"] = order[half:][torch.randint(0, batch - half, (half,), generator=g, device="cuda")].contiguous()
        s["children"] = order[:half].contiguous()
        s["ended"] = order[:max(1, half // 4)].contiguous()
    else:
        full, s["num"] = _table(g, lens, block, s["max_blocks"], 16)
        kept = torch.rand(batch, generator=g, device="cuda") < case["keep"]
        kept[0], kept[-1] = True, False
        s["seq_lens"] = torch.where(kept, lens, torch.zeros_like(lens))
        s["table0"] = torch.where(kept[:, None], full, torch.full_like(full, -1)).contiguous()
        s["refs0"] = _refs(s["table0"], s["num"])
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        s["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["caches"] = _caches(g, case["layers"], s["num"], block, kpool)
    return s


# ---- the plain forms ------------------------------------------------------------------------------


def _attend(s):
    rows, heads, topk = s["rows"], s["heads"], s["topk"]
    t = s["token_ids"].long()
    b = s["row_seq"].long()[:, None]
    at = t.clamp(min=0)
    if s["table"] is None:
        at = b * s["max_len"] + at
    else:
        at = s["table"].long()[b, at // s["block"]] * s["block"] + at % s["block"]
    at = torch.where(t >= 0, at, torch.zeros_like(at))
    if rows * topk > s["codes"].shape[0]:
        v = _decode(s["codes"], s["scales"], s["cache_exp"])[at.view(-1)].view(rows, topk, KVL)
    else:
        v = _decode(s["codes"][at], s["scales"][at], s["cache_exp"])
    v = torch.where((t >= 0)[:, :, None], v, torch.zeros_like(v))
    logit = torch.matmul(s["qlat"].float(), v.transpose(1, 2)) * s["scale"]
    logit = logit.masked_fill((t < 0)[:, None], -math.inf)
    top = logit.amax(2, keepdim=True)
    p = torch.exp(logit - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    z = p.sum(2, keepdim=True)
    return (torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))).to(torch.bfloat16)


def _append(s):
    block, kpool, batch = s["block"], s["kpool"].shape[1], s["batch"]
    kp = block // kpool
    s["seq_lens"].copy_(s["lens0"])
    t = s["seq_lens"].long()
    page = s["table"].gather(1, (t // block)[:, None])[:, 0].long()
    row = page * block + t % block
    s["k_raw"].view(-1, 128)[row] = s["k_new"]
    s["gate"].view(-1, 128)[row] = s["gate_new"]
    s["valid"].view(-1)[row] = 1
    c, sc = _encode(s["ckv_new"], s["cache_exp"])
    s["codes"][row], s["scales"][row] = c, sc
    s["seq_lens"] += 1
    s["row_ctx"].copy_(s["seq_lens"])
    # the pool that the token completes, where it does
    pool = t // kp
    done = (t + 1) % kp == 0
    slot = page[:, None] * block + ((pool * kp) % block)[:, None] + torch.arange(kp, device=t.device)
    k = s["k_raw"].view(-1, 128)[slot].float()
    mean = k.mean(2, keepdim=True)
    kn = (k - mean) / torch.sqrt(((k - mean) ** 2).mean(2, keepdim=True) + EPS) * s["ln_w"].float() + s["ln_b"].float()
    kn = kn.to(torch.bfloat16).float()  # the norm's output is bf16 by its definition
    e = s["gate"].view(-1, 128)[slot].float() + s["ape"]
    e = torch.exp(e - e.amax(1, keepdim=True))
    key = ((e * kn).sum(1) / e.sum(1)).to(torch.bfloat16)
    ok = s["valid"].view(-1)[slot].amin(1) > 0
    key = torch.where(ok[:, None], key, torch.zeros_like(key))
    out = (page * kpool + pool % kpool)
    old = s["kpool"].view(-1, 128)[out]
    s["kpool"].view(-1, 128)[out] = torch.where(done[:, None], key, old)
    flag = s["pool_valid"].view(-1)[out]
    s["pool_valid"].view(-1)[out] = torch.where(done, ok.to(torch.uint8), flag)
    return _decode(c, sc, s["cache_exp"]).to(torch.bfloat16)


def _release(table, refs, rows):
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), -(rows >= 0).int().view(-1))


def _turn(s):
    table, refs, lens, block = s["table"], s["refs"], s["seq_lens"], s["block"]
    ended, parents, children = s["ended"].long(), s["parents"].long(), s["children"].long()
    # free
    _release(table, refs, table[ended])
    table[ended] = -1
    lens[ended] = 0
    # fork: a child's former pages are released, its parent's shared
    _release(table, refs, table[children])
    j = torch.arange(table.shape[1], device=table.device)
    rows = table[parents]
    rows = torch.where(j[None] < ((lens[parents] + block - 1) // block)[:, None], rows, torch.full_like(rows, -1))
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).int().view(-1))
    table[children] = rows
    lens[children] = lens[parents]
    # reserve one token: a new page at a page's end, a copy of a shared page
    at = (lens.long() // block)[:, None]
    old = table.gather(1, at)[:, 0].long()
    share = (old >= 0) & (refs[old.clamp(min=0)] > 1)
    need = share | (old < 0)
    order = torch.sort((refs > 0).to(torch.uint8), stable=True).indices
    new = torch.where(need, order[(need.long().cumsum(0) - 1).clamp(min=0)], old)
    refs.index_add_(0, old.clamp(min=0), -share.int())
    refs.index_add_(0, new, need.int())
    table.scatter_(1, at, new.int()[:, None])
    src = torch.where(share, old, new)
    for c in s["caches"].values():
        c[:, new] = c[:, src]
    return {"table": table, "refs": refs, "seq_lens": lens, **s["caches"]}


def _compact(s):
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    live = refs > 0
    n = live.sum(dtype=torch.int32)
    ids = torch.arange(refs.numel(), device=refs.device)
    src = torch.nonzero(live & (ids >= n))[:, 0]
    dst = torch.nonzero(~live & (ids < n))[:, 0]
    remap = ids.int()
    remap[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], table))
    s["live"].copy_(n)
    for c in s["caches"].values():
        c[:, dst] = c[:, src]
    return {"table": table, "refs": refs, "live": s["live"], **s["caches"]}


# ---- one pass -------------------------------------------------------------------------------------


def _own(s):
    """The framework's calls. Descriptors and workspaces are made on a state's first pass and kept."""
    from sparse_attention_decode_kpool_gb300 import api

    if s["op"] == "store":
        api.dsa_quantize_latent_fp4(s["x"], s["codes"], s["scales"], s["cache_exp"])
        api.dsa_dequantize_latent_fp4(s["codes"], s["scales"], s["out"], s["cache_exp"])
        return s["out"]
    if "pg" not in s:
        s["pg"] = api.paging(s["seq_lens"], s["max_len"] + (0 if s["op"] == "attend" else 1), s["table"], s["block"] or 0, s["num"])
        if s["op"] == "attend":
            n = api.dsa_sparse_mla_decode_fp4_workspace(s["rows"], s["heads"], s["topk"], 0, False)
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        if s["op"] in ("turn", "compact"):
            s["arrays"] = api.page_arrays([layer for c in s["caches"].values() for layer in c], s["num"])
            n = api.dsa_pages_workspace(s["num"], s["batch"])
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    if s["op"] == "attend":
        api.dsa_sparse_mla_decode_fp4(s["qlat"], s["row_seq"], s["codes"], s["scales"], s["cache_exp"], s["pg"], s["token_ids"],
                                      s["scale"], olat=s["olat"], status=s["status"], workspace=s["ws"])
        return s["olat"]
    if s["op"] == "append":
        s["seq_lens"].copy_(s["lens0"])
        api.dsa_decode_append_fp4(s["k_new"], s["gate_new"], s["ckv_new"], s["ape"], s["ln_w"], s["ln_b"], EPS, s["pg"],
                                  s["seq_lens"], 0, s["block"] // s["kpool"].shape[1], s["k_raw"], s["gate"], s["valid"],
                                  s["codes"], s["scales"], s["cache_exp"], s["kpool"], s["pool_valid"], row_ctx=s["row_ctx"],
                                  status=s["status"])
        api.dsa_dequantize_latent_fp4(s["codes"], s["scales"], s["out"], s["cache_exp"], rows=s["new_rows"], status=s["status"])
        return s["out"]
    if s["op"] == "turn":
        api.dsa_pages_free(s["ended"], s["pg"], s["table"], s["seq_lens"], s["refs"], status=s["status"])
        api.dsa_pages_fork(s["parents"], s["children"], s["pg"], s["table"], s["seq_lens"], s["refs"], status=s["status"])
        api.dsa_pages_reserve(s["pg"], s["table"], s["refs"], 1, s["arrays"], 0, 4, status=s["status"], workspace=s["ws"])
        return {"table": s["table"], "refs": s["refs"], "seq_lens": s["seq_lens"], **s["caches"]}
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    api.dsa_pages_compact(s["pg"], s["table"], s["refs"], s["arrays"], live=s["live"], status=s["status"], workspace=s["ws"])
    return {"table": s["table"], "refs": s["refs"], "live": s["live"], **s["caches"]}


def run(state):
    op = state["op"]
    if own:
        out = _own(state)
    elif op == "store":
        codes, scales = _encode(state["x"], state["cache_exp"])
        state["codes"].copy_(codes)
        state["scales"].copy_(scales)
        out = _decode(state["codes"], state["scales"], state["cache_exp"]).to(torch.bfloat16)
    elif op == "attend":
        out = _attend(state)
    elif op == "append":
        out = _append(state)
    elif op == "turn":
        return _turn(state)
    else:
        return _compact(state)
    if op == "append":
        return {"latent": out, "seq_lens": state["seq_lens"], "row_ctx": state["row_ctx"], "k_raw": state["k_raw"],
                "gate": state["gate"], "valid": state["valid"], "kpool": state["kpool"], "pool_valid": state["pool_valid"]}
    return out


def work(case):
    op = case["op"]
    if op == "store":
        # bf16 rows in, the 4-bit rows out and in again, bf16 rows out
        return {"bytes": case["rows"] * (1024 + 288 + 288 + 1024), "flops": 0}
    if op == "append":
        # the staged rows in, the stored ones out, a pool's rows in and its key out for one token in kpool
        return {"bytes": case["batch"] * (2 * 512 + 1024 + 288 + (512 * case["kpool"] + 256) // case["kpool"] + 288 + 1024), "flops": 0}
    if op == "attend":
        rows, heads, topk = case["rows"], case["heads"], min(case["topk"], case["max_len"])
        tokens = min(rows * topk, case["batch"] * case["max_len"])
        return {"bytes": rows * heads * KVL * 4 + tokens * 288 + rows * case["topk"] * 4, "flops": 4 * rows * heads * KVL * topk}
    page = case["layers"] * (case["block"] * (256 * 3 + 32 + 1) + case["block"] // case["kpool"] * 257)
    mean = (case["max_len"] // 8 + case["max_len"]) / 2 / case["block"]
    if op == "turn":
        # about three sequences in four copy a page; the forked rows of the table; the reference counts once
        half = case["batch"] // 2
        return {"bytes": int(0.75 * case["batch"] * 2 * page + half * mean * 16 + case["batch"] * mean * 4), "flops": 0}
    num, live = case["batch"] * mean, case["batch"] * mean * case["keep"]
    return {"bytes": int(2 * page * live * (1 - case["keep"]) + 2 * num * 4 + 2 * live * 4), "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def _nearest(a, low, bits):
    """a >= 0 rounded to `bits` significant bits (ties to even), steps no finer than 2^low."""
    _, e = torch.frexp(a)
    step = torch.exp2((e - bits).clamp(min=low).double())
    return torch.round(a / step) * step


def _values64(x, cache_exp):
    """What the 4-bit cache holds of rows x, in 64 bits."""
    a = x.double().reshape(-1, KVL // 16, 16) * 2.0 ** -cache_exp
    s = _nearest(a.abs().amax(-1) / 6, -9, 4).clamp(max=448)[..., None]
    m = torch.where(s > 0, a.abs() / torch.where(s > 0, s, 1.0), 0.0)
    v = torch.sign(a) * _nearest(m, -1, 2).clamp(max=6) * s
    return (v * 2.0 ** cache_exp).reshape(-1, KVL)


def _cache64(codes, scales, cache_exp):
    c = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], KVL).long()
    mag = torch.tensor(LUT[:8], dtype=torch.float64, device=codes.device)[c % 8] * torch.where(c >= 8, -1.0, 1.0).double()
    e, m = (scales.long() >> 3).double(), (scales.long() & 7).double()
    s = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), 2.0 ** -6 * m / 8)
    return mag * s.repeat_interleave(16, -1) * 2.0 ** cache_exp


def exact(case, seed):
    if case["op"] in ("turn", "compact"):
        return None  # copies and whole numbers
    s = prepare(case, seed)
    if case["op"] == "store":
        out = torch.empty(case["rows"], KVL, dtype=torch.float64, device="cuda")
        for i in range(0, case["rows"], 1 << 16):
            out[i:i + (1 << 16)] = _values64(s["x"][i:i + (1 << 16)], case["cache_exp"])
        return out
    if case["op"] == "attend":
        out = torch.zeros(case["rows"], case["heads"], KVL, dtype=torch.float64, device="cuda")
        step = max(1, min(64, (1 << 33) // (case["topk"] * KVL * 8) // 4))
        for i in range(0, case["rows"], step):
            t = s["token_ids"][i:i + step].long()
            seq = s["row_seq"][i:i + step].long()[:, None].expand_as(t)
            t0 = torch.where(t < 0, 0, t)
            at = seq * case["max_len"] + t0 if s["table"] is None else s["table"][seq, t0 // case["block"]].long() * case["block"] + t0 % case["block"]
            at = torch.where(t < 0, 0, at)
            v = _cache64(s["codes"][at], s["scales"][at], case["cache_exp"])
            z = torch.einsum("rhc,rtc->rht", s["qlat"][i:i + step].double(), v) / 16
            z = torch.where((t < 0)[:, None], -math.inf, z)
            w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            out[i:i + step] = torch.einsum("rht,rtc->rhc", w, v)
        return out
    # append: the pooled keys of the pools that became whole; the rest is copied
    block, kp, L = case["block"], case["kpool"], s["lens0"].tolist()
    keys = s["kpool"].double()
    k_raw, gate, valid = s["k_raw"].double(), s["gate"].double(), s["valid"].clone()
    for b, t in enumerate(L):
        page = int(s["table"][b, t // block])
        k_raw[page, t % block], gate[page, t % block], valid[page, t % block] = s["k_new"][b].double(), s["gate_new"][b].double(), 1
        if (t + 1) % kp == 0:
            at = slice(t % block + 1 - kp, t % block + 1)
            k = k_raw[page, at]
            d = k - k.mean(1, keepdim=True)
            kn = d / (d.square().mean(1, keepdim=True) + EPS).sqrt() * s["ln_w"].double() + s["ln_b"].double()
            kn = kn.to(torch.bfloat16).double()
            w = torch.softmax(gate[page, at] + s["ape"].double(), 0)
            keys[page, t % block // kp] = (w * kn).sum(0) * float(valid[page, at].min() > 0)
    return {"latent": _values64(s["ckv_new"], case["cache_exp"]), "seq_lens": None, "row_ctx": None, "k_raw": k_raw, "gate": gate,
            "valid": None, "kpool": keys, "pool_valid": None}
