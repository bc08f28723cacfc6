"""dsa_rmsnorm, dsa_dequantize_latent, dsa_route and dsa_router_logits against plain 64-bit
restatements."""
import math

import numpy as np
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_TOKEN

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _rows(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF16).cuda()


# ---- norm -----------------------------------------------------------------------------------------

# The value to f32 and then to bf16: half of bf16's eps of 2^-7, and half of f32's.
NORM_TOL = 2.0 ** -8 + 2.0 ** -24


def _norm_ref(x, res, w, eps):
    v = x.double() + (0 if res is None else res.double())
    return v, v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * w.double()


def _close(got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol * want.abs() + 1e-38).all()), float((err / want.abs().clamp(min=1e-30)).max())


@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 8), (2, 250), (9, 256), (33, 264), (8, 512),
                                        (17, 1000), (4, 1024), (7, 2048), (1021, 1000), (3, 4096),
                                        (5, 5000), (2, 8192), (3, 16384), (2, 32768), (2, 40000),
                                        (700, 4096)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(rows, width, residual):
    x, w = _rows(1, rows, width, std=2.0), _rows(2, width)
    res = _rows(3, rows, width, std=5.0) if residual else None
    out = torch.full_like(x, math.nan)
    ro = torch.full_like(x, math.nan) if residual else None
    api.dsa_rmsnorm(x, w, 1e-6, out, residual=res, residual_out=ro)
    v, want = _norm_ref(x, res, w, 1e-6)
    _close(out, want, NORM_TOL)
    if residual:
        assert torch.equal(ro, v.float().to(BF16))  # one f32 addition of bf16 values, one rounding


@pytest.mark.parametrize("rows,width", [(1, 128), (5, 256), (3, 384), (6, 512), (9, 1024), (2, 2048),
                                        (131, 4096), (2, 7168), (2, 16384), (2, 33024)])
def test_rmsnorm_fp8_rows_are_the_codec_of_out(rows, width):
    x, w, res = _rows(4, rows, width), _rows(5, width), _rows(6, rows, width)
    x[0, :128] = 0
    res[0, :128] = 0  # an all-zero group
    out = torch.empty_like(x)
    mk = lambda: (torch.full((rows, width), 0xAA, dtype=torch.uint8, device="cuda"),  # noqa: E731
                  torch.full((rows, width // 128), -1.0, device="cuda"))
    (codes, scales), (c2, s2), (c3, s3) = mk(), mk(), mk()
    ro = torch.empty_like(x)
    api.dsa_rmsnorm(x, w, 1e-6, out, residual=res, residual_out=ro, codes=codes, scales=scales)
    api.dsa_quantize_latent(out, c2, s2)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    api.dsa_rmsnorm(x, w, 1e-6, residual=res, codes=c3, scales=s3)  # FP8 rows alone
    assert torch.equal(codes, c3) and torch.equal(scales, s3)
    _close(out, _norm_ref(x, res, w, 1e-6)[1], NORM_TOL)


@pytest.mark.parametrize("rows,width", [(4000, 128), (2000, 1000), (1200, 4096), (60, 20001)])
def test_rmsnorm_is_the_formula_rounded_twice(rows, width):
    """To f32, then to bf16, of the 64-bit value: not a value of them is off, though plain f32
    arithmetic would put about one in 50,000 one step off. (A 64-bit value within 2^-40 of a
    border of f32, where the second word's own error could decide, is one in 2^15, and it has to
    be on a border of bf16 too: one in 2^31.)"""
    x, w, res = _rows(31, rows, width, std=3.0), _rows(32, width), _rows(33, rows, width)
    out = torch.empty_like(x)
    eps = 2.0 ** -20
    api.dsa_rmsnorm(x, w, eps, out, residual=res)
    v, want = _norm_ref(x, res, w, eps)
    assert torch.equal(out, want.float().to(BF16))


@pytest.mark.parametrize("width", [1000, 1001, 4096])
def test_rmsnorm_in_place_and_unaligned(width):
    rows = 37
    x, w, res = _rows(7, rows, width), _rows(8, width), _rows(9, rows, width)
    want_o, want_r = torch.empty_like(x), torch.empty_like(x)
    api.dsa_rmsnorm(x, w, 1e-5, want_o, residual=res, residual_out=want_r)
    xa, ra = x.clone(), res.clone()
    api.dsa_rmsnorm(xa, w, 1e-5, xa, residual=ra, residual_out=ra)
    assert torch.equal(xa, want_o) and torch.equal(ra, want_r)
    xa, ra = x.clone(), res.clone()
    api.dsa_rmsnorm(xa, w, 1e-5, ra, residual=ra, residual_out=xa)
    assert torch.equal(ra, want_o) and torch.equal(xa, want_r)
    # two bytes off a 16-byte boundary: the other kernel, the same definition
    buf = torch.zeros(rows * width + 1, dtype=BF16, device="cuda")
    xu = buf[1:].view(rows, width)
    xu.copy_(x)
    out = torch.empty_like(x)
    api.dsa_rmsnorm(xu, w, 1e-5, out)
    _close(out, _norm_ref(x, None, w, 1e-5)[1], NORM_TOL)


def test_rmsnorm_zero_rows_and_special_values():
    x, w = _rows(10, 6, 512), _rows(11, 512)
    x[1] = 0
    x[2, 3] = math.nan
    x[3, 4] = math.inf
    w[7] = math.inf
    out = torch.empty_like(x)
    api.dsa_rmsnorm(x, w, 0.0, out)
    assert bool(torch.isnan(out[1]).all())  # 0 * (1 / 0), as the formula
    api.dsa_rmsnorm(x, w, 1e-6, out)
    assert not bool(out[1, 8:].any()) and bool(torch.isnan(out[1, 7]))  # 0 * inf
    assert bool(torch.isnan(out[2]).all())
    assert bool(torch.isnan(out[3, 4])) and not bool(out[3, 10:].any())
    assert bool(torch.isinf(out[[0, 4, 5], 7]).all())
    w[7] = 1
    api.dsa_rmsnorm(x, w, 1e-6, out)
    _close(out[[0, 4, 5]], _norm_ref(x[[0, 4, 5]], None, w, 1e-6)[1], NORM_TOL)
    api.dsa_rmsnorm(x[:0], w, 1e-6, out[:0])  # no rows


def test_norm_on_a_stream_and_in_a_graph():
    x, w, res = _rows(12, 64, 4096), _rows(13, 4096), _rows(14, 64, 4096)
    want, got = torch.empty_like(x), torch.empty_like(x)
    api.dsa_rmsnorm(x, w, 1e-6, want, residual=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.dsa_rmsnorm(x, w, 1e-6, got, residual=res, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    gr = torch.cuda.CUDAGraph()
    ro = torch.empty_like(x)
    with torch.cuda.graph(gr):
        api.dsa_rmsnorm(x, w, 1e-6, got, residual=res, residual_out=ro)
    x.mul_(2)
    gr.replay()
    api.dsa_rmsnorm(x, w, 1e-6, want, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ---- reading FP8 rows back ------------------------------------------------------------------------


@pytest.mark.parametrize("rows,width", [(1, 128), (7, 512), (300, 640), (70001, 512)])
def test_dequantize_latent(rows, width):
    x = _rows(15, rows, width)
    x[0, 0] = -0.0
    codes = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, width // 128, device="cuda")
    api.dsa_quantize_latent(x, codes, scales)
    back = torch.empty_like(x)
    api.dsa_dequantize_latent(codes, scales, back)
    want = codes.view(torch.float8_e4m3fn).double().view(rows, -1, 128) * scales.double().unsqueeze(-1)
    assert torch.equal(back.double(), want.view(rows, width))  # exact
    # named rows, one of them outside the cache, one twice
    ids = torch.tensor([rows - 1, 0, rows, 0, -1], dtype=torch.int32, device="cuda")
    some = torch.full((5, width), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_dequantize_latent(codes, scales, some, rows=ids, status=status)
    assert torch.equal(some[[0, 1, 3]], back[[rows - 1, 0, 0]])
    assert not bool(some[[2, 4]].any()) and int(status) == DSA_STATUS_BAD_TOKEN
    with pytest.raises(ValueError):
        api.dsa_dequantize_latent(codes, scales, some)


# ---- routing --------------------------------------------------------------------------------------


def _route_ref(logits, k, bias, score, groups, tg, gt, renorm, scale, shared):
    """Row by row in numpy's 64 bits."""
    z = logits.cpu().double().numpy()
    b = None if bias is None else bias.cpu().double().numpy()
    rows, n = z.shape
    ids = np.full((rows, k + shared), -1, dtype=np.int32)
    w = np.zeros((rows, k + shared))
    for r in range(rows):
        row = z[r].copy()
        nan = np.isnan(row) | (np.isposinf(row) if score == "softmax" else False)
        if b is not None:
            nan |= np.isnan(b)
        row[np.isnan(z[r]) | (np.isposinf(z[r]) if score == "softmax" else False)] = -np.inf
        cand = ~nan & (row > -np.inf)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-row))
            else:
                e = np.where(row > -np.inf, np.exp(row - row.max()), 0.0)
                s = e / e.sum()
            c = s if b is None else s + b
        cand &= c > -np.inf
        if groups > 1:
            size = n // groups
            sums = []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if cand[e]), reverse=True)[:gt]
                sums.append(sum(best) if best else -np.inf)
            order = [g for g in sorted(range(groups), key=lambda g: (-sums[g], g)) if sums[g] > -np.inf]
            for g in range(groups):
                if g not in order[:tg]:
                    cand[g * size:(g + 1) * size] = False
        chosen = sorted(sorted((e for e in range(n) if cand[e]), key=lambda e: (-c[e], e))[:k])
        ids[r, :len(chosen)] = chosen
        v = s[chosen]
        if renorm:
            t = v.sum()
            v = v / t if t > 0 else v * 0
        w[r, :len(chosen)] = np.nan if nan.any() else v * scale
        for j in range(shared):
            ids[r, k + j], w[r, k + j] = n + j, 1.0
    return ids, w


ROUTE = [
    # rows, experts, topk, score, bias, groups, topk_group, group_top, renorm, shared
    (1, 1, 1, "sigmoid", False, 1, 1, 1, True, 0),
    (3, 5, 5, "softmax", True, 1, 1, 2, True, 0),
    (64, 64, 8, "softmax", False, 1, 1, 1, True, 1),
    (100, 128, 6, "sigmoid", True, 1, 1, 1, False, 0),
    (257, 256, 8, "sigmoid", True, 8, 4, 2, True, 1),
    (130, 160, 6, "softmax", False, 8, 3, 1, False, 2),
    (65, 96, 16, "sigmoid", True, 3, 2, 2, True, 0),
    (40, 512, 22, "softmax", True, 16, 5, 2, True, 0),
    (33, 320, 10, "sigmoid", False, 32, 9, 1, True, 0),
    (21, 1000, 64, "sigmoid", True, 5, 5, 2, True, 0),
    (9, 1024, 1, "softmax", True, 32, 1, 2, False, 0),
    (50, 66, 2, "sigmoid", True, 22, 1, 1, True, 0),
    (20, 16, 3, "sigmoid", True, 16, 5, 1, True, 0),
]

# The scores, in roundings of 2^-24: an exponential 4 (two units in the last place), its argument
# |z - max| of them (the logits here differ by under 16), the softmax's sum 32 in a lane's chain and
# 5 of the tree, a division and a product; the renormalising sum 37 and product, the scale: under
# 100 of them.
W_TOL = 100 * 2.0 ** -24


def _check_route(logits, k, bias, score, groups, tg, gt, renorm, shared, scale=2.5):
    rows, n = logits.shape
    ids = torch.full((rows, k + shared), -7, dtype=torch.int32, device="cuda")
    w = torch.full((rows, k + shared), -7.0, device="cuda")
    api.dsa_route(logits, k, ids, w, score=score, bias=bias, n_group=groups, topk_group=tg,
                  group_top=gt, renorm=renorm, scale=scale, shared=shared)
    want_ids, want_w = _route_ref(logits, k, bias, score, groups, tg, gt, renorm, scale, shared)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=W_TOL, atol=1e-37)
    return ids, w


@pytest.mark.parametrize("case", ROUTE, ids=["-".join(map(str, c)) for c in ROUTE])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_route(case, kind):
    rows, n, k, score, with_bias, groups, tg, gt, renorm, shared = case
    g = torch.Generator().manual_seed(rows * 31 + n)
    logits = torch.randn(rows, n, generator=g) * 1.5
    bias = torch.randn(n, generator=g) * 0.1 if with_bias else None
    if kind == "ties":  # a handful of distinct values: the lowest id decides
        logits = (logits * 1.5).round() / 1.5
        bias = None if bias is None else (bias * 20).round() / 16
    if kind == "masked":
        logits[torch.rand(rows, n, generator=g) < 0.4] = -math.inf
        logits[0] = -math.inf  # an empty row
        logits[-1] = -math.inf
        logits[-1, n // 2] = 3.0  # a single candidate
    _check_route(logits.cuda(), k, None if bias is None else bias.cuda(), score, groups, tg, gt, renorm,
                 shared)


def test_route_near_ties_are_decided_in_64_bits():
    """Sigmoids a few parts in 1e8 apart (less than an f32 score's own error) in an order that
    f32 arithmetic would not resolve."""
    g = torch.Generator().manual_seed(5)
    rows, n = 400, 256
    base = torch.full((rows, n), 1.0)
    for step in range(3):
        base = torch.where(torch.rand(rows, n, generator=g) < 0.5,
                           torch.nextafter(base, torch.full_like(base, 2.0)), base)
    _check_route(base.cuda(), 8, None, "sigmoid", 1, 1, 1, True, 0)
    _check_route(base.cuda(), 8, None, "softmax", 8, 3, 2, True, 0)
    bias = (torch.randn(n, generator=g) * 1e-7).cuda()
    _check_route(base.cuda(), 8, bias, "sigmoid", 8, 4, 2, True, 0)


def test_route_extreme_logits():
    z = torch.zeros(7, 64)
    z[0] = torch.arange(64) - 120.0   # sigmoids below f32's smallest: their ratios still count
    z[1] = torch.arange(64) * 0.25 - 103.0
    z[2, :3] = 3e38
    z[3] = -3e38
    z[4, 5] = math.inf
    z[5, 9] = math.nan
    z[6, 1], z[6, 2] = -math.inf, math.inf
    for score in ("sigmoid", "softmax"):
        _check_route(z.cuda(), 8, None, score, 1, 1, 1, True, 0)
    bias = torch.zeros(64)
    bias[3], bias[4], bias[60] = -math.inf, math.inf, 1e30
    _check_route(z.cuda(), 8, bias.cuda(), "sigmoid", 4, 2, 2, True, 1)
    bias[7] = math.nan
    _check_route(z.cuda(), 8, bias.cuda(), "softmax", 1, 1, 1, False, 0)


def test_route_padded_logits_and_graph():
    g = torch.Generator().manual_seed(6)
    rows, n, ld = 70, 100, 128
    full = torch.randn(rows, ld, generator=g).cuda()
    full[:, n:] = 50.0  # what lies behind the experts is not read
    ids = torch.empty(rows, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(rows, 8, device="cuda")
    gr = torch.cuda.CUDAGraph()
    api.dsa_route(full, 8, ids, w, n_experts=n)
    with torch.cuda.graph(gr):
        api.dsa_route(full, 8, ids, w, n_experts=n)
    full.copy_(full.flip(0))
    gr.replay()
    torch.cuda.synchronize()
    want = _route_ref(full[:, :n], 8, None, "sigmoid", 1, 1, 1, True, 1.0, 0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want[0])
    np.testing.assert_allclose(w.cpu().numpy(), want[1], rtol=W_TOL)


@pytest.mark.parametrize("rows,hidden,n", [(1, 256, 64), (5, 1024, 128), (70, 512, 256), (200, 768, 192)])
def test_router_logits(rows, hidden, n):
    x, w = _rows(20, rows, hidden), _rows(21, n, hidden)
    logits = torch.full((rows, n), math.nan, device="cuda")
    ws = torch.zeros(max(1, api.dsa_router_logits_workspace(rows, hidden, n)), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_router_logits(x, w, logits, status, ws)
    a, b = x.double(), w.double()
    # products are exact in f32; a sum of `hidden` of them in any order is off by at most
    # hidden * 2^-24 of the sum of magnitudes (twice that for a truncating accumulator)
    bound = 2 * hidden * 2.0 ** -24 * (a.abs() @ b.abs().T)
    assert bool(((logits.double() - a @ b.T).abs() <= bound).all()) and int(status) == 0
