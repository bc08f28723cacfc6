"""Refusals of the layer's other half (dsa_rmsnorm, dsa_dequantize_latent, dsa_route,
dsa_router_logits): host-visible errors before anything touches CUDA, and the binding's own
checks of shapes."""
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import _build, _lib, api
from sparse_attention_decode_kpool_gb300._lib import (DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED,
                                                       DSA_OK)

FAKE = 0x10000  # a non-NULL device address the host never dereferences
FAR = 0x4000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def _err(lib):
    return lib.dsa_last_error().decode()


def test_rmsnorm_refusals(lib):
    def call(x=FAKE, res=None, w=FAR, rows=4, width=256, eps=1e-6, ro=None, out=2 * FAR, codes=None,
             scales=None):
        return lib.dsa_rmsnorm(x, res, w, rows, width, eps, ro, out, codes, scales, None)

    assert call(rows=0) == DSA_OK
    assert call(rows=-1) == DSA_ERR_INVALID_ARG
    assert call(width=0) == DSA_ERR_INVALID_ARG
    assert call(width=(1 << 24) + 128) == DSA_ERR_UNSUPPORTED
    assert call(rows=1 << 31) == DSA_ERR_UNSUPPORTED
    assert call(eps=-1e-6) == DSA_ERR_INVALID_ARG and "eps" in _err(lib)
    assert call(eps=float("nan")) == DSA_ERR_INVALID_ARG
    assert call(x=None) == DSA_ERR_INVALID_ARG
    assert call(w=None) == DSA_ERR_INVALID_ARG
    assert call(out=None) == DSA_ERR_INVALID_ARG and "neither" in _err(lib)
    assert call(codes=3 * FAR) == DSA_ERR_INVALID_ARG and "together" in _err(lib)
    assert call(scales=3 * FAR) == DSA_ERR_INVALID_ARG
    assert call(ro=3 * FAR) == DSA_ERR_INVALID_ARG and "residual" in _err(lib)
    assert call(width=200, codes=3 * FAR, scales=4 * FAR) == DSA_ERR_UNSUPPORTED
    assert call(codes=3 * FAR, scales=4 * FAR + 2) == DSA_ERR_INVALID_ARG
    # overlaps: shifted by a row, an output on the weight, two outputs on one another
    n = 4 * 256 * 2
    assert call(out=FAKE + 512) == DSA_ERR_INVALID_ARG and "overlaps" in _err(lib)
    assert call(out=FAKE - 512) == DSA_ERR_INVALID_ARG
    assert call(out=FAR) == DSA_ERR_INVALID_ARG
    assert call(res=3 * FAR, ro=3 * FAR + 16) == DSA_ERR_INVALID_ARG
    assert call(res=3 * FAR, ro=2 * FAR) == DSA_ERR_INVALID_ARG and "two outputs" in _err(lib)
    assert call(codes=FAKE + n - 16, scales=4 * FAR) == DSA_ERR_INVALID_ARG
    assert call(codes=FAKE, scales=4 * FAR) == DSA_ERR_INVALID_ARG  # not element for element


def test_dequantize_latent_refusals(lib):
    def call(codes=FAKE, scales=FAR, cache=8, ids=None, rows=8, kvl=512, out=2 * FAR):
        return lib.dsa_dequantize_latent(codes, scales, cache, ids, rows, kvl, out, None, None)

    assert call(rows=0) == DSA_OK
    assert call(rows=-1) == DSA_ERR_INVALID_ARG
    assert call(kvl=64) == DSA_ERR_INVALID_ARG
    assert call(kvl=200) == DSA_ERR_INVALID_ARG
    assert call(rows=9) == DSA_ERR_INVALID_ARG and "cache of 8" in _err(lib)
    assert call(cache=-1, ids=FAR) == DSA_ERR_INVALID_ARG
    assert call(codes=None) == DSA_ERR_INVALID_ARG
    assert call(out=2 * FAR + 8) == DSA_ERR_INVALID_ARG and "aligned" in _err(lib)
    assert call(ids=FAR, rows=1 << 31) == DSA_ERR_UNSUPPORTED


def test_route_refusals(lib):
    def call(logits=FAKE, rows=2, n=64, ld=64, score=0, bias=None, groups=1, tg=1, gt=2, k=8,
             renorm=1, scale=1.0, shared=0, ids=FAR, w=2 * FAR):
        return lib.dsa_route(logits, rows, n, ld, score, bias, groups, tg, gt, k, renorm, scale,
                             shared, ids, w, None)

    assert call(rows=0) == DSA_OK
    for bad in (dict(rows=-1), dict(n=0), dict(ld=63), dict(k=0), dict(shared=-1), dict(score=2),
                dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=4, tg=5),
                dict(groups=4, tg=0), dict(gt=0), dict(gt=3), dict(groups=64, tg=64, n=64, gt=2),
                dict(k=65), dict(n=4, ld=4, k=5), dict(groups=8, tg=1, k=9),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(logits=None),
                dict(ids=None), dict(w=None), dict(ids=FAR + 2), dict(logits=FAKE + 1)):
        rc = call(**bad)
        assert rc in (DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED), bad
        assert "dsa_route" in _err(lib), bad
    assert call(n=1025, ld=1025) == DSA_ERR_UNSUPPORTED
    assert call(n=1024, ld=1024, k=65) == DSA_ERR_UNSUPPORTED
    assert call(n=66, ld=66, groups=33, tg=8) == DSA_ERR_UNSUPPORTED


def test_router_logits_refusals(lib):
    def call(x=FAKE, rows=2, hidden=512, w=FAR, n=64, out=2 * FAR):
        return lib.dsa_router_logits(x, rows, hidden, w, n, out, None, None, 0, None)

    assert call(rows=0) == DSA_OK
    assert call(rows=-1) == DSA_ERR_INVALID_ARG
    assert call(hidden=500) == DSA_ERR_UNSUPPORTED
    assert call(n=60) == DSA_ERR_UNSUPPORTED and "zeros" in _err(lib)
    assert call(x=None) == DSA_ERR_INVALID_ARG
    assert call(w=FAR + 8) == DSA_ERR_INVALID_ARG
    assert lib.dsa_router_logits_workspace(2, 512, 64, None) == DSA_ERR_INVALID_ARG


def test_binding_checks_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="weight"):
        api.dsa_rmsnorm(x, w[:128], 1e-6, x)
    with pytest.raises(ValueError, match="out, residual"):
        api.dsa_rmsnorm(x, w, 1e-6, x[:2])
    with pytest.raises(ValueError, match="codes"):
        api.dsa_rmsnorm(x, w, 1e-6, x, codes=torch.zeros(4, 256, dtype=torch.uint8),
                        scales=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_rmsnorm(x, w, 1e-6, x)
    logits = torch.zeros(4, 64)
    ids, wt = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score"):
        api.dsa_route(logits, 8, ids, wt, score="relu")
    with pytest.raises(ValueError, match="bias"):
        api.dsa_route(logits, 8, ids, wt, bias=torch.zeros(63))
    with pytest.raises(ValueError, match="of 65 experts"):
        api.dsa_route(logits, 8, ids, wt, n_experts=65)
    with pytest.raises(ValueError, match="ids and weights"):
        api.dsa_route(logits, 8, ids, wt, shared=1)
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_route(logits, 8, ids, wt)
    codes = torch.zeros(4, 256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="multiple of 128"):
        api.dsa_dequantize_latent(codes, torch.zeros(4, 1), x)
    with pytest.raises(ValueError, match="cache's 4 rows"):
        api.dsa_dequantize_latent(codes, torch.zeros(4, 2), x[:3])
    with pytest.raises(ValueError, match="logits"):
        api.dsa_router_logits(x, torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(4, 63))


def test_experts_refusals(lib):
    import ctypes

    need = ctypes.c_size_t(0)
    assert lib.dsa_experts_workspace(8, 2, 4, 256, 128, 0, ctypes.byref(need)) == DSA_OK
    bf16_bytes = need.value
    assert bf16_bytes >= 16 * (256 * 2 + 128 * 2)
    assert lib.dsa_experts_workspace(8, 2, 4, 256, 128, 1, ctypes.byref(need)) == DSA_OK
    assert lib.dsa_experts_workspace(8, 2, 4, 256, 128, 0, None) == DSA_ERR_INVALID_ARG

    def call(x=FAKE, xs=None, rows=8, hidden=256, ids=FAR, w=FAR, topk=2, w13=FAR, s13=None, w2=FAR,
             s2=None, n=4, inter=128, y=FAR, ws=FAR, nbytes=1 << 30):
        return lib.dsa_experts(x, xs, rows, hidden, ids, w, topk, w13, s13, w2, s2, n, inter, y, None,
                               ws, nbytes, None)

    assert call(rows=0) == DSA_OK
    for bad in (dict(rows=-1), dict(topk=0), dict(n=0), dict(hidden=0), dict(inter=0), dict(x=None),
                dict(ids=None), dict(w=None), dict(w13=None), dict(w2=None), dict(y=None),
                dict(ws=None), dict(nbytes=bf16_bytes - 1), dict(x=FAKE + 8), dict(y=FAR + 2),
                dict(ids=FAR + 2), dict(xs=FAR), dict(s13=FAR, s2=FAR), dict(xs=FAR, s13=FAR, s2=FAR + 1)):
        assert call(**bad) == DSA_ERR_INVALID_ARG, bad
        assert "dsa_experts" in _err(lib), bad
    for bad in (dict(hidden=192), dict(inter=64), dict(inter=200), dict(n=1089),
                dict(rows=1 << 20, topk=64), dict(inter=65664), dict(hidden=65664)):
        assert call(**bad) == DSA_ERR_UNSUPPORTED, bad


def test_experts_binding_checks():
    bf16, u8 = torch.bfloat16, torch.uint8
    x, y = torch.zeros(4, 256, dtype=bf16), torch.zeros(4, 256, dtype=bf16)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w13, w2 = torch.zeros(3, 256, 256, dtype=bf16), torch.zeros(3, 256, 128, dtype=bf16)
    with pytest.raises(ValueError, match="w13"):
        api.dsa_experts(x, ids, w, w13[:, :128], w2, y)
    with pytest.raises(ValueError, match="weights"):
        api.dsa_experts(x, ids, w[:, :1], w13, w2, y)
    with pytest.raises(ValueError, match="y must"):
        api.dsa_experts(x, ids, w, w13, w2, y[:2])
    with pytest.raises(ValueError, match="FP8 takes"):
        api.dsa_experts(x, ids, w, w13, w2, y, x_scales=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="scales must"):
        api.dsa_experts(x, ids, w, w13, w2, y, x_scales=torch.zeros(4, 2),
                        w13_scales=torch.zeros(3, 256, 2), w2_scales=torch.zeros(3, 256, 2))
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_experts(x, ids, w, w13, w2, y)
