"""dsa_rmsnorm of rows whose squares f32 does not hold, with an eps that leaves them."""
import math

import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from tests.test_gpu_layer_ops import BF16, NORM_TOL, _close, _norm_ref, _rows

pytestmark = pytest.mark.gpu
TOL = NORM_TOL + 2.0 ** -24  # and v's own rounding to f32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# every kernel variant: rows a warp, rows a team of warps, a row a block; any width
WIDTHS = [8, 250, 256, 512, 1000, 1024, 2048, 4096, 8192, 16384, 32768, 40000]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-39, 1e-33, 1e-27])
def test_small_rows(width, eps):
    """Rows from 2^-20 down to the smallest subnormals, side by side with ordinary ones. (v, a sum of two
    bf16 values below 2^-126, is exact; out is the formula's value rounded as ever.)"""
    exps = [0, -20, -40, -47, -48, -49, -56, -60, -64, -66, -72, -80, -100, -120, -127, -131]
    x, res, w = _rows(41, len(exps), width), _rows(42, len(exps), width), _rows(43, width)
    by = torch.tensor([2.0 ** e for e in exps], dtype=torch.float64, device="cuda")[:, None]
    x, res = (x.double() * by).to(BF16), (res.double() * by).to(BF16)
    out, ro = torch.full_like(x, math.nan), torch.full_like(x, math.nan)
    api.dsa_rmsnorm(x, w, eps, out, residual=res, residual_out=ro)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    v, want = _norm_ref(x, res, w, eps)
    assert torch.equal(ro, v.float().to(BF16))
    some = v.abs().amax(1) > 0  # (0 times the root of 1/0 is NaN, as the formula's)
    _close(out[some], want[some], TOL)
    if eps == 0:
        assert bool(torch.isnan(out[~some]).all())
    # in place: both outputs over the inputs
    xa, ra = x.clone(), res.clone()
    api.dsa_rmsnorm(xa, w, eps, xa, residual=ra, residual_out=ra)
    assert torch.equal(xa[some], out[some]) and torch.equal(ra, ro)


@pytest.mark.parametrize("width", [128, 640, 4096, 33024])
def test_small_rows_as_fp8(width):
    x, w = _rows(44, 9, width), _rows(45, width)
    x = (x.double() * 2.0 ** -70).to(BF16)
    x[4] = 1.0
    out = torch.empty_like(x)
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(9, width // 128, device="cuda")
    api.dsa_rmsnorm(x, w, 0.0, out, codes=codes, scales=scales)
    _close(out, _norm_ref(x, None, w, 0.0)[1], TOL)
    want = torch.empty_like(codes), torch.empty_like(scales)
    api.dsa_quantize_latent(out, *want)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
