"""dsa_experts: a row's products keep f32's digits until they are summed, also where they cancel."""
import math

import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from tests.test_gpu_experts import BF16, _encode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _call(x, ids, weights, w13, w2, fp8):
    (n, hidden, inter), rows = w2.shape, x.shape[0]
    y = torch.full((rows, hidden), math.nan, dtype=BF16, device="cuda")
    need = api.dsa_experts_workspace(rows, ids.shape[1], n, hidden, inter, fp8)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        (x, xs), (w13, s13), (w2, s2) = _encode(x), _encode(w13), _encode(w2)
        api.dsa_experts(x, ids, weights, w13, w2, y, xs, s13, s2, status=status, workspace=ws)
    else:
        api.dsa_experts(x, ids, weights, w13, w2, y, status=status, workspace=ws)
    assert int(status) == 0
    return y.double()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [3, 12, 40, 90, 300])  # two experts a row: every pair-tile size
def test_products_that_cancel(rows, fp8):
    """Expert 0's second product is h_c + h_d / 64 for channel c (d another one), expert 1's is -h_c, of
    the same h. Their sum is h_d / 64, of which 11 bits of the products would leave little.

    h_d has bf16's 8 bits or fewer, so y = h_d / 128 needs no rounding of its own. The product and the sum
    may be off by 2^-23 of |h_c| + |h_d| / 64 each (an accumulator that truncates), halved by the
    weights; where that reaches half a step of y, y's rounding can add as much again. h itself is read off by a third
    expert whose second product is the identity, of one summand and exact."""
    hidden = inter = 256
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, hidden, generator=g).to(BF16).cuda()
    w13 = (torch.randn(1, 2 * inter, hidden, generator=g) * hidden ** -0.5).to(BF16).cuda()
    one = torch.eye(hidden, device="cuda")
    other = (torch.arange(hidden, device="cuda") * 77 + 5) % hidden
    w2 = torch.stack([one + one[other] / 64, -one]).to(BF16).contiguous()
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(rows, 1)
    half = torch.full((rows, 2), 0.5, device="cuda")
    got = _call(x, ids, half, w13.repeat(2, 1, 1), w2, fp8)
    h = _call(x, ids[:, :1].contiguous(), 2 * half[:, :1].contiguous(), w13, one.to(BF16)[None].contiguous(), fp8)
    want = h[:, other] / 128
    off = 2.0 ** -23 * (h.abs() + h[:, other].abs() / 64)
    err = (got - want).abs()
    assert bool((err <= 2 * off).all()), (float((err / off).max()), int((err > 2 * off).sum()))
