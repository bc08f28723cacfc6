"""dsa_router_logits over a prefill chunk's rows, and what dsa_route makes of them."""
import math

import numpy as np
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from tests import test_gpu_layer_ops as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("rows,hidden,n", [(64, 4096, 256), (65, 4096, 256), (1999, 2048, 64), (4096, 4096, 256)])
def test_many_rows(rows, hidden, n):
    x, w = L._rows(51, rows, hidden), L._rows(52, n, hidden, std=hidden ** -0.5)
    logits = torch.full((rows, n), math.nan, device="cuda")
    ws = torch.full((max(1, api.dsa_router_logits_workspace(rows, hidden, n)),), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_router_logits(x, w, logits, status, ws)
    a, b = x.double(), w.double()
    # as in the test of few rows: exact products, f32 sums in any order, an accumulator that truncates
    bound = 2 * hidden * 2.0 ** -24 * (a.abs() @ b.abs().T)
    assert bool(((logits.double() - a @ b.T).abs() <= bound).all()) and int(status) == 0
    ids = torch.empty(rows, 4, dtype=torch.int32, device="cuda")
    wt = torch.empty(rows, 4, device="cuda")
    api.dsa_route(logits, 4, ids, wt)
    want = L._route_ref(logits, 4, None, "sigmoid", 1, 1, 1, True, 1.0, 0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want[0])
    np.testing.assert_allclose(wt.cpu().numpy(), want[1], rtol=L.W_TOL)
