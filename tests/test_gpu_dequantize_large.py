"""dsa_dequantize_latent on both sides of its size rule."""
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_TOKEN

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# 16-byte pieces of codes: 4,915,200, 5,120,000 and 5,111,832 around 16 x 2,048 x 152 = 4,980,736
@pytest.mark.parametrize("rows,width", [(19200, 4096), (20000, 4096), (212993, 384)])
@pytest.mark.parametrize("named", [False, True])
def test_many_rows(rows, width, named):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, width // 128, device="cuda")
    api.dsa_quantize_latent(x, codes, scales)
    want = codes.view(torch.float8_e4m3fn).float().view(rows, -1, 128) * scales.unsqueeze(-1)
    want = want.view(rows, width).to(torch.bfloat16)  # exact: 4 bits under a power of two
    out = torch.full((rows, width), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = None
    if named:
        ids = torch.randint(0, rows, (rows,), generator=g, device="cuda", dtype=torch.int32)
        ids[[1, rows // 2, rows - 1]] = torch.tensor([-1, rows, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        ok = (ids >= 0) & (ids < rows)
        want = torch.where(ok[:, None], want[torch.where(ok, ids, 0).long()], torch.zeros_like(want))
    api.dsa_dequantize_latent(codes, scales, out, rows=ids, status=status)
    assert torch.equal(out, want)
    assert int(status) == (DSA_STATUS_BAD_TOKEN if named else 0)
