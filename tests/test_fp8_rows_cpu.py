"""The binding's checks of FP8 rows that have no width or no row."""
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api


def test_rows_without_width_are_refused():
    codes, scales = torch.zeros(4, 0, dtype=torch.uint8), torch.zeros(4, 0)
    out = torch.zeros(4, 0, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiple of 128"):
        api.dsa_dequantize_latent(codes, scales, out)
    with pytest.raises(ValueError):
        api.dsa_rmsnorm(out, out[0], 1e-6, codes=codes, scales=scales)


def test_no_rows_is_no_call():
    codes, scales = torch.zeros(0, 256, dtype=torch.uint8), torch.zeros(0, 2)
    api.dsa_dequantize_latent(codes, scales, torch.zeros(0, 256, dtype=torch.bfloat16))
