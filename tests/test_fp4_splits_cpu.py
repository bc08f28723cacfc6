"""dsa_sparse_mla_decode_fp4_splits without a GPU: its refusals."""
import ctypes

import pytest

from sparse_attention_decode_kpool_gb300 import _build, _lib
from sparse_attention_decode_kpool_gb300._lib import (DSA_ERR_CONFIG, DSA_ERR_INVALID_ARG,
                                                      DSA_ERR_UNSUPPORTED)


@pytest.mark.parametrize("a,code", [((-1, 8, 512, 64), DSA_ERR_INVALID_ARG),
                                    ((4, 0, 512, 64), DSA_ERR_INVALID_ARG),
                                    ((4, 8, 512, -1), DSA_ERR_INVALID_ARG),
                                    ((4, 8, 0, 64), DSA_ERR_CONFIG),
                                    ((4, 8, 576, 64), DSA_ERR_UNSUPPORTED),
                                    ((65536, 8, 512, 64), DSA_ERR_UNSUPPORTED)])
def test_splits_refusals(a, code):
    _build.build()
    lib = _lib.load()
    n = ctypes.c_int(0)
    assert lib.dsa_sparse_mla_decode_fp4_splits(*a, 1000, ctypes.byref(n)) == code
    assert lib.dsa_sparse_mla_decode_fp4_splits(4, 8, 512, 64, 1000, None) == DSA_ERR_INVALID_ARG
