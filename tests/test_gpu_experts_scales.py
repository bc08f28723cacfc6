"""dsa_experts reads the exponents of FP8 scales: one that is no power of two is reported."""
import math

import pytest
import torch

from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_SCALE
from tests.test_gpu_experts import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("rows", [4, 30, 90, 170, 330])  # every pair-tile size
def test_scales_that_are_no_powers_of_two(rows):
    p = Problem(rows, rows, 5, 1, 384, 256, True)
    p.ids[:, 0] = torch.arange(rows, device="cuda") % 3  # experts 3 and 4 are nobody's
    p.ids[-1] = -1
    p.run()
    p.check()
    assert int(p.status) == 0

    def status_with(t, at, value):
        before = t[at].clone()
        t[at] = value(before) if callable(value) else value
        p.status.zero_()
        p.run()
        t[at] = before
        return int(p.status)

    last = (0, 0, -1), (2, -1, 1)
    for t, places in ((p.xs, ((0, 1), (rows - 2, 2))), (p.s13, last), (p.s2, last)):
        for at in places:
            assert status_with(t, at, lambda v: v * 1.5) == DSA_STATUS_BAD_SCALE
            assert status_with(t, at, lambda v: v * (1 + 2.0 ** -23)) == DSA_STATUS_BAD_SCALE
            assert status_with(t, at, lambda v: -v) == DSA_STATUS_BAD_SCALE
            for quiet in (math.nan, math.inf, 0.0, 2.0 ** -126, 2.0 ** 127):
                assert status_with(t, at, quiet) == 0
    for t in (p.s13, p.s2):  # not read: nobody chose expert 3
        assert status_with(t, (3, 0, 0), 1.5) == 0
    p.status.zero_()
    p.run()
    p.check()
    assert int(p.status) == 0
