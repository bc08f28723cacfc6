"""FP4 attention whose heads differ by many powers of two: each head's logits are its own,
whatever is in the heads beside it."""
import numpy as np
import pytest
import torch

from tests import _harness as H
from tests.test_gpu_fp4 import KERNELS, KVL, Case
from tests.test_gpu_fp4_large_logits import check_one_hot, run_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _check_heads(c, got, heads):
    """The listed heads against their definition, with the tolerance of the heads alone."""
    q, n = c.q, c.heads
    c.q, c.heads = q[:, heads], len(heads)
    want, tol = c.want()
    c.q, c.heads = q, n
    err, bound = np.abs(got[:, heads] - want), tol + 2.0 ** -23 * np.abs(want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-30)).max())


@pytest.mark.parametrize("loud", [31, 35, 39, 60, 100])
@pytest.mark.parametrize("heads", [16, 24, 64, 80])
def test_loud_heads_beside_quiet_ones(heads, loud):
    """Every third head 2^loud above the others. Those keep logits of order one; the loud
    ones are one-hot."""
    c = Case(71, 2, heads, 150, [300], hole=0.1)
    q = H.f(c.q).reshape(2, heads, KVL)
    big = np.arange(heads) % 3 == 1
    q[:, big] *= 2.0 ** loud
    c.q = torch.from_numpy(q).to(torch.bfloat16)  # exact: a power of two
    for which in KERNELS:
        got = run_f32(c, which)
        _check_heads(c, got, np.flatnonzero(~big))
        assert check_one_hot(c, got, np.flatnonzero(big)) >= big.sum()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3e38, -3e38])
def test_one_head_out_of_range(value):
    """A head with an infinity, a NaN or bf16's largest values changes no other head."""
    c = Case(73, 3, 64, 200, [400], hole=0.1)
    c.q[:, 7, 100] = value
    others = np.flatnonzero(np.arange(64) != 7)
    for which in KERNELS:
        _check_heads(c, run_f32(c, which), others)


@pytest.mark.parametrize("heads", [16, 64])
def test_every_head_its_own_magnitude(heads):
    """Heads from 2^-60 to 2^60, each alone in its magnitude, equal bit for bit to the same
    heads at one magnitude under a scale that undoes the factor, head by head."""
    c = Case(79, 2, heads, 130, [200], hole=0.1)
    e = np.linspace(-60, 60, heads).astype(int)
    q = H.f(c.q).reshape(2, heads, KVL)
    mixed = torch.from_numpy(q * np.exp2(e)[:, None]).to(torch.bfloat16)
    for which in KERNELS:
        for h in (0, heads // 3, heads - 1):
            c.q, c.scale = mixed, 2.0 ** (-4 - e[h])
            a = run_f32(c, which)[:, h]
            c.q, c.scale = torch.from_numpy(q).to(torch.bfloat16), 2.0 ** -4
            b = run_f32(c, which)[:, h]
            np.testing.assert_array_equal(a, b)


def test_units_of_both_kinds():
    """More rows than SMs, several units per CTA and several chunks per unit, every fifth row
    with heads far apart: units with one power of two and with one per head follow one
    another in a CTA."""
    c = Case(89, 330, 64, 300, [500], hole=0.1)
    q0 = c.q
    q = H.f(c.q).reshape(330, 64, KVL)
    for r in range(0, 330, 5):
        q[r, r % 64] *= 2.0 ** 45
    c.q = torch.from_numpy(q).to(torch.bfloat16)
    got = run_f32(c, "tcgen05")
    c.rows, sub = 30, np.arange(0, 330, 11)  # rows of either kind
    c.q, c.ids, c.row_seq = q0[sub], c.ids[sub], c.row_seq[sub]
    loud = np.array([(r % 64 if r % 5 == 0 else -1) for r in sub])
    want, tol = c.want()
    bound = tol + 2.0 ** -23 * np.abs(want)
    ok = np.abs(got[sub] - want) <= bound
    ok[np.flatnonzero(loud >= 0), loud[loud >= 0]] = True  # the heads that q0 has not
    assert ok.all()
