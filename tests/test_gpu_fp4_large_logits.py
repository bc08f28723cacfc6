"""FP4 attention with logits far beyond the range of a softmax's weights: the result is the
row of the token with the largest logit, as for any other one-hot softmax."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import api
from tests import _harness as H
from tests.test_gpu_fp4 import KERNELS, KVL, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def run_f32(c, which):
    with api.mla_kernel(which):
        c.cuda()
        out = torch.empty((c.rows, c.heads, KVL), dtype=torch.float32, device="cuda")
        c.run(out)
        torch.cuda.synchronize()
        assert int(c.status) == 0
        return out.double().cpu().numpy()


def check_one_hot(c, got, heads):
    """The listed heads' results, wherever the best logit leads the next by 30 more than the
    two logits' f32 error (2^-17 scale sum |q v| each; doubled here): the best token's row, up
    to a weight of 2^-43 for each other token and to p / sum(p), which is one token's weight
    over itself: the weight in the product is rounded to f16 (eleven bits: half a step is
    2^-11 of a weight just above a power of two), the sum of the tensor-core kernel takes it
    unrounded; ex2 (2^-22, twice), the sum, the quotient and the result's own rounding (2^-24
    each) add less than 2^-20. Returns how many
    results were compared."""
    q = H.f(c.q).reshape(c.rows, c.heads, KVL)
    checked = 0
    for r in range(c.rows):
        _, rows = c.at(r)
        v = O.dequantize_latent_fp4(c.codes[rows], c.scales[rows], c.exp)
        s = c.scale * (q[r] @ v.T)
        delta = c.scale * 2.0 ** -17 * (np.abs(q[r]) @ np.abs(v).T)
        for h in heads:
            k = int(np.argmax(s[h]))
            rest = rows != rows[k]  # a token may be selected twice
            if (s[h, k] - s[h, rest] > 30 + 2 * (delta[h, k] + delta[h, rest])).all():
                tol = (2.0 ** -11 + 2.0 ** -20) * np.abs(v[k]) + len(rows) * 2.0 ** -43 * np.abs(v).max()
                assert (np.abs(got[r, h] - v[k]) <= tol).all(), (r, h, got[r, h, :3], v[k, :3])
                checked += 1
    return checked


@pytest.mark.parametrize("order", [0, 1, -1], ids=["any", "rising", "falling"])
@pytest.mark.parametrize("power", [10, 16, 20, 23, 25, 27, 29, 31, 40, 60, 100])
def test_large_logits(power, order):
    """Logits of about 2^power, in one split and in several; in any order, and sorted by a
    head's logits so that the running maximum moves at every chunk, or never."""
    for ow in (150, 600):
        c = Case(83, 2, 64, ow, [700], hole=0.1, q_mul=1.0)
        c.q = torch.from_numpy(H.f(c.q) * 2.0 ** power).to(torch.bfloat16)
        if order:
            q = H.f(c.q).reshape(2, 64, KVL)
            for r in range(2):
                t, rows = c.at(r)
                v = O.dequantize_latent_fp4(c.codes[rows], c.scales[rows], c.exp)
                c.ids[r, c.ids[r] >= 0] = t[np.argsort(order * (q[r, 5] @ v.T), kind="stable")]
        for which in KERNELS:
            got = run_f32(c, which)
            assert np.isfinite(got).all(), which
            assert check_one_hot(c, got, range(64)) >= 64


@pytest.mark.parametrize("order", ["low first", "low last", "mixed", "low only"])
@pytest.mark.parametrize("rows", [2, 160], ids=["splits", "one split"])
def test_logits_that_overflow_downwards(rows, order):
    """Logits below f32's lowest number have no weight, wherever they stand in the list. One
    channel of q counts: tokens with -1 there have a logit of -5e39, the others of 0 and so
    equal weights (a power of two each: their mean, up to the f32 sums of at most 300 terms).
    With no other token the sum of the weights is 0, and so is the result."""
    c = Case(91, rows, 64, 600, [600], hole=0.0, exp=-8, scale=16.0)
    x = np.random.default_rng(92).normal(0, 1, (600, KVL))
    low = np.arange(600) < 300
    x[:, 0] = np.where(low, -1.0, 0.0)
    c.codes, c.scales = O.quantize_latent_fp4(H.f(torch.from_numpy(x).to(torch.bfloat16)), -8)
    v = O.dequantize_latent_fp4(c.codes, c.scales, -8)
    ids = np.arange(600)
    if order == "low last":
        ids = ids[::-1].copy()
    elif order == "mixed":
        ids = np.random.default_rng(93).permutation(600)
    elif order == "low only":
        ids[300:] = -1
    c.ids[:] = ids
    q = torch.zeros((rows, 64, KVL), dtype=torch.bfloat16)
    q[:, :, 0] = 3e38
    c.q = q
    want = np.zeros(KVL) if order == "low only" else v[~low].mean(0)
    tol = 300 * 2.0 ** -22 * np.abs(v[~low]).mean(0)
    for which in KERNELS:
        got = run_f32(c, which)
        assert (np.abs(got - want) <= tol).all(), (which, got[0, 0, :4], want[:4])
