"""dsa_route where f32 scores and factors run short of digits or of range: the choice and the weights
are those of 64 bits there too."""
import pytest
import torch

from tests.test_gpu_layer_ops import _check_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("mean", [-1, -8, -20, -30, -40, -60, -68, -85])
def test_groups_nearly_alike_far_below_zero(mean):
    """The sigmoid's argument z log2(e) is rounded, so an f32 score is off by |z| times as much as one near
    zero, and the groups' sums with it."""
    g = torch.Generator().manual_seed(-mean)
    z = mean + 1e-5 * torch.randn(4000, 16, generator=g)
    _check_route(z.cuda(), 4, None, "sigmoid", 2, 1, 2, True, 0)
    _check_route(z[:500].cuda(), 3, None, "sigmoid", 4, 2, 1, True, 0)
    z = mean + 0.01 * torch.randn(500, 256, generator=g)
    _check_route(z.cuda(), 8, None, "sigmoid", 8, 4, 2, True, 0)


@pytest.mark.parametrize("score,mean,scale,renorm", [
    ("sigmoid", -65.0, 1e12, True),    # 1e12 over a sum of 1e-28 passes f32's largest, the weights do not
    ("sigmoid", -65.0, -1e12, True),
    ("sigmoid", -95.0, 1e30, False),   # scores below f32's smallest, scaled into its range
    ("sigmoid", -89.0, 2.5, False),
    ("softmax", -60.0, 1e30, False),
    ("sigmoid", 0.0, 3e38, True),
    ("sigmoid", -20.0, 1e-30, True),
])
def test_weights_under_large_scales(score, mean, scale, renorm):
    g = torch.Generator().manual_seed(17)
    z = mean + torch.randn(50, 64, generator=g)
    if score == "softmax":
        z[:, 9] = 40.0  # the others' shares are near 1e-44
    _check_route(z.cuda(), 8, None, score, 1, 1, 1, renorm, 0, scale=scale)
    _check_route(z.cuda(), 8, None, score, 4, 2, 2, renorm, 1, scale=scale)
