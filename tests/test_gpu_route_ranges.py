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
