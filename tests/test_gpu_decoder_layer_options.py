"""The layer's router takes every option of dsa_route, and refuses at its construction what that refuses."""
import dataclasses

import numpy as np
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import workloads as W
from sparse_attention_decode_kpool_gb300._lib import DsaError
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer
from tests import test_gpu_layer_ops as L

pytestmark = pytest.mark.gpu
GEOM = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8, hidden=512)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_layer_routes_by_its_options(group_top, renorm, score):
    rows = 24
    wl = W.make_workload("decoder", 81, GEOM, [100] * rows)
    ex = W.make_experts(GEOM, rows, 24, 3, 128, seed=82, n_group=6, topk_group=1, score=score, group_top=group_top,
                        renorm=renorm)
    lay = DsaDecodeLayer(wl, experts=ex)
    lay.compress()
    lay.step()
    lay.mlp()
    args = lay.logits[:, :24], 3, lay.route_bias, score, 6, 1
    ids, w = L._route_ref(*args, group_top, renorm, ex.scale, ex.shared)
    np.testing.assert_array_equal(lay.expert_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(lay.expert_weights.cpu().numpy(), w, rtol=L.W_TOL, atol=1e-37)
    # the options decide something here
    assert (ids != L._route_ref(*args, 3 - group_top, renorm, ex.scale, ex.shared)[0]).any()
    assert (w != L._route_ref(*args, group_top, not renorm, ex.scale, ex.shared)[1]).any()


def test_a_group_for_each_expert():
    wl = W.make_workload("decoder", 83, GEOM, [100] * 5)
    ex = W.make_experts(GEOM, 5, 16, 3, 128, seed=84, n_group=16, topk_group=3, group_top=1)
    lay = DsaDecodeLayer(wl, experts=ex)
    lay.compress()
    lay.step()
    lay.mlp()
    ids, w = L._route_ref(lay.logits[:, :16], 3, lay.route_bias, "sigmoid", 16, 3, 1, True, ex.scale, ex.shared)
    np.testing.assert_array_equal(lay.expert_ids.cpu().numpy(), ids)


def test_refused_at_construction():
    wl = W.make_workload("decoder", 85, GEOM, [100] * 2)
    ex = W.make_experts(GEOM, 2, 16, 3, 128, n_group=4, topk_group=2)
    for bad in (dict(group_top=3), dict(n_group=16, topk_group=3), dict(n_group=5), dict(topk=9), dict(topk_group=5)):
        with pytest.raises(DsaError, match="dsa_route"):
            DsaDecodeLayer(wl, experts=dataclasses.replace(ex, **bad))
    with pytest.raises(ValueError, match="score"):
        DsaDecodeLayer(wl, experts=dataclasses.replace(ex, score="relu"))
    with pytest.raises(ValueError, match="bias"):
        DsaDecodeLayer(wl, experts=dataclasses.replace(ex, bias=ex.bias[:15]))
    with pytest.raises(ValueError, match="shared"):
        DsaDecodeLayer(wl, experts=dataclasses.replace(ex, shared=2))
