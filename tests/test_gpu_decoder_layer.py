"""The whole decoder layer: input norm, front-end, append, step, norm, router, experts. Each
operator of the second half is checked against a 64-bit restatement on the layer's own
tensors, and a captured layer against the same calls made eagerly."""
import numpy as np
import pytest
import torch

from sparse_attention_decode_kpool_gb300 import workloads as W
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer
from tests import test_gpu_experts as E, test_gpu_layer_ops as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _layer(seed, n_experts=12, topk=3, inter=256, rows=(300, 517, 77), n_group=3, topk_group=2, shared=1,
           fp8=False, **kw):
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8, hidden=512)
    wl = W.make_workload("decoder", seed, g, list(rows))
    fe = W.make_frontend(g, wl.rows, q_lora_rank=512, seed=seed + 1)
    ex = W.make_experts(g, wl.rows, n_experts, topk, inter, seed=seed + 2, n_group=n_group, topk_group=topk_group,
                        shared=shared)
    layer = DsaDecodeLayer(wl, keep_olat=True, decode_from=wl.seq_lens.astype(np.int64) - 4, frontend=fe, experts=ex,
                           experts_fp8=fp8, **kw)
    layer.compress()
    return layer


def _check_mlp(lay, resid_before):
    """The second half on the layer's own y."""
    ex = lay.ex
    v, want = L._norm_ref(lay.y, resid_before, lay.mlp_norm, ex.eps)
    assert torch.equal(lay.resid, v.float().to(torch.bfloat16))
    L._close(lay.mlp_x, want, L.NORM_TOL)
    a, b = lay.mlp_x.double(), lay.w_router.double()
    bound = 2 * a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs().T)
    assert bool(((lay.logits.double() - a @ b.T).abs() <= bound).all())
    ids, w = L._route_ref(lay.logits[:, :ex.n_experts], ex.topk, lay.route_bias, ex.score, ex.n_group, ex.topk_group,
                          2, True, ex.scale, ex.shared)
    np.testing.assert_array_equal(lay.expert_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(lay.expert_weights.cpu().numpy(), w, rtol=L.W_TOL, atol=1e-37)
    p = E.Problem.__new__(E.Problem)
    p.rows, p.hidden, p.inter, p.n, p.k, p.fp8 = (lay.wl.rows, lay.geom.hidden, ex.inter, lay.w2.shape[0],
                                                  ids.shape[1], lay.experts_fp8)
    if lay.experts_fp8:
        c, s = E._encode(lay.mlp_x)
        assert torch.equal(lay.mlp_codes, c) and torch.equal(lay.mlp_scales, s)
        p.x64 = E._values(lay.mlp_codes, lay.mlp_scales)
        p.w13_64, p.w2_64 = E._values(lay.w13, lay.w13_scales), E._values(lay.w2, lay.w2_scales)
    else:
        p.x64, p.w13_64, p.w2_64 = a, lay.w13.double(), lay.w2.double()
    p.ids, p.weights, p.y = lay.expert_ids, lay.expert_weights, lay.mlp_out
    p.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_decoder_layer_steps(fp8):
    lay = _layer(71, fp8=fp8)
    lay.status.zero_()
    for _ in range(4):
        given, added = lay.resid.clone(), lay.mlp_out.clone()
        lay.attn_input()
        _, want = L._norm_ref(added, given, lay.attn_norm, lay.ex.eps)
        L._close(lay.x, want, L.NORM_TOL)
        lay.frontend()
        lay.append()
        lay.step()
        before = lay.resid.clone()
        lay.mlp()
        _check_mlp(lay, before)
    assert int(lay.status.item()) == 0
    assert lay.seq_lens.tolist() == lay.wl.seq_lens.tolist()


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_decoder_layer_equals_eager(fp8):
    a, b = _layer(72, fp8=fp8), _layer(72, fp8=fp8)
    for lay in (a, b):
        lay.status.zero_()
    a.capture_layer()
    for i in range(4):
        a.layer_graph.replay()
        b.layer_step()
        torch.cuda.synchronize()
        for k in ("x", "y", "resid", "mlp_x", "logits", "expert_ids", "expert_weights", "mlp_out", "seq_lens"):
            assert torch.equal(getattr(a, k), getattr(b, k)), f"step {i}: {k}"
    assert int(a.status.item()) == 0


def test_two_layers_chained_over_one_stream():
    """The second layer takes the first one's stream and output."""
    a, b = _layer(73), _layer(74, n_experts=8, topk=2, n_group=1, topk_group=1, shared=0)
    b.resid, b_in = a.resid, b.mlp_out
    a.layer_step()
    b.mlp_out = a.mlp_out
    b.attn_input()
    b.mlp_out = b_in
    b.frontend()
    b.append()
    b.step()
    before = b.resid.clone()
    b.mlp()
    assert b.resid.data_ptr() == a.resid.data_ptr()
    _check_mlp(b, before)


def test_launches_of_the_experts_half():
    """What the experts add to launches_per_layer_step is what a profiler sees, on both sides of
    the copy of x."""
    from torch.profiler import ProfilerActivity, profile
    for rows, n_experts in (((300, 517, 77), 12), ((40,) * 70, 30), ((40,) * 60, 4)):
        lay = _layer(75, rows=rows, n_experts=n_experts, n_group=1, topk_group=1)
        lay.layer_step()
        torch.cuda.synchronize()
        for _ in range(4):  # a process's first profiles may come back empty
            with profile(activities=[ProfilerActivity.CUDA]) as prof:
                lay.attn_input()
                lay.mlp()
                torch.cuda.synchronize()
            seen = [e.name for e in prof.events() if "dsa::" in e.name]
            if seen:
                break
        else:
            pytest.skip("the profiler records no kernels here")
        whole, ex = lay.launches_per_layer_step(), lay.ex
        lay.ex = None
        assert len(seen) == whole - lay.launches_per_layer_step(), seen
        lay.ex = ex


def test_experts_of_a_layer_are_checked():
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8, hidden=512)
    wl = W.make_workload("decoder", 5, g, [100, 100])
    ex = W.make_experts(g, 3, 8, 2, 128)
    with pytest.raises(ValueError, match="stream"):
        DsaDecodeLayer(wl, experts=ex)
    ex = W.make_experts(g, 2, 8, 2, 128)
    with pytest.raises(ValueError, match="projected output"):
        DsaDecodeLayer(wl, experts=ex, with_o_absorb=False)
    lay = DsaDecodeLayer(wl, experts=ex)
    with pytest.raises(ValueError, match="front-end"):
        lay.attn_input()
    with pytest.raises(ValueError, match="experts"):
        DsaDecodeLayer(wl).mlp()
    # without a front-end the half that follows the attention still runs
    lay.compress()
    lay.step()
    before = lay.resid.clone()
    lay.mlp()
    _check_mlp(lay, before)
