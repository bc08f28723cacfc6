"""The layer's FP4 latent cache: its default exponent, its memory and its launch count."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import api, workloads as W
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer
from tests import _harness as H
from tests.test_gpu_fp4 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _workload(seed=61, paged=True):
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=128, heads=8,
                   hidden=256)
    return W.make_workload("fp4-layer", seed, g, [300, 517, 130], block_size=64 if paged else None,
                           max_seq_len=576 if paged else None, invalid_per_seq=0)


@pytest.mark.parametrize("mul", [1.0, 2.0 ** 20, 2.0 ** -20])
def test_default_exponent_leaves_room_for_larger_tokens(mul):
    """Tokens appended later, up to 16 times as large as any uploaded one, are stored within
    their format's steps, whatever the cache's magnitude. A block's scale is within 2^-4 of
    its maximum over 6, and a code within half a step of 2, so a value is off by at most
    1 + 2^-4 scales or, where it is cut off at 6, by 6 * 2^-4 / (1 - 2^-4) of one."""
    wl = _workload()
    wl.ckv.mul_(mul)  # a power of two: exact
    lay = DsaDecodeLayer(wl, decode_from=wl.seq_lens.astype(np.int64) - 3, latent_fp4=True)
    amax = float(wl.ckv.float().abs().max())
    assert 16 * amax <= 2688.0 * 2.0 ** lay.fp4_exp <= 32 * amax
    lay.compress()
    lay.stage(0)
    lay.ckv_new.mul_(16 * amax / float(lay.ckv_new.float().abs().max()))
    lay.append()
    torch.cuda.synchronize()
    x = H.f(lay.ckv_new.cpu())
    for b in range(wl.batch):
        at = lay._token_rows(b, int(wl.seq_lens[b]) - 3, int(wl.seq_lens[b]) - 2)
        codes = lay.ckv_codes.view(-1, 256)[at].cpu().numpy()
        scales = lay.ckv_scales.view(-1, 32)[at].cpu().numpy()
        got = O.dequantize_latent_fp4(codes, scales, lay.fp4_exp)[0]
        want = O.dequantize_latent_fp4(*O.quantize_latent_fp4(x[b:b + 1], lay.fp4_exp),
                                       lay.fp4_exp)[0]
        np.testing.assert_array_equal(got, want)
        step = np.abs(x[b]).reshape(32, 16).max(1) / 6.0
        assert (np.abs(got - x[b]).reshape(32, 16) <= (1 + 2.0 ** -4) * step[:, None]).all()


def test_default_exponent_keeps_small_blocks():
    """Blocks down to 1/896 of the cache's largest magnitude are stored as under any other
    exponent that does not saturate."""
    wl = _workload()
    flat = wl.ckv.view(-1, 512)
    flat.fill_(1.0)
    flat[0, 0] = 840.0
    lay = DsaDecodeLayer(wl, latent_fp4=True)
    codes, scales = lay.ckv_codes.view(-1, 256)[1:], lay.ckv_scales.view(-1, 32)[1:]
    want = O.dequantize_latent_fp4(*O.quantize_latent_fp4(np.ones((1, 512)), 0), 0)[0]
    got = O.dequantize_latent_fp4(codes[:4].cpu().numpy(), scales[:4].cpu().numpy(), lay.fp4_exp)
    np.testing.assert_array_equal(got, np.tile(want, (4, 1)))


@pytest.mark.parametrize("paged", [False, True], ids=["contig", "paged"])
def test_one_latent_cache(paged, monkeypatch):
    """The layer holds the 4-bit cache alone, the same one whether its rows are uploaded at
    once or a few at a time, with zeros where tokens are still to come."""
    wl = _workload(paged=paged)
    L0 = wl.seq_lens.astype(np.int64) - 5
    whole = DsaDecodeLayer(wl, latent_fp4=True)
    want_c, want_s = O.quantize_latent_fp4(H.f(wl.ckv.reshape(-1, 512)), whole.fp4_exp)
    np.testing.assert_array_equal(whole.ckv_codes.cpu().numpy().reshape(want_c.shape), want_c)
    np.testing.assert_array_equal(whole.ckv_scales.cpu().numpy().reshape(want_s.shape), want_s)
    monkeypatch.setattr(DsaDecodeLayer, "_FP4_UPLOAD", 100)
    lay = DsaDecodeLayer(wl, latent_fp4=True, decode_from=L0, manage_pages=paged)
    assert lay.ckv is None and lay.fp4_exp == whole.fp4_exp
    for b in range(wl.batch):
        at = lay._token_rows(b, int(L0[b]), int(wl.seq_lens[b]))
        want_c[at], want_s[at] = 0, 0
    np.testing.assert_array_equal(lay.ckv_codes.cpu().numpy().reshape(want_c.shape), want_c)
    np.testing.assert_array_equal(lay.ckv_scales.cpu().numpy().reshape(want_s.shape), want_s)


@pytest.mark.parametrize("rows,heads,ow", [(3, 8, 200), (100, 8, 512), (3, 64, 600), (100, 64, 256)])
def test_splits_say_whether_there_is_a_merge(rows, heads, ow):
    """The split count is one where the call leaves the workspace alone, and only there,
    although the workspace is sized for either kernel."""
    for which in ("auto", "mma", "tcgen05"):
        with api.mla_kernel(which):
            c = Case(97, rows, heads, ow, [700, 650]).cuda()
            need = api.dsa_sparse_mla_decode_fp4_workspace(rows, heads, ow, 0, False)
            splits = api.dsa_sparse_mla_decode_fp4_splits(rows, heads, ow, c.d_codes.numel() // 256)
            c.ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
            c.run(torch.empty((rows, heads, 512), dtype=torch.bfloat16, device="cuda"))
            part = rows * splits * heads * 512 * 4
            assert bool((c.ws == 0x5A).all()) == (splits == 1), (which, splits)
            if splits > 1:
                assert need >= part and (c.ws[need:] == 0x5A).all()


def test_layer_counts_its_launches():
    """100 rows: the attention takes one launch, 3 rows: two; score, selection, projection
    (one launch per 64 rows) and the prefetch are the same for both."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=512, heads=8,
                   hidden=256)
    for batch, splits in ((100, 1), (3, 8)):
        wl = W.make_workload("fp4-launches", 67, g, [600] * batch, invalid_per_seq=0)
        lay = DsaDecodeLayer(wl, latent_fp4=True)
        rows = lay.ckv_scales.numel() // 32
        assert api.dsa_sparse_mla_decode_fp4_splits(batch, 8, g.out_width, rows) == splits
        assert lay._mla_workspace(0, False) > 0
        assert lay.launches_per_step() == 3 + (splits > 1) + (batch + 63) // 64 + 1
