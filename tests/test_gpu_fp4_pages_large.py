"""The FP4 codec and the page operators above the sizes at which they take another form:
many rows, pools of more pages than one pass of the plan covers, batches of more sequences
than it has threads, and a layer that uses managed pages with every cache format."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import api, workloads as W
from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_TOKEN
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer
from tests import _harness as H
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("rows,kvl", [(155_647, 512), (155_648, 512), (160_003, 512),
                                      (1_250_007, 64)])
def test_codec_many_rows(rows, kvl):
    """Above 4.98 million blocks a thread takes four: the same bytes as a few rows at a time
    (which are the oracle's), nothing behind the last row, and the same rows back."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = torch.randn((rows, kvl), generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g, device="cuda"))
    x = x.to(torch.bfloat16)
    x[-1, 3] = float("nan")
    codes = torch.full((rows + 1, kvl // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 1, kvl // 16), 0x55, dtype=torch.uint8, device="cuda")
    api.dsa_quantize_latent_fp4(x, codes[:rows], scales[:rows], -8)
    assert (codes[rows] == 0xAA).all() and (scales[rows] == 0x55).all()
    few_c, few_s = torch.empty_like(codes[:rows]), torch.empty_like(scales[:rows])
    part = 20_000
    for i in range(0, rows, part):
        api.dsa_quantize_latent_fp4(x[i:i + part], few_c[i:i + part], few_s[i:i + part], -8)
    assert torch.equal(codes[:rows], few_c) and torch.equal(scales[:rows], few_s)
    pick = torch.randint(0, rows, (300,), generator=g, device="cuda")
    pick[0] = rows - 1
    want_c, want_s = O.quantize_latent_fp4(H.f(x[pick].cpu()), -8)
    np.testing.assert_array_equal(codes[pick].cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales[pick].cpu().numpy(), want_s)

    out = torch.full((rows + 1, kvl), 7.0, dtype=torch.bfloat16, device="cuda")
    api.dsa_dequantize_latent_fp4(codes[:rows], scales[:rows], out[:rows], -8)
    assert (out[rows] == 7.0).all()
    few = torch.empty((rows, kvl), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, part):
        api.dsa_dequantize_latent_fp4(few_c[i:i + part], few_s[i:i + part], few[i:i + part], -8)
    assert torch.equal(out[:rows].view(torch.int16), few.view(torch.int16))
    np.testing.assert_array_equal(out[pick].double().cpu().numpy(),
                                  O.dequantize_latent_fp4(want_c, want_s, -8))

    # rows by their numbers, two of them outside the cache
    ids = torch.randint(0, rows, (rows,), generator=g, device="cuda", dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_dequantize_latent_fp4(codes[:rows], scales[:rows], out[:rows], -8, rows=ids,
                                  status=status)
    assert int(status) == 0 and (out[rows] == 7.0).all()
    assert torch.equal(out[:rows].view(torch.int16), few[ids.long()].view(torch.int16))
    ids[5], ids[-1] = -1, rows
    api.dsa_dequantize_latent_fp4(codes[:rows], scales[:rows], out[:rows], -8, rows=ids,
                                  status=status)
    assert int(status) == DSA_STATUS_BAD_TOKEN
    assert (out[5] == 0).all() and (out[rows - 1] == 0).all()


def _big_pool(seed, n_seq, pages, spare):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 2 * pages * 2 // n_seq, n_seq)
    lens[::50] = 0
    need = -(-lens // 2)
    return Pool(seed, lens, 2, int(need.max()) + 12, pages - int(need.sum()) + spare,
                widths=(16, 3))


@pytest.mark.parametrize("pages", [32_768, 33_000, 70_001])
def test_pages_of_a_large_pool(pages):
    """More than 32,768 pages: several passes over the counts. Fork, reserve (a token and a
    prompt), free and compact, against the oracle."""
    p = _big_pool(pages, 1500, pages, 6000)
    assert p.ref.n >= pages
    rng = np.random.default_rng(1)
    order = rng.permutation(1500)
    p.fork(order[:300], order[300:600])
    p.reserve(1, 4, 2)
    p.check("token")
    p.append()
    p.reserve(14, 2, 2, seqs=order[500:900])
    p.check("prompt")
    p.free(order[::3])
    p.check("free")
    p.compact()
    p.check("compact")
    p.reserve(3)
    p.check("again")
    assert p.ref.bad <= {"pages", "full"}


def test_compact_a_large_pool_that_is_full_or_empty():
    p = _big_pool(3, 1500, 40_000, 0)
    p.compact()
    p.check("as it is")
    p.free(np.arange(1500))
    p.compact()
    p.check("empty")
    assert (p.ref.refs == 0).all()


def test_reserve_more_sequences_than_threads():
    """9,000 sequences: those of a thread one after another."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 9, 9000)
    p = Pool(5, lens, 4, 6, 20_000, widths=(16,))
    p.fork(np.arange(0, 3000), np.arange(6000, 9000))
    p.reserve(1, 4, 2)
    p.check("one")
    p.append()
    p.reserve(3, seqs=rng.permutation(9000)[:8500])
    p.check("list")
    assert not p.ref.bad


@pytest.mark.parametrize("first_key", [4 * 28, 4 * 29, 4 * 40])
def test_reserve_far_pooled_keys(first_key):
    """A pooled key 28 and more pages before its token's: past 32 entries between the two
    they no longer fit a thread's mask."""
    p = Pool(6, [4 * 45 + 3, 4 * 41, 4 * 29 + 1, 0, 7, 0], 4, 60, 200, widths=(16,))
    p.fork([0, 1], [3, 5])
    for i in range(7):
        p.reserve(2, first_key, 2)
        p.check(i)
        p.append(2)
    assert not p.ref.bad


@pytest.mark.parametrize("kw", [{}, {"latent_fp8": True}, {"latent_fp4": True}],
                         ids=["bf16", "fp8", "fp4"])
def test_managed_layer_equals_a_plain_one(kw):
    """Front-end, append and step with managed pages, captured, against a layer whose table
    names every page from the start: the same bits, past a page's end."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8,
                   hidden=512)
    wl = W.make_workload("managed", 55, g, [300, 517, 77], block_size=64, max_seq_len=640)
    fe = W.make_frontend(g, wl.rows, q_lora_rank=512, seed=56)
    L0 = np.array([250, 509, 60])
    a = DsaDecodeLayer(wl, keep_olat=True, decode_from=L0, frontend=fe, manage_pages=True, **kw)
    b = DsaDecodeLayer(wl, keep_olat=True, decode_from=L0, frontend=fe, **kw)
    for lay in (a, b):
        lay.status.zero_()
        lay.compress()
    a.capture_layer()
    for i in range(9):
        a.layer_graph.replay()
        b.layer_step()
        if i == 6:
            a.compact_pages()
    torch.cuda.synchronize()
    for k in ("qlat", "scores", "pool_ids", "token_ids", "olat", "y", "seq_lens", "row_ctx"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert int(a.status) == 0 and a.seq_lens.tolist() == (L0 + 9).tolist()
    assert int(a.block_table.max()) < int(a.pages_live) + 3
    assert a.launches_per_layer_step() == b.launches_per_layer_step() + 2


def test_managed_layer_refusals():
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8,
                   hidden=512)
    wl = W.make_workload("unmanaged", 57, g, [100, 30], block_size=64, max_seq_len=128)
    lay = DsaDecodeLayer(wl)
    for call in (lambda: lay.free_sequences([0]), lambda: lay.fork_sequences([0], [1]),
                 lambda: lay.pause_sequences([0]), lambda: lay.resume_sequences([0]),
                 lay.reserve_pages, lay.compact_pages):
        with pytest.raises(ValueError, match="manage_pages"):
            call()
    managed = DsaDecodeLayer(wl, manage_pages=True)
    with pytest.raises(TypeError, match="int32"):
        managed.free_sequences(torch.tensor([0], device="cuda"))
    with pytest.raises(ValueError, match="same length"):
        managed.fork_sequences([0, 1], [1])
