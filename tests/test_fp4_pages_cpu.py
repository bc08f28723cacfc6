"""The FP4 codec and the page operators without a GPU: the oracle pinned against values
fixed apart from it, and the library's refusals (argument errors are found on the host,
before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import _build, _lib, api
from sparse_attention_decode_kpool_gb300._lib import (DSA_ERR_CONFIG, DSA_ERR_INVALID_ARG,
                                                      DSA_ERR_UNSUPPORTED, DSA_OK)

FAKE = 0x10000  # a device address that is never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def _err(lib):
    return lib.dsa_last_error().decode()


# -- the codec -------------------------------------------------------------


def test_e2m1_codes_by_hand():
    v = [0, 0.25, 0.2500001, 0.5, 0.75, 0.7499, 1.0, 1.25, 1.2501, 1.5, 1.75, 2.0, 2.5, 2.51, 3.0,
         3.5, 3.49, 4.0, 5.0, 5.01, 6.0, 7.0, np.inf]
    want = [0, 0, 1, 1, 2, 1, 2, 2, 3, 3, 4, 4, 4, 5, 5, 6, 5, 6, 6, 7, 7, 7, 7]
    np.testing.assert_array_equal(O.e2m1_encode(v), want)
    np.testing.assert_array_equal(O.e2m1_encode(-np.array(v)), np.array(want) + 8)
    np.testing.assert_array_equal(O.e2m1_decode(range(16)),
                                  [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def test_e2m1_is_the_nearest_value():
    rng = np.random.default_rng(0)
    v = rng.uniform(-7, 7, 4000)
    table = O.e2m1_decode(range(16))
    best = np.abs(v[:, None] - table[None]).min(1)
    np.testing.assert_allclose(np.abs(v - O.e2m1_decode(O.e2m1_encode(v))), best, rtol=0, atol=0)


def test_fp4_block_by_hand():
    """One block: amax 3 -> scale E4M3(0.5) = 0.5; the codes are of x / 0.5."""
    x = np.zeros((1, 16))
    x[0, :6] = [3.0, -1.5, 0.25, -0.125, 0.75, 0.1]
    codes, scales = O.quantize_latent_fp4(x)
    assert O.e4m3_decode(scales)[0, 0] == 0.5
    # quotients 6, -3, .5, -.25 (tie to 0, sign kept), 1.5, .2
    np.testing.assert_array_equal(codes[0, :3], [7 | (13 << 4), 1 | (8 << 4), 3 | (0 << 4)])
    np.testing.assert_array_equal(O.dequantize_latent_fp4(codes, scales)[0, :6],
                                  [3.0, -1.5, 0.25, 0.0, 0.75, 0.0])


def test_fp4_properties():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (64, 512)) * np.exp2(rng.integers(-6, 6, (64, 1)))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    for e in (-8, 0, 5):
        c, s = O.quantize_latent_fp4(np.ldexp(x, e), e)
        c0, s0 = O.quantize_latent_fp4(x, 0)
        np.testing.assert_array_equal(c, c0)  # a power of two moves into cache_exp
        np.testing.assert_array_equal(s, s0)
        v = O.dequantize_latent_fp4(c, s, e)
        # exact in bf16 and, without the power of two, in f16
        np.testing.assert_array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
        u = np.ldexp(v, -e)
        np.testing.assert_array_equal(u.astype(np.float16).astype(np.float64), u)
        # half a code step of the scale, plus what the scale's own rounding cuts off at 6
        amax = np.abs(x.reshape(64, 32, 16)).max(2, keepdims=True)
        sc = O.e4m3_decode(s0)[:, :, None]
        err = np.abs(u - x).reshape(64, 32, 16)
        assert (err <= np.maximum(sc, amax - 6 * sc) + 1e-12).all()


def test_fp4_special_values():
    x = np.zeros((1, 64))
    x[0, 3], x[0, 16], x[0, 17], x[0, 32] = np.nan, np.inf, 5.0, 1e-9
    codes, scales = O.quantize_latent_fp4(x)
    v = O.dequantize_latent_fp4(codes, scales)
    assert scales[0, 0] == O.FP4_NAN_SCALE and np.isnan(v[0, :16]).all()
    assert v[0, 16] == 2688.0 and v[0, 17] == 0.0
    assert scales[0, 2] == 0 and (codes[0, 16:24] == 0).all()


# -- the page oracle -------------------------------------------------------


def test_page_pool_by_hand():
    """Two sequences of 5 and 4 tokens in pages of 4."""
    pool = O.PagePool([[3, 1, -1], [0, -1, -1], [-1, -1, -1]], [5, 4, 0], 8, 4,
                      caches=[np.arange(8)])
    np.testing.assert_array_equal(pool.refs, [1, 1, 0, 1, 0, 0, 0, 0])
    pool.fork([0], [2])
    np.testing.assert_array_equal(pool.table[2], [3, 1, -1])
    np.testing.assert_array_equal(pool.refs, [1, 2, 0, 2, 0, 0, 0, 0])
    # the next token: sequences 0 and 2 share page 1, sequence 1 starts a page
    pool.reserve(1)
    np.testing.assert_array_equal(pool.table, [[3, 2, -1], [0, 4, -1], [3, 5, -1]])
    np.testing.assert_array_equal(pool.refs, [1, 0, 1, 2, 1, 1, 0, 0])
    np.testing.assert_array_equal(pool.caches[0], [0, 1, 1, 3, 4, 1, 6, 7])
    pool.free([1, 1])
    np.testing.assert_array_equal(pool.refs, [0, 0, 1, 2, 0, 1, 0, 0])
    n, remap = pool.compact()
    assert n == 3
    np.testing.assert_array_equal(remap, [-1, -1, 2, 0, -1, 1, -1, -1])
    np.testing.assert_array_equal(pool.table, [[0, 2, -1], [-1, -1, -1], [0, 1, -1]])
    np.testing.assert_array_equal(pool.refs, [2, 1, 1, 0, 0, 0, 0, 0])
    assert not pool.bad


def test_written_pages_of_lagging_pools():
    """With first_key > 0 the pool that a token completes lies in an earlier page."""
    pool = O.PagePool([[0, 1, 2, 3]], [23], 4, 8)
    assert pool.written_pages(0, 1, 0, 4) == [2]      # token 23 and pool 5
    assert pool.written_pages(0, 1, 8, 4) == [1, 2]   # token 23, pool 3 = slot 1 of page 1
    assert pool.written_pages(0, 2, 16, 4) == [0, 2, 3]


# -- refusals --------------------------------------------------------------


def _pg(batch=2, paged=True, **kw):
    pg = _lib.DsaPaging()
    pg.batch, pg.max_seq_len, pg.seq_lens = batch, 256, FAKE
    pg.block_table = FAKE if paged else None
    pg.max_blocks, pg.block_size, pg.num_blocks = (4, 64, 16) if paged else (0, 0, 0)
    for k, v in kw.items():
        setattr(pg, k, v)
    return pg


@pytest.mark.parametrize("rows,kvl,exp,x,code", [
    (-1, 512, 0, FAKE, DSA_ERR_INVALID_ARG), (4, 500, 0, FAKE, DSA_ERR_INVALID_ARG),
    (4, 0, 0, FAKE, DSA_ERR_INVALID_ARG), (4, 512, 65, FAKE, DSA_ERR_INVALID_ARG),
    (4, 512, -65, FAKE, DSA_ERR_INVALID_ARG), (4, 512, 0, None, DSA_ERR_INVALID_ARG),
    (4, 512, 0, FAKE + 8, DSA_ERR_INVALID_ARG), (1 << 32, 512, 0, FAKE, DSA_ERR_UNSUPPORTED),
    (0, 512, 0, None, DSA_OK),
])
def test_fp4_codec_refusals(lib, rows, kvl, exp, x, code):
    assert lib.dsa_quantize_latent_fp4(x, rows, kvl, exp, FAKE, FAKE, None) == code
    assert lib.dsa_dequantize_latent_fp4(FAKE, FAKE, 1 << 40, None, rows, kvl, exp, x, None,
                                         None) == code
    if code:
        assert "fp4" in _err(lib)


def test_fp4_dequantize_needs_the_rows(lib):
    assert lib.dsa_dequantize_latent_fp4(FAKE, FAKE, 3, None, 4, 512, 0, FAKE, None,
                                         None) == DSA_ERR_INVALID_ARG
    assert "4 rows of a cache of 3" in _err(lib)


def _attend(lib, **kw):
    a = dict(q=FAKE, rows=2, heads=4, kvl=512, row_seq=None, codes=FAKE, scales=FAKE, exp=0,
             pg=_pg(), ids=FAKE, ow=8, o=None, hidden=0, y=None, olat=FAKE, olat16=None, ws=None,
             ws_bytes=0)
    a.update(kw)
    return lib.dsa_sparse_mla_decode_fp4(
        a["q"], a["rows"], a["heads"], a["kvl"], a["row_seq"], a["codes"], a["scales"], a["exp"],
        ctypes.byref(a["pg"]), a["ids"], a["ow"], 1.0, a["o"], a["hidden"], a["y"], a["olat"],
        a["olat16"], None, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(rows=-1), DSA_ERR_INVALID_ARG, "rows"),
    (dict(heads=0), DSA_ERR_INVALID_ARG, "heads"),
    (dict(ow=-1), DSA_ERR_INVALID_ARG, "out_width"),
    (dict(kvl=0), DSA_ERR_CONFIG, "kv_lora_rank"),
    (dict(kvl=576), DSA_ERR_UNSUPPORTED, "kv_lora_rank"),
    (dict(rows=65536), DSA_ERR_UNSUPPORTED, "rows"),
    (dict(heads=5000), DSA_ERR_UNSUPPORTED, "heads"),
    (dict(exp=65), DSA_ERR_INVALID_ARG, "cache_exp"),
    (dict(o=FAKE, hidden=64), DSA_ERR_INVALID_ARG, "both given"),
    (dict(y=FAKE), DSA_ERR_INVALID_ARG, "both given"),
    (dict(o=FAKE, y=FAKE, hidden=96), DSA_ERR_UNSUPPORTED, "hidden"),
    (dict(q=None), DSA_ERR_INVALID_ARG, "NULL"),
    (dict(codes=None), DSA_ERR_INVALID_ARG, "NULL"),
    (dict(scales=None), DSA_ERR_INVALID_ARG, "NULL"),
    (dict(ids=None), DSA_ERR_INVALID_ARG, "NULL"),
    (dict(q=FAKE + 4), DSA_ERR_INVALID_ARG, "aligned"),
    (dict(scales=FAKE + 8), DSA_ERR_INVALID_ARG, "aligned"),
    (dict(olat=FAKE + 8), DSA_ERR_INVALID_ARG, "aligned"),
    (dict(pg=_pg(seq_lens=None)), DSA_ERR_INVALID_ARG, "seq_lens"),
    (dict(rows=0, q=None), DSA_OK, ""),
    (dict(olat=None), DSA_OK, ""),  # nothing requested
])
def test_fp4_attention_refusals(lib, kw, code, text):
    assert _attend(lib, **kw) == code
    if code:
        assert text in _err(lib)


def test_fp4_append_refusals(lib):
    def call(**kw):
        a = dict(ckv_new=FAKE, kvl=512, codes=FAKE, scales=FAKE, exp=0, lens=FAKE, ihd=128)
        a.update(kw)
        return lib.dsa_decode_append_fp4(FAKE, FAKE, a["ckv_new"], FAKE, FAKE, FAKE, 1e-6,
                                         ctypes.byref(_pg()), a["lens"], 0, 4, a["ihd"], a["kvl"],
                                         FAKE, FAKE, FAKE, None, a["codes"], a["scales"], a["exp"],
                                         FAKE, FAKE, None, None, None, None)
    for kw, code, text in [(dict(codes=None), DSA_ERR_INVALID_ARG, "NULL"),
                           (dict(scales=None), DSA_ERR_INVALID_ARG, "NULL"),
                           (dict(ckv_new=None), DSA_ERR_INVALID_ARG, "ckv_new"),
                           (dict(kvl=200), DSA_ERR_INVALID_ARG, "multiple of 128"),
                           (dict(exp=100), DSA_ERR_INVALID_ARG, "cache_exp"),
                           (dict(ihd=96), DSA_ERR_UNSUPPORTED, "index_head_dim"),
                           (dict(lens=FAKE + 16), DSA_ERR_INVALID_ARG, "seq_lens"),
                           (dict(scales=FAKE + 4), DSA_ERR_INVALID_ARG, "aligned")]:
        assert call(**kw) == code, kw
        assert text in _err(lib), kw


def test_pages_refusals(lib):
    ref = ctypes.byref
    pa = _lib.DsaPageArrays()
    ws = ctypes.c_size_t(0)
    assert lib.dsa_pages_workspace(0, 1, ref(ws)) == DSA_ERR_INVALID_ARG
    assert lib.dsa_pages_workspace(16, 0, ref(ws)) == DSA_ERR_INVALID_ARG
    assert lib.dsa_pages_workspace(16, 2, None) == DSA_ERR_INVALID_ARG
    assert lib.dsa_pages_workspace(16, 2, ref(ws)) == DSA_OK and ws.value > 0
    big = ws.value

    def free(pg=None, n=1, seqs=FAKE, table=FAKE, lens=FAKE, refs=FAKE):
        return lib.dsa_pages_free(seqs, n, ref(pg or _pg()), table, lens, refs, None, None)

    def fork(pg=None, n=1, par=FAKE, kids=FAKE, table=FAKE, lens=FAKE, refs=FAKE):
        return lib.dsa_pages_fork(par, kids, n, ref(pg or _pg()), table, lens, refs, None, None)

    for call in (free, fork):
        for kw, text in [(dict(pg=_pg(paged=False)), "not paged"), (dict(table=FAKE + 64), "block_table"),
                         (dict(table=None), "block_table"), (dict(lens=FAKE + 64), "seq_lens"),
                         (dict(refs=None), "refs"), (dict(n=-1), "sequences"),
                         (dict(n=3), "the batch has 2")]:
            assert call(**kw) == DSA_ERR_INVALID_ARG, kw
            assert text in _err(lib), kw
        assert call(pg=_pg(num_blocks=1 << 31)) == DSA_ERR_UNSUPPORTED
        assert call(n=0) == DSA_OK
    assert free(seqs=None) == DSA_ERR_INVALID_ARG
    assert fork(par=None) == DSA_ERR_INVALID_ARG
    assert fork(kids=None) == DSA_ERR_INVALID_ARG

    def reserve(pg=None, n=1, seqs=FAKE, new=1, first=0, kp=4, arrays=None, w=FAKE, wb=big, table=FAKE):
        return lib.dsa_pages_reserve(seqs, n, ref(pg or _pg()), table, FAKE, new, first, kp, arrays,
                                     None, w, wb, None)

    def compact(pg=None, arrays=None, w=FAKE, wb=big, table=FAKE):
        return lib.dsa_pages_compact(ref(pg or _pg()), table, FAKE, arrays, None, None, None, w, wb,
                                     None)

    for kw, code, text in [(dict(new=0), DSA_ERR_INVALID_ARG, "new_tokens"),
                           (dict(kp=17), DSA_ERR_UNSUPPORTED, "kpool"),
                           (dict(kp=3), DSA_ERR_UNSUPPORTED, "multiples"),
                           (dict(first=2), DSA_ERR_UNSUPPORTED, "multiples"),
                           (dict(first=-4), DSA_ERR_INVALID_ARG, "first_key"),
                           (dict(n=3), DSA_ERR_INVALID_ARG, "the batch has 2")]:
        assert reserve(**kw) == code, kw
        assert text in _err(lib), kw
    for call in (reserve, compact):
        for kw in (dict(w=None), dict(wb=big - 1), dict(w=FAKE + 8)):
            assert call(**kw) == DSA_ERR_INVALID_ARG
            assert "workspace" in _err(lib)
        assert call(pg=_pg(paged=False)) == DSA_ERR_INVALID_ARG
        assert call(table=FAKE + 64) == DSA_ERR_INVALID_ARG
        pa.num_pages = 16
        pa.n = 129
        assert call(arrays=ref(pa)) == DSA_ERR_INVALID_ARG
        pa.n = 1
        pa.base[0], pa.page_bytes[0] = None, 64
        assert call(arrays=ref(pa)) == DSA_ERR_INVALID_ARG
        pa.base[0], pa.page_bytes[0] = FAKE, 0
        assert call(arrays=ref(pa)) == DSA_ERR_INVALID_ARG
        assert "page array 0" in _err(lib)
        pa.num_pages = 15
        assert call(arrays=ref(pa)) == DSA_ERR_INVALID_ARG
        assert "15 pages" in _err(lib)


def test_binding_refusals():
    """Shapes that the binding checks before the library is called."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="codes"):
        api.dsa_quantize_latent_fp4(x, u8(4, 512), u8(4, 32))
    with pytest.raises(ValueError, match="match x"):
        api.dsa_quantize_latent_fp4(x, u8(3, 256), u8(3, 32))
    with pytest.raises(ValueError, match="codes"):
        api.dsa_quantize_latent_fp4(x, u8(4, 256), u8(3, 32))
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_quantize_latent_fp4(x, u8(4, 256), u8(4, 32))
    with pytest.raises(ValueError, match="4 rows"):
        api.dsa_dequantize_latent_fp4(u8(4, 256), u8(4, 32), x[:3])
    with pytest.raises(ValueError, match="3 row numbers"):
        api.dsa_dequantize_latent_fp4(u8(4, 256), u8(4, 32), x[:3], rows=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="cache 0"):
        api.page_arrays([u8(3, 4)], 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.page_arrays([u8(4, 4)], 4)
    with pytest.raises(ValueError, match="at most 128"):
        api.page_arrays([u8(4, 4)] * 129, 4)
