"""The guarded append without a GPU: its refusals, the layer's, and the oracle's rule for
which pages a sequence holds alone."""
import ctypes

import pytest

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import _build, _lib, workloads as W
from sparse_attention_decode_kpool_gb300._lib import DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer

FAKE = 0x10000  # a device address that is never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def _pg(paged=True):
    pg = _lib.DsaPaging()
    pg.batch, pg.max_seq_len, pg.seq_lens = 2, 256, FAKE
    pg.block_table = FAKE if paged else None
    pg.max_blocks, pg.block_size, pg.num_blocks = (4, 64, 16) if paged else (0, 0, 0)
    return pg


@pytest.mark.parametrize("kw,code,text", [
    (dict(latent=3), DSA_ERR_INVALID_ARG, "latent 3"),
    (dict(latent=-1), DSA_ERR_INVALID_ARG, "latent -1"),
    (dict(latent=_lib.DSA_LATENT_BF16), DSA_ERR_INVALID_ARG, "ckv_codes"),
    (dict(latent=_lib.DSA_LATENT_FP8, codes=None), DSA_ERR_INVALID_ARG, "ckv_codes"),
    (dict(latent=_lib.DSA_LATENT_FP4, scales=None), DSA_ERR_INVALID_ARG, "ckv_scales"),
    (dict(latent=_lib.DSA_LATENT_BF16, codes=None, scales=None, ckv=None), DSA_ERR_INVALID_ARG,
     "together"),
    (dict(paged=False), DSA_ERR_INVALID_ARG, "not paged"),
    (dict(exp=65), DSA_ERR_INVALID_ARG, "cache_exp"),
    (dict(kpool=17), DSA_ERR_UNSUPPORTED, "kpool"),
    (dict(scales=FAKE + 8), DSA_ERR_INVALID_ARG, "aligned"),
    (dict(lens=FAKE + 16), DSA_ERR_INVALID_ARG, "seq_lens"),
])
def test_guarded_append_refusals(lib, kw, code, text):
    a = dict(latent=_lib.DSA_LATENT_FP4, ckv=FAKE, codes=FAKE, scales=FAKE, exp=0, kpool=4,
             lens=FAKE, paged=True)
    a.update(kw)
    rc = lib.dsa_decode_append_guarded(
        FAKE, FAKE, a["latent"], FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1e-6,
        ctypes.byref(_pg(a["paged"])), a["lens"], 0, a["kpool"], 128, 512, FAKE, FAKE, FAKE,
        a["ckv"], a["codes"], a["scales"], a["exp"], FAKE, FAKE, None, None, None, None)
    assert rc == code
    assert text in lib.dsa_last_error().decode()


def test_pages_serve_refusals(lib):
    def call(n=1, batch=2, seqs=FAKE, serving=FAKE):
        return lib.dsa_pages_serve(None, seqs, n, batch, 1, serving, None, None)

    for kw, text in [(dict(batch=0), "batch 0"), (dict(n=-1), "-1 sequences"),
                     (dict(n=3), "the batch has 2"), (dict(serving=None), "serving"),
                     (dict(seqs=None), "NULL sequences")]:
        assert call(**kw) == DSA_ERR_INVALID_ARG, kw
        assert text in lib.dsa_last_error().decode(), kw
    assert call(n=0, seqs=None) == _lib.DSA_OK


def test_managed_pages_need_the_fused_append():
    with pytest.raises(ValueError, match="fuse_append"):
        DsaDecodeLayer(W.tiny(), device="cpu", manage_pages=True, fuse_append=False)


def test_holds_alone():
    """Pages of 4 tokens, pools of 2; sequences 0 and 1 share page 3, sequence 0's second
    page is its own."""
    pool = O.PagePool([[3, 0, -1], [3, -1, -1], [1, -1, -1]], [5, 3, 0], 5, 4)
    assert pool.holds_alone(0) and not pool.holds_alone(1) and pool.holds_alone(2)
    # with first_key 2, token 5 completes pool 1: the second slot of the shared page
    assert pool.holds_alone(0, 0, 2) and not pool.holds_alone(0, 2, 2)
    pool.lens[0] = 8
    assert not pool.holds_alone(0)  # unmapped
    pool.lens[0] = 12
    assert not pool.holds_alone(0)  # full
