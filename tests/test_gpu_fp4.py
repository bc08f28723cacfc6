"""FP4 latent cache on the GPU: the codec bit for bit against the oracle, sparse attention
against its definition in 64 bits, the decode-time append, and a layer that uses them
together.

The attention's tolerance. Decoded rows are exact in the kernels' f16, q loses nothing
(bf16 times a power of two). Left are: the logits' f32 sums, 32 steps of 16 products each
of which may lose 2^-22 of the sum of magnitudes (2 ulp; the tensor core truncates),
delta = scale * 2^-17 * sum |q v| in all; the weights' rounding to f16 (half a step,
2^-12) in numerator and denominator; ex2's 2^-22 and the f32 sums over at most 4096
weights, below 2^-13 together. With A = sum_t p_t |v_t| that is
A * (2^-11 + 2 * delta + 2^-13), and the result's own rounding: 2^-8 of it for bf16,
2^-23 for f32.

Half a step is 2^-12 of a weight only down to f16's smallest normal number, 2^-14; below it
the step is 2^-24 whatever the weight. The kernels hold weights at 2^7 or more times
p_t / max p, so a weight's absolute error there is at most 2^-25 / 2^7 = 2^-32 of the
largest weight: 2^-32 max(p) * sum |v_t| in the numerator, 2^-32 max(p) * T of the result
from the denominator (sum of T weights)."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import api, workloads as W
from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_BLOCK, DSA_STATUS_BAD_TOKEN
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer
from tests import _harness as H

pytestmark = pytest.mark.gpu

KVL = 512


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


# -- codec -----------------------------------------------------------------


def _codec_rows(rng, n, kvl=KVL):
    x = rng.normal(0, 1, (n, kvl)) * np.exp2(rng.integers(-12, 13, (n, 1)))
    x[0] = 0.0
    if n > 8:
        x[1, :16] = 0.0
        x[2, 5] = -0.0
        x[3] = rng.normal(0, 1, kvl) * 2.0 ** -130
        x[4] = np.where(np.arange(kvl) % 2, 3.0, -1.25)           # E2M1 ties under scale 0.5
        x[5] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], kvl // 8)
        x[6] = rng.normal(0, 1e30, kvl)
        x[7, 3], x[7, 20 % kvl], x[7, 40 % kvl] = np.nan, np.inf, -np.inf
        x[8] = 2.0 ** -10 * rng.integers(-15, 16, kvl)            # E4M3's subnormal scales
    return _bf16(x)


@pytest.mark.parametrize("n,kvl,exp", [(1, 512, 0), (300, 512, 0), (257, 512, -8), (64, 512, 12),
                                       (33, 128, 0), (9, 16, -3), (20, 48, 0), (40, 512, -64),
                                       (40, 512, 64)])
def test_fp4_codec_parity(n, kvl, exp):
    x = _codec_rows(np.random.default_rng(n + kvl), n, kvl)
    codes = torch.full((n + 1, kvl // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((n + 1, kvl // 16), 0x55, dtype=torch.uint8, device="cuda")
    api.dsa_quantize_latent_fp4(x.cuda(), codes[:n], scales[:n], exp)
    want_c, want_s = O.quantize_latent_fp4(H.f(x), exp)
    np.testing.assert_array_equal(scales[:n].cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes[:n].cpu().numpy(), want_c)
    assert (codes[n] == 0xAA).all() and (scales[n] == 0x55).all()  # nothing behind the last row
    out = torch.full((n + 1, kvl), 7.0, dtype=torch.bfloat16, device="cuda")
    api.dsa_dequantize_latent_fp4(codes[:n], scales[:n], out[:n], exp)
    got = out.float().cpu().numpy()
    want = O.dequantize_latent_fp4(want_c, want_s, exp)
    np.testing.assert_array_equal(got[:n], want)
    assert (got[n] == 7.0).all()


def test_fp4_every_tie():
    """Every bf16 significand against every scale significand, near and on each midpoint."""
    m = np.arange(128, 256) / 128.0
    blocks = []
    for amax in (np.arange(96, 192) / 16.0):                      # scales 1 .. 2 in steps and between
        for k in range(0, 128, 15):
            blocks.append(np.concatenate(([amax], m[k:k + 15], np.zeros(15 - len(m[k:k + 15])))))
    x = np.array(blocks)
    x = np.concatenate((x, x * np.concatenate(([1.0], np.full(15, 0.25)))))
    xb = _bf16(x)
    codes = torch.empty((len(x), 8), dtype=torch.uint8, device="cuda")
    scales = torch.empty((len(x), 1), dtype=torch.uint8, device="cuda")
    api.dsa_quantize_latent_fp4(xb.cuda(), codes, scales)
    want_c, want_s = O.quantize_latent_fp4(H.f(xb))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)


def test_fp4_every_byte_decodes():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()     # [256, 256]
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 32)
    scales[0x80:] = scales[:0x80]                                          # scales are positive
    out = torch.empty((256, KVL), dtype=torch.bfloat16, device="cuda")
    api.dsa_dequantize_latent_fp4(codes, scales.cuda(), out, 3)
    want = O.dequantize_latent_fp4(codes.cpu().numpy(), scales.numpy(), 3)
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)


def test_fp4_dequantize_rows():
    rng = np.random.default_rng(5)
    x = _codec_rows(rng, 50)
    codes = torch.empty((50, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((50, 32), dtype=torch.uint8, device="cuda")
    api.dsa_quantize_latent_fp4(x.cuda(), codes, scales)
    rows = torch.tensor([3, 49, 3, -1, 0, 50, 12], dtype=torch.int32, device="cuda")
    out = torch.full((7, KVL), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_dequantize_latent_fp4(codes, scales, out, rows=rows, status=status)
    assert int(status) == DSA_STATUS_BAD_TOKEN
    want = O.dequantize_latent_fp4(codes.cpu().numpy(), scales.cpu().numpy())
    got = out.float().cpu().numpy()
    for i, r in enumerate([3, 49, 3, None, 0, None, 12]):
        np.testing.assert_array_equal(got[i], 0.0 if r is None else want[r])
    status.zero_()
    api.dsa_dequantize_latent_fp4(codes, scales, out, rows=rows.clamp(0, 49), status=status)
    assert int(status) == 0


# -- attention -------------------------------------------------------------


class Case:
    """Inputs of one attention call: a cache whose unselected rows hold NaN, selections
    with holes, and the result by definition."""

    def __init__(self, seed, rows, heads, ow, lens, block=0, exp=-8, q_mul=1.0, hole=0.2,
                 empty_rows=(), scale=1 / 16, row_seq=None):
        rng = np.random.default_rng(seed)
        self.rows, self.heads, self.ow, self.exp, self.scale = rows, heads, ow, exp, scale
        self.lens = np.array(lens, dtype=np.int32)
        B = len(lens)
        self.max_len = max(int(self.lens.max()), 1)
        self.block = block
        if block:
            mb = -(-self.max_len // block)
            need = -(-self.lens // block)
            self.num = int(need.sum()) + 3
            perm = rng.permutation(self.num)
            self.table = np.full((B, mb), -1, dtype=np.int32)
            k = 0
            for b in range(B):
                self.table[b, :need[b]] = perm[k:k + need[b]]
                k += need[b]
            n = self.num * block
        else:
            self.table, self.num = None, 0
            n = B * self.max_len
        self.row_seq = np.array(rng.integers(0, B, rows) if row_seq is None else row_seq, dtype=np.int32)
        self.ids = np.full((rows, ow), -1, dtype=np.int32)
        for r in range(rows):
            L = int(self.lens[self.row_seq[r]])
            if L == 0 or ow == 0 or r in empty_rows:
                continue
            t = rng.integers(0, L, ow)
            self.ids[r] = np.where(rng.random(ow) < hole, -1, t)
        x = _bf16(rng.normal(0, 1, (n, KVL)) * np.exp(0.3 * rng.normal(size=KVL)))
        self.codes, self.scales = O.quantize_latent_fp4(H.f(x), exp)
        used = np.zeros(n, dtype=bool)
        for r in range(rows):
            used[self.at(r)[1]] = True
        self.codes[~used] = 0x77
        self.scales[~used] = O.FP4_NAN_SCALE
        self.q = _bf16(rng.normal(0, 1, (rows, heads, KVL)) * q_mul)

    def at(self, r):
        """(selected tokens, their cache rows) of row r."""
        t = self.ids[r][self.ids[r] >= 0].astype(np.int64)
        b = int(self.row_seq[r])
        if self.block:
            return t, self.table[b, t // self.block].astype(np.int64) * self.block + t % self.block
        return t, b * self.max_len + t

    def want(self):
        """(result, tolerance without the result's own rounding), 64 bits."""
        out = np.zeros((self.rows, self.heads, KVL))
        tol = np.zeros_like(out)
        q = H.f(self.q).reshape(self.rows, self.heads, KVL)
        for r in range(self.rows):
            _, rows = self.at(r)
            if not len(rows):
                continue
            v = O.dequantize_latent_fp4(self.codes[rows], self.scales[rows], self.exp)
            s = self.scale * (q[r] @ v.T)
            delta = abs(self.scale) * 2.0 ** -17 * (np.abs(q[r]) @ np.abs(v).T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[r] = p @ v
            tol[r] = (p * (2.0 ** -11 + 2.0 ** -13 + 2 * np.expm1(delta))) @ np.abs(v)
            tol[r] += (p * 2 * np.expm1(delta)).sum(1, keepdims=True) * np.abs(out[r])
            small = 2.0 ** -32 * p.max(1, keepdims=True)
            tol[r] += small * (np.abs(v).sum(0) + len(rows) * np.abs(out[r]))
        return out, tol

    def cuda(self):
        d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d_lens, self.d_table = d(self.lens), d(self.table)
        self.pg = api.paging(self.d_lens, self.max_len, self.d_table, self.block, self.num)
        self.d_codes, self.d_scales = d(self.codes), d(self.scales)
        self.d_q, self.d_ids, self.d_seq = self.q.cuda(), d(self.ids), d(self.row_seq)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = api.dsa_sparse_mla_decode_fp4_workspace(self.rows, self.heads, self.ow, 0, False)
        self.ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN bytes
        return self

    def run(self, olat, **kw):
        api.dsa_sparse_mla_decode_fp4(self.d_q, kw.pop("row_seq", self.d_seq), self.d_codes,
                                      self.d_scales, self.exp, self.pg, self.d_ids, self.scale,
                                      olat=olat, status=self.status, workspace=self.ws, **kw)


def _check(case, kernels=("auto",), dtypes=(torch.bfloat16, torch.float32)):
    want, tol = case.want()
    for which in kernels:
        with api.mla_kernel(which):
            case.cuda()
            for dt in dtypes:
                out = torch.full((case.rows + 1, case.heads, KVL), 7.0, dtype=dt, device="cuda")
                case.run(out[:case.rows])
                torch.cuda.synchronize()
                assert int(case.status) == 0
                got = out.double().cpu().numpy()
                assert (got[case.rows] == 7.0).all()  # nothing behind the last row
                half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -23
                err = np.abs(got[:case.rows] - want)
                bound = tol * (1 + half) + half * np.abs(want)
                assert (err <= bound).all(), (which, dt, float((err - bound).max()),
                                              float(np.nanmax(err / np.maximum(bound, 1e-30))))


KERNELS = ("mma", "tcgen05")


@pytest.mark.parametrize("heads", [1, 3, 16, 17, 32, 33, 63, 64, 65, 96, 128])
def test_fp4_attention_heads(heads):
    _check(Case(heads, 3, heads, 200, [150, 400]), KERNELS)


@pytest.mark.parametrize("ow", [0, 1, 5, 63, 64, 65, 127, 128, 129, 130, 300, 2048])
def test_fp4_attention_widths(ow):
    _check(Case(ow, 2, 64, ow, [700, 90], hole=0.1), KERNELS)


@pytest.mark.parametrize("block", [0, 1, 16, 64, 100])
def test_fp4_attention_layouts(block):
    _check(Case(block + 7, 9, 64, 257, [1, 100, 517, 0, 64], block=block), KERNELS)


@pytest.mark.parametrize("block", [0, 64])
def test_fp4_attention_empty_rows(block):
    """Rows whose selection is empty, the first and the last among them."""
    _check(Case(11, 7, 64, 140, [300, 50], block=block, empty_rows=(0, 3, 6)), KERNELS)
    _check(Case(12, 3, 8, 140, [300, 50], block=block, empty_rows=(0, 1, 2)), KERNELS)


def test_fp4_attention_sparse_holes():
    """Whole chunks without a token, single tokens at a row's ends."""
    c = Case(13, 4, 64, 600, [900], hole=0.0)
    c.ids[0, 1:] = -1
    c.ids[1, :-1] = -1
    c.ids[2, 64:512] = -1
    c.ids[3, :300] = -1
    _check(c, KERNELS)


@pytest.mark.parametrize("q_mul", [0.0, 1e-30, 2.0 ** -126, 1e-3, 30.0, 1e30])
def test_fp4_attention_query_magnitudes(q_mul):
    """q far outside f16's range; the large ones make the softmax one-hot (the scale keeps
    the logits finite)."""
    scale = 1 / 16 if q_mul <= 100 else 4.0 / q_mul
    _check(Case(17, 3, 64, 260, [300], q_mul=q_mul, scale=scale), KERNELS)


@pytest.mark.parametrize("scale", [0.0, -1 / 16, 1e-30])
def test_fp4_attention_scales(scale):
    """No scale (equal weights), a negative and a vanishing one."""
    _check(Case(18, 3, 64, 260, [300], scale=scale), KERNELS)


def test_fp4_attention_both_outputs_and_no_status():
    """f32 and bf16 results of one call, and calls without a status word or row_seq."""
    c = Case(20, 4, 64, 700, [900, 50, 300, 7], row_seq=[0, 1, 2, 3]).cuda()
    a = torch.empty((4, 64, KVL), dtype=torch.float32, device="cuda")
    b = torch.empty((4, 64, KVL), dtype=torch.bfloat16, device="cuda")
    for which in KERNELS:
        with api.mla_kernel(which):
            c.run(a)
            c.run(b, row_seq=None)
            assert torch.equal(a.to(torch.bfloat16), b)
            api.dsa_sparse_mla_decode_fp4(c.d_q, c.d_seq, c.d_codes, c.d_scales, c.exp, c.pg, c.d_ids,
                                          c.scale, olat=b, workspace=c.ws)
            assert torch.equal(a.to(torch.bfloat16), b)


@pytest.mark.parametrize("exp", [-30, -3, 0, 20])
def test_fp4_attention_cache_exp(exp):
    c = Case(19, 3, 64, 260, [300], exp=-8)
    c.exp, c.scale = exp, 2.0 ** (-exp - 12)
    _check(c, KERNELS)


def test_fp4_attention_growing_maxima():
    """Logits that grow by hundreds along the list, and a list that starts at its maximum:
    the running maximum moves at every chunk, or never."""
    for order in (1, -1):
        c = Case(23, 2, 64, 1024, [1024], hole=0.0, q_mul=12.0)
        q = H.f(c.q)
        v = O.dequantize_latent_fp4(c.codes, c.scales, c.exp)
        for r in range(2):
            t = np.argsort(order * (q[r, 0] @ v[:1024].T), kind="stable")
            c.ids[r] = t
        # every token is selected: none of the rows may stay NaN
        x = _bf16(np.random.default_rng(24).normal(0, 1, v.shape))
        c.codes, c.scales = O.quantize_latent_fp4(H.f(x), c.exp)
        v = O.dequantize_latent_fp4(c.codes, c.scales, c.exp)
        for r in range(2):
            c.ids[r] = np.argsort(order * (q[r, 0] @ v[:1024].T), kind="stable")
        _check(c, KERNELS)


def test_fp4_attention_nan_and_inf_stay():
    """A NaN in a selected row or in q shows in exactly the results that depend on it; a NaN
    in a row that is not selected does not show (every case above has such rows)."""
    for which in KERNELS:
        c = Case(29, 3, 64, 130, [400], hole=0.1)
        t, rows = c.at(1)
        others = set(c.at(0)[1]) | set(c.at(2)[1])
        bad = next(r for r in rows if r not in others)
        c.scales[bad, 2] = O.FP4_NAN_SCALE
        c.q[2, 5, 17] = float("nan")
        with api.mla_kernel(which):
            c.cuda()
            out = torch.empty((3, 64, KVL), dtype=torch.float32, device="cuda")
            c.run(out)
        nan = torch.isnan(out).cpu()
        assert not nan[0].any()
        assert nan[1].all()  # the row's logits with that token are NaN for every head
        assert nan[2, 5].all() and not nan[2, :5].any() and not nan[2, 6:].any()


def test_fp4_attention_bad_ids():
    """Out-of-range tokens, sequences and pages are left out and flagged."""
    for which in KERNELS:
        c = Case(31, 3, 64, 140, [200, 130], block=64, hole=0.1, row_seq=[0, 1, 0])
        with api.mla_kernel(which):
            want, tol = c.want()
            ids = c.ids.copy()
            c.cuda()
            ids[0][ids[0] < 0] = 200
            ids[1][ids[1] < 0] = -2
            c.d_ids.copy_(torch.from_numpy(ids))
            out = torch.empty((3, 64, KVL), dtype=torch.float32, device="cuda")
            c.run(out)
            assert int(c.status) == DSA_STATUS_BAD_TOKEN
            assert (np.abs(out.cpu().numpy() - want) <= tol + 2.0 ** -23 * np.abs(want)).all()
            c.status.zero_()
            c.d_seq.copy_(torch.tensor([0, 2, -1], dtype=torch.int32))
            c.run(out)
            assert int(c.status) == DSA_STATUS_BAD_TOKEN
            assert (out[1:] == 0).all()
            c.status.zero_()
            c.d_seq.copy_(torch.tensor([0, 1, 0], dtype=torch.int32))
            c.d_table[1] = torch.tensor([c.num, -5, 0, 0], dtype=torch.int32)[:c.d_table.shape[1]]
            c.run(out)
            assert int(c.status) & DSA_STATUS_BAD_BLOCK


def test_fp4_attention_is_deterministic_and_per_row():
    """The same bits again, and for a row alone what it gave among others with the same
    number of splits."""
    for which in KERNELS:
        with api.mla_kernel(which):
            c = Case(37, 5, 64, 513, [800, 300], block=16).cuda()
            a, b = (torch.empty((5, 64, KVL), dtype=torch.float32, device="cuda") for _ in range(2))
            c.run(a)
            c.ws.fill_(0x3C)
            c.run(b)
            assert torch.equal(a, b)


def test_fp4_attention_projection():
    """y is the projection of the bf16 olat: the two calls in one give the same bits."""
    for rows, heads, hidden in [(3, 64, 256), (2, 8, 192), (70, 16, 128)]:
        c = Case(41, rows, heads, 200, [300, 100]).cuda()
        A = torch.randn(hidden, heads * KVL, device="cuda").mul_(0.02).to(torch.bfloat16)
        n = api.dsa_sparse_mla_decode_fp4_workspace(rows, heads, 200, hidden, True)
        c.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        y = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
        y2, olat = torch.empty_like(y), torch.empty((rows, heads, KVL), dtype=torch.float32, device="cuda")
        c.run(olat, o_absorb=A, y=y)
        pws = api.dsa_latent_project_workspace(rows, heads, hidden)
        ws = torch.empty(pws, dtype=torch.uint8, device="cuda")
        api.dsa_latent_project(olat, A, y2, workspace=ws)
        assert torch.equal(y, y2)
        y3 = torch.empty_like(y)
        c.run(None, o_absorb=A, y=y3)
        assert torch.equal(y, y3)


def test_fp4_attention_graph_and_streams():
    """Captured and replayed with new contents; two streams with a workspace each."""
    for which in KERNELS:
        with api.mla_kernel(which):
            c = Case(43, 4, 64, 300, [500, 200]).cuda()
            out = torch.empty((4, 64, KVL), dtype=torch.float32, device="cuda")
            c.run(out)
            ref = out.clone()
            q0 = c.d_q.clone()
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                c.run(out)
            c.d_q.copy_(q0.flip(0))
            g.replay()
            c.d_q.copy_(q0)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
            s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
            o1, o2 = torch.empty_like(out), torch.empty_like(out)
            ws2 = torch.empty_like(c.ws)
            torch.cuda.synchronize()
            for _ in range(4):
                c.run(o1, stream=s1)
                ws1, c.ws = c.ws, ws2
                c.run(o2, stream=s2)
                c.ws = ws1
            torch.cuda.synchronize()
            assert torch.equal(o1, ref) and torch.equal(o2, ref)


def test_fp4_attention_many_rows():
    """A prefill-like call: more rows than SMs, several units per CTA."""
    _check(Case(47, 333, 64, 150, [260], hole=0.05), KERNELS, (torch.bfloat16,))


def test_fp4_attention_far_cache_rows():
    """Cache rows past 2^31 bytes of codes."""
    n = (1 << 31) // 256 + 4096
    codes = torch.zeros((n, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, 32), dtype=torch.uint8, device="cuda")
    x = _bf16(np.random.default_rng(3).normal(0, 1, (600, KVL)))
    api.dsa_quantize_latent_fp4(x.cuda(), codes[n - 600:], scales[n - 600:], -8)
    for which in KERNELS:
        with api.mla_kernel(which):
            c = Case(53, 2, 64, 200, [600], hole=0.1)
            c.codes, c.scales = O.quantize_latent_fp4(H.f(x), -8)
            want, tol = c.want()
            c.cuda()
            lens = torch.tensor([n], dtype=torch.int32, device="cuda")
            c.pg = api.paging(lens, n)
            c.d_codes, c.d_scales = codes, scales
            c.d_ids = torch.where(c.d_ids >= 0, c.d_ids + (n - 600), c.d_ids)
            out = torch.empty((2, 64, KVL), dtype=torch.float32, device="cuda")
            c.run(out)
            assert int(c.status) == 0
            assert (np.abs(out.cpu().numpy() - want) <= tol + 2.0 ** -23 * np.abs(want)).all()


def test_fp4_attention_workspace_is_needed():
    c = Case(59, 2, 64, 600, [600]).cuda()
    out = torch.empty((2, 64, KVL), dtype=torch.float32, device="cuda")
    need = api.dsa_sparse_mla_decode_fp4_workspace(2, 64, 600, 0, False)
    assert need > 0
    c.ws = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(Exception, match="workspace"):
        c.run(out)


# -- append and the whole layer --------------------------------------------


@pytest.mark.parametrize("paged", [False, True], ids=["contig", "paged"])
def test_fp4_layer_decode(paged):
    """A layer that grows its FP4 cache (eager, then a replayed graph): its cache rows equal
    the oracle's encoding, its last step that of a layer encoded in one piece, and the
    attention its definition over the decoded cache."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=256, heads=8,
                   hidden=256)
    n = 7
    wl = W.make_workload(f"fp4-append-{int(paged)}", 43, g, [300, 517, 130],
                         block_size=64 if paged else None, max_seq_len=576 if paged else None,
                         invalid_per_seq=3)
    L0 = wl.seq_lens.astype(np.int64) - n
    grow = DsaDecodeLayer(wl, keep_olat=True, decode_from=L0, latent_fp4=True)
    grow.compress()
    for i in range(n):
        grow.stage(i)
        if i == 0:
            grow.append_step()
        else:
            if grow.append_graph is None:
                grow.capture_append()
            grow.append_graph.replay()
    torch.cuda.synchronize()
    assert int(grow.status.item()) == 0
    np.testing.assert_array_equal(grow.seq_lens.cpu().numpy(), wl.seq_lens)
    codes = grow.ckv_codes.view(-1, 256).cpu().numpy()
    scales = grow.ckv_scales.view(-1, 32).cpu().numpy()
    src = wl.ckv.reshape(-1, KVL)
    deq = np.zeros((src.shape[0], KVL))
    for b in range(wl.batch):
        rows = grow._token_rows(b, 0, int(wl.seq_lens[b]))
        c, sc = O.quantize_latent_fp4(H.f(src[torch.from_numpy(rows)]), grow.fp4_exp)
        np.testing.assert_array_equal(codes[rows], c)
        np.testing.assert_array_equal(scales[rows], sc)
        deq[rows] = O.dequantize_latent_fp4(c, sc, grow.fp4_exp)

    whole = DsaDecodeLayer(wl, keep_olat=True, latent_fp4=True, fp4_exp=grow.fp4_exp)
    for b in range(wl.batch):
        rows = torch.from_numpy(whole._token_rows(b, int(L0[b]), int(wl.seq_lens[b])))
        whole.valid.view(-1)[rows.to(whole.valid.device)] = 1
    whole.compress()
    whole.step()
    torch.cuda.synchronize()
    assert int(whole.status.item()) == 0
    for k in ("kpool", "scores", "pool_ids", "token_ids", "olat", "y"):
        assert torch.equal(getattr(grow, k), getattr(whole, k)), k
    for r in range(wl.rows):
        rows = grow._token_rows(r, 0, int(wl.seq_lens[r]))
        o, y, _ = O.sparse_mla_decode_row(H.f(wl.qlat[r]), deq[rows],
                                          grow.token_ids[r].cpu().numpy(), g.softmax_scale,
                                          H.f(wl.o_absorb))
        H.check_attention(grow.y[r].float().cpu().numpy()[None], y[None], f"row {r} y")
        # the projection's inputs: 2^-9 relative would be a bf16 weight's error
        got = grow.olat[r].cpu().numpy()
        assert np.abs(got - o).max() <= 2.0 ** -10 * np.abs(o).max()


def test_fp4_refuses_mixed_devices_and_small_caches():
    c = Case(61, 2, 8, 64, [100]).cuda()
    out = torch.empty((2, 8, KVL), dtype=torch.float32, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_sparse_mla_decode_fp4(c.q, c.d_seq, c.d_codes, c.d_scales, c.exp, c.pg, c.d_ids, c.scale,
                                      olat=out, workspace=c.ws)
    with pytest.raises(ValueError, match="holds 99 rows"):
        api.dsa_sparse_mla_decode_fp4(c.d_q, c.d_seq, c.d_codes[:99], c.d_scales[:99], c.exp, c.pg,
                                      c.d_ids, c.scale, olat=out, workspace=c.ws)
    with pytest.raises(ValueError, match="contiguous"):
        api.dsa_sparse_mla_decode_fp4(c.d_q, c.d_seq, c.d_codes, c.d_scales, c.exp, c.pg, c.d_ids,
                                      c.scale, olat=out.transpose(0, 1).contiguous().transpose(0, 1),
                                      workspace=c.ws)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        api.dsa_sparse_mla_decode_fp4(c.d_q, c.d_seq, c.d_codes, c.d_scales, c.exp, c.pg, c.d_ids,
                                      c.scale, olat=out.half(), workspace=c.ws)


def test_fp4_layer_rejects_two_formats():
    wl = W.tiny()
    with pytest.raises(ValueError, match="one latent cache format"):
        DsaDecodeLayer(wl, latent_fp4=True, latent_fp8=True)
    with pytest.raises(ValueError, match="paged"):
        DsaDecodeLayer(wl, latent_fp4=True, manage_pages=True)
