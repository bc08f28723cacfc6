"""dsa_experts against a plain 64-bit restatement: every pair-tile size in both formats, uneven
and empty experts, padding and bad ids, reuse of a workspace, graphs, streams."""
import math

import pytest
import torch

from sparse_attention_decode_kpool_gb300 import api
from sparse_attention_decode_kpool_gb300._lib import DSA_STATUS_BAD_EXPERT

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _encode(x):
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(*x.shape[:-1], x.shape[-1] // 128, device="cuda")
    api.dsa_quantize_latent(x, codes, scales)
    return codes, scales


def _values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().view(*codes.shape[:-1], -1, 128)
    return (v * scales.double().unsqueeze(-1)).view(codes.shape)


def _hidden(h, fp8):
    """h as the second product takes it."""
    if not fp8:
        return h.float().to(BF16).double()
    a = h.reshape(*h.shape[:-1], -1, 32)
    m, e = torch.frexp(a.abs().amax(-1, keepdim=True))
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    k = torch.where(m > 0, k, torch.zeros_like(k)).double()
    b = a / torch.exp2(k)
    _, be = torch.frexp(b)
    step = torch.exp2((be - 4).clamp(min=-9).double())
    return (torch.round(b / step).mul(step).clamp(-448, 448) * torch.exp2(k)).reshape(h.shape)


class Problem:
    def __init__(self, seed, rows, n, k, hidden, inter, fp8, std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.rows, self.n, self.k, self.hidden, self.inter, self.fp8 = g, rows, n, k, hidden, inter, fp8
        mk = lambda *s, std: (torch.randn(*s, generator=g) * std).to(BF16).cuda()  # noqa: E731
        x, w13, w2 = (mk(rows, hidden, std=std), mk(n, 2 * inter, hidden, std=hidden ** -0.5),
                      mk(n, hidden, inter, std=inter ** -0.5))
        if fp8:
            (self.x, self.xs), (self.w13, self.s13), (self.w2, self.s2) = _encode(x), _encode(w13), _encode(w2)
            self.x64, self.w13_64, self.w2_64 = (_values(self.x, self.xs), _values(self.w13, self.s13),
                                                 _values(self.w2, self.s2))
        else:
            self.x, self.w13, self.w2 = x, w13, w2
            self.xs = self.s13 = self.s2 = None
            self.x64, self.w13_64, self.w2_64 = x.double(), w13.double(), w2.double()
        self.ids = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(rows)]).int().cuda()
        self.weights = torch.softmax(torch.randn(rows, k, generator=g), 1).cuda()
        self.y = torch.full((rows, hidden), math.nan, dtype=BF16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        need = api.dsa_experts_workspace(rows, k, n, hidden, inter, fp8)
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs

    def run(self, **kw):
        api.dsa_experts(self.x, self.ids, self.weights, self.w13, self.w2, self.y, self.xs, self.s13, self.s2,
                        status=self.status, workspace=self.ws, **kw)
        return self.y

    def check(self):
        """|y - exact| within what the arithmetic allows, element by element: bf16's rounding of
        y (2^-8 of it); f32 sums (2 K 2^-24 of the sum of magnitudes: twice a rounding sum's
        bound, for an accumulator that truncates); what a hidden value that lies that near
        to a rounding border may become; and each expert's product's rounding to 11 bits under a
        power of two for 32 channels (2^-11 of it, or of 2^-28 of the largest of the 32: f16's
        smallest step is 2^-24 where the largest lies in [2^14, 2^15))."""
        want = torch.zeros(self.rows, self.hidden, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        u = 2.0 ** -24
        for e in range(self.n):
            row, j = torch.nonzero(self.ids == e, as_tuple=True)
            if not row.numel():
                continue
            x = self.x64[row]
            z, dz = x @ self.w13_64[e].T, 2 * self.hidden * u * (x.abs() @ self.w13_64[e].abs().T)
            (gate, up), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
            silu = gate * torch.sigmoid(gate)
            h = silu * up
            # silu' is at most 1.1; its exponential is off by (2 + |gate|) units, the rest is roundings
            dh = 1.1 * up.abs() * dg + silu.abs() * du + h.abs() * (8 + gate.abs()) * 2 * u
            s = torch.sign(h)
            held = _hidden(h, self.fp8)
            off = torch.maximum((_hidden(h + s * dh, self.fp8) - held).abs(), (_hidden(h - s * dh, self.fp8) - held).abs())
            w2 = self.w2_64[e].T
            wt = self.weights[row, j].double()[:, None]
            p = held @ w2
            want.index_add_(0, row, wt * p)
            least = p.abs().reshape(len(row), -1, 32).amax(2).repeat_interleave(32, 1) * 2.0 ** -28
            tol.index_add_(0, row, wt.abs() * (off @ w2.abs() + 2 * self.inter * u * (held.abs() @ w2.abs())
                                               + 2.0 ** -11 * torch.maximum(p.abs(), least)))
        tol = tol * (1 + 2 * self.k * u) + 2.0 ** -8 * (want.abs() + tol) + self.k * u * want.abs() + 1e-38
        err = (self.y.double() - want).abs()
        assert bool((err <= tol).all()), (float((err / tol).max()), int((err > tol).sum()), err.numel())
        return want


CASES = [
    # rows, experts, topk, hidden, inter: pairs per expert of every tile size
    (1, 1, 1, 128, 128),
    (1, 8, 2, 256, 128),
    (5, 64, 8, 512, 256),
    (16, 4, 2, 384, 128),      # mean 8
    (17, 4, 2, 128, 384),      # mean 9: 32 a tile
    (33, 3, 2, 640, 256),
    (95, 4, 2, 256, 256),      # mean 48
    (97, 4, 2, 256, 128),      # mean 49: 128 a tile
    (190, 5, 2, 128, 128),
    (195, 4, 2, 256, 256),     # mean 98: the largest tile
    (1100, 3, 2, 256, 128),    # several tiles an expert
    (257, 1, 1, 128, 256),
    (40, 100, 3, 1024, 128),
    (600, 40, 4, 256, 768),    # more items than SMs
    (64, 40, 4, 128, 128),     # 256 pairs, ordered by each block
    (257, 40, 1, 256, 128),    # 257, by the dispatch
    (100, 64, 4, 256, 128),    # mean 7: 16 a tile behind the dispatch
    (90, 32, 4, 128, 256),     # mean 12: 32 a tile behind the dispatch
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_experts(case, fp8):
    p = Problem(sum(case), *case, fp8)
    p.run()
    p.check()
    assert int(p.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [6, 70, 400])
def test_uneven_padding_and_bad_ids(rows, fp8):
    p = Problem(rows, rows, 12, 3, 256, 256, fp8)
    p.ids[:, 0] = 7                    # one expert takes every row
    p.ids[:, 1] = torch.where(p.ids[:, 1] == 7, 8, p.ids[:, 1])
    p.ids[:, 2] = torch.where(p.ids[:, 2] > 5, -1, p.ids[:, 2])
    p.ids[rows // 2] = -1              # a row without an expert
    p.ids[-2:] = -1                    # padding
    p.run()
    want = p.check()
    assert not bool(want[rows // 2].any()) and not bool(p.y[rows // 2].any()) and not bool(p.y[-2:].any())
    assert int(p.status) == 0
    p.ids[0, 1], p.ids[1, 2] = 12, -5  # refused one by one
    p.y.fill_(math.nan)
    p.run()
    p.check()
    assert int(p.status) == DSA_STATUS_BAD_EXPERT
    p.status.zero_()
    p.ids.fill_(-1)                    # nobody chose anything
    p.run()
    assert not bool(p.y.any()) and int(p.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("last", [1, 15, 16, 17, 33])
def test_few_pairs_behind_many(last, fp8):
    """Large tiles, and the last expert's pairs so few that half a tile's rows lie behind the end."""
    p = Problem(last, 330, 3, 1, 256, 128, fp8)
    p.ids[:, 0] = torch.arange(330, device="cuda") % 2
    p.ids[100:100 + last, 0] = 2
    p.run()
    p.check()
    assert int(p.status) == 0


def test_odd_number_of_row_tiles():
    """A pair of blocks' second tile of the down product lies behind the last expert's rows."""
    for fp8 in (False, True):
        p = Problem(31, 420, 2, 1, 384, 128, fp8)
        p.run()
        p.check()


def test_output_over_the_input():
    p = Problem(12, 45, 4, 2, 256, 128, False)
    p.run()
    want, x = p.y.clone(), p.x.clone()
    api.dsa_experts(x, p.ids, p.weights, p.w13, p.w2, x, workspace=p.ws)
    assert torch.equal(x, want)
    p.run()
    assert torch.equal(p.y, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_same_expert_twice_counts_twice(fp8):
    p = Problem(3, 9, 4, 2, 128, 128, fp8)
    p.ids[:, 1] = p.ids[:, 0]
    p.run()
    p.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_inf_stay_in_their_row(fp8):
    p = Problem(4, 50, 4, 2, 256, 128, fp8)
    p.run()
    before = p.y.clone()
    if fp8:
        p.x[3, 5] = 0x7F
        p.xs[20, 1] = math.nan
    else:
        p.x[3, 5] = math.nan
        p.x[20, 200] = math.inf
    p.run()
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[[3, 20]] = False
    assert torch.equal(p.y[keep], before[keep])
    assert bool(torch.isnan(p.y[3]).all()) and not bool(torch.isfinite(p.y[20]).any())


@pytest.mark.parametrize("fp8", [False, True])
def test_results_do_not_depend_on_the_other_rows(fp8):
    """A row's result is the same alone, in a batch and on a used workspace (the sums run over
    the same K order whatever the tile)."""
    p = Problem(5, 300, 6, 2, 384, 256, fp8)
    p.run()
    whole = p.y.clone()
    p.run()
    assert torch.equal(p.y, whole)
    for n in (1, 13, 40):
        y = torch.empty(n, p.hidden, dtype=BF16, device="cuda")
        api.dsa_experts(p.x[:n], p.ids[:n].contiguous(), p.weights[:n].contiguous(), p.w13, p.w2, y,
                        None if p.xs is None else p.xs[:n], p.s13, p.s2, workspace=p.ws)
        assert torch.equal(y, whole[:n])


@pytest.mark.parametrize("fp8", [False, True])
def test_experts_in_graphs_and_streams(fp8):
    """Two captured calls share a workspace on one stream and take new inputs at each replay."""
    p, q = Problem(6, 64, 16, 4, 256, 256, fp8), Problem(7, 64, 16, 4, 256, 256, fp8)
    q.ws = p.ws
    p.run()
    q.run()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        p.run()
        q.run()
    for turn in range(3):
        p.ids.copy_(p.ids.roll(1, 0))
        q.weights.mul_(0.5)
        p.y.fill_(math.nan)
        q.y.fill_(math.nan)
        gr.replay()
        torch.cuda.synchronize()
        p.check()
        q.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = p.y.clone()
    p.y.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    p.run(stream=s)
    s.synchronize()
    assert torch.equal(p.y, want)
    gr.reset()


def test_large_activations_fp8_scales():
    """Hidden values far from one in both directions: the 32-channel scales follow them."""
    for std in (1e-4, 30.0):
        p = Problem(8, 40, 4, 2, 256, 256, True, std=std)
        p.run()
        p.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_without_pdl(fp8):
    from sparse_attention_decode_kpool_gb300._lib import DSA_OPT_PDL
    p = Problem(9, 30, 8, 4, 256, 256, fp8)
    p.run()
    want = p.y.clone()
    try:
        api.dsa_set_option(DSA_OPT_PDL, 0)
        p.y.fill_(math.nan)
        p.run()
        torch.cuda.synchronize()
    finally:
        api.dsa_set_option(DSA_OPT_PDL, 1)
    assert torch.equal(p.y, want)
