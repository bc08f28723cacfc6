"""Appends to pools whose pages are shared: what each sequence reads back is what a private
cache that saw its own tokens alone would hold, whether or not the pool has pages left."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import _lib, api, workloads as W
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer

pytestmark = pytest.mark.gpu

IHD, KVL, KP, BS, EPS = 128, 512, 4, 16, 1e-6
FORMATS = ("bf16", "fp8", "fp4")
# cache name -> (width, type); token caches first
TOKEN = {"k_raw": (IHD, torch.bfloat16), "gate": (IHD, torch.bfloat16), "valid": (1, torch.uint8)}
LATENT = {"bf16": {"ckv": (KVL, torch.bfloat16)},
          "fp8": {"codes": (KVL, torch.uint8), "scales": (KVL // 128, torch.float32)},
          "fp4": {"codes": (KVL // 2, torch.uint8), "scales": (KVL // 16, torch.uint8)}}
POOLED = {"kpool": (IHD, torch.bfloat16), "pvalid": (1, torch.uint8)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Shared:
    """A paged pool on the device beside one private contiguous cache per sequence."""

    def __init__(self, fmt, lens, max_blocks, spare, first_key, seed=0):
        self.fmt, self.fk = fmt, first_key
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        B = len(lens)
        need = [-(-n // BS) for n in lens]
        num = sum(need) + spare
        perm = np.random.default_rng(seed).permutation(num)
        table = np.full((B, max_blocks), -1)
        k = 0
        for b in range(B):
            table[b, :need[b]] = perm[k:k + need[b]]
            k += need[b]
        self.ref = O.PagePool(table, lens, num, BS)
        self.B, self.cap = B, max_blocks * BS
        self.widths = {**TOKEN, **LATENT[fmt], **POOLED}
        self.caches = {n: self._rand((num * (BS // KP if n in POOLED else BS), w), dt)
                       for n, (w, dt) in self.widths.items()}
        self.caches["valid"].fill_(1)
        self.ape = torch.randn(KP, IHD, generator=self.g, device="cuda") * 0.1
        self.ln_w, self.ln_b = self._rand((IHD,), torch.bfloat16), self._rand((IHD,), torch.bfloat16)
        self.table, self.lens, self.refs = _i32(table), _i32(lens), _i32(self.ref.refs)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pg = api.paging(self.lens, self.cap, self.table, BS, num)
        self.arrays = api.page_arrays(
            [c.view(num, -1) for c in self.caches.values()], num)
        self.ws = torch.empty(api.dsa_pages_workspace(num, B), dtype=torch.uint8, device="cuda")
        # pooled keys of the tokens there are, by the library's own one-shot form
        c = self.caches
        api.dsa_compress(c["k_raw"], c["gate"], c["valid"], self.ape, self.ln_w, self.ln_b, EPS,
                         self.pg, self.fk, KP, c["kpool"], c["pvalid"])
        self.own = [{n: self._rows(b, n, lens[b]) for n in self.widths} for b in range(B)]

    def _rand(self, shape, dt):
        if dt == torch.uint8:
            return torch.randint(0, 256, shape, generator=self.g, device="cuda", dtype=dt)
        return torch.randn(shape, generator=self.g, device="cuda").to(dt)

    def _at(self, b, name, n):
        """Rows of the paged cache that hold sequence b's first n tokens (or their pools)."""
        per = BS // KP if name in POOLED else BS
        count = O.pools_completed(0, n, self.fk, KP).stop if name in POOLED else n
        t = np.arange(count)
        at = self.ref.table[b][t // per] * per + t % per
        return torch.from_numpy(at.astype(np.int64)).cuda()

    def _rows(self, b, name, n):
        """A private cache of self.cap tokens (or their pools): sequence b's rows, then zeros."""
        rows = self.cap // KP if name in POOLED else self.cap
        out = torch.zeros((rows, self.widths[name][0]), dtype=self.widths[name][1], device="cuda")
        at = self._at(b, name, n)
        out[:len(at)] = self.caches[name][at]
        return out

    def fork(self, parents, children):
        self.ref.fork(parents, children)
        api.dsa_pages_fork(_i32(parents), _i32(children), self.pg, self.table, self.lens,
                           self.refs, self.status)
        for p, c in zip(parents, children):
            self.own[c] = {n: t.clone() for n, t in self.own[p].items()}

    def free(self, seqs):
        self.ref.free(seqs)
        api.dsa_pages_free(_i32(seqs), self.pg, self.table, self.lens, self.refs, self.status)

    def _call(self, c, pg, lens, new, **kw):
        k, gt, ckv = new
        common = (pg, lens, self.fk, KP, c["k_raw"], c["gate"], c["valid"])
        if self.fmt == "bf16":
            api.dsa_decode_append(k, gt, self.ape, self.ln_w, self.ln_b, EPS, *common, c["kpool"],
                                  c["pvalid"], ckv_new=ckv, ckv=c["ckv"], **kw)
        elif self.fmt == "fp8":
            api.dsa_decode_append_fp8(k, gt, ckv, self.ape, self.ln_w, self.ln_b, EPS, *common,
                                      c["codes"], c["scales"], c["kpool"], c["pvalid"], **kw)
        else:
            api.dsa_decode_append_fp4(k, gt, ckv, self.ape, self.ln_w, self.ln_b, EPS, *common,
                                      c["codes"], c["scales"], -8, c["kpool"], c["pvalid"], **kw)

    def step(self, serving=None):
        """Reserve and append one token each; returns who was stored."""
        self.ref.reserve(1, self.fk, KP)
        api.dsa_pages_reserve(self.pg, self.table, self.refs, 1, self.arrays, self.fk, KP,
                              status=self.status, workspace=self.ws)
        new = tuple(self._rand((self.B, w), torch.bfloat16) for w in (IHD, IHD, KVL))
        go = [self.ref.holds_alone(b, self.fk, KP) and (serving is None or serving[b] >= 0)
              for b in range(self.B)]
        self._call(self.caches, self.pg, self.lens, new, row_ctx=self.ctx, status=self.status,
                   refs=self.refs, serving=None if serving is None else _i32(serving))
        for b in range(self.B):
            if go[b]:  # the same token into the private cache
                one = _i32([self.ref.lens[b]])
                self._call({n: t.view(1, *t.shape) for n, t in self.own[b].items()},
                           api.paging(one, self.cap), one, tuple(x[b:b + 1] for x in new))
                self.ref.lens[b] += 1
        return go

    def check(self, what):
        torch.cuda.synchronize()
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.ref.lens, err_msg=str(what))
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.ref.table, err_msg=str(what))
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.ref.refs, err_msg=str(what))
        for b in range(self.B):
            for n in self.widths:
                at = self._at(b, n, int(self.ref.lens[b]))
                assert torch.equal(self.caches[n][at].view(torch.uint8),
                                   self.own[b][n][:len(at)].view(torch.uint8)), (what, b, n)


@pytest.mark.parametrize("first_key", [0, 8])
@pytest.mark.parametrize("fmt", FORMATS)
def test_append_leaves_shared_pages_alone(fmt, first_key):
    """Two children of one parent in a full pool: nobody stores into the pages they share,
    and all go on once there are pages again."""
    p = Shared(fmt, [20, 16, 0, 0, 47, 112], 8, 0, first_key)
    p.fork([0, 0], [2, 3])
    before = {n: c.clone() for n, c in p.caches.items()}
    for i in range(3):
        go = p.step()
        assert go[0] == go[2] == go[3] == go[1] is False  # shared, shared, shared, no new page
        p.check(i)
        assert int(p.status) & _lib.DSA_STATUS_NO_PAGES
        assert torch.equal(p.ctx, p.lens)
    shared = p._at(0, "k_raw", 20)
    for n in TOKEN:
        assert torch.equal(before[n][shared], p.caches[n][shared])
    p.free([1, 4, 5])
    p.status.zero_()
    stored = [p.step() for _ in range(6)]
    p.check("pages again")
    assert stored[-1][0] and stored[-1][2] and stored[-1][3]


@pytest.mark.parametrize("first_key", [0, 8, 16])
@pytest.mark.parametrize("spare", [1, 3, 5])
def test_append_runs_out_and_recovers(spare, first_key):
    """Pages run out somewhere along the way: with first_key > 0 also where only the pooled
    key's page is still shared."""
    p = Shared("fp4", [31, 16, 5, 0, 0, 64], 8, spare, first_key, seed=spare)
    p.fork([0, 1], [3, 4])
    seen = set()
    for i in range(22):
        go = p.step()
        p.check(i)
        seen.add(tuple(go))
        if i == 12:
            p.free([5])
            p.fork([4], [5])
    assert len(seen) > 1 and int(p.status) & _lib.DSA_STATUS_NO_PAGES


def test_append_pooled_key_page_alone_is_shared():
    """The token's own page is private, the page of the pooled key it completes is not."""
    p = Shared("bf16", [16, 0], 4, 2, 8)
    p.fork([0], [1])
    for i in range(3):  # tokens 16, 17, 18 in private pages; none completes a pool
        assert p.step() == [True, True]
        p.check(i)
    assert p.step() == [False, False]  # token 19 completes pool 2, in the shared page 0
    p.check("refused")
    assert int(p.status) == _lib.DSA_STATUS_NO_PAGES


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_serving_list(fmt):
    """Sequences with a negative entry stay as they are, without a flag, whatever page they
    would be written to."""
    p = Shared(fmt, [20, 16, 3, 47], 8, 6, 0)
    for i, s in enumerate(([0, -1, 2, -1], [-1, -1, -1, -1], [0, 1, -1, 3])):
        go = p.step(s)
        assert go == [x >= 0 for x in s]
        p.check(i)
        assert torch.equal(p.ctx, p.lens)
    assert int(p.status) == 0


def test_guarded_append_without_refusal_equals_the_plain_one():
    for fmt in FORMATS:
        a, b = (Shared(fmt, [20, 16, 3, 47], 8, 20, 8, seed=4) for _ in range(2))
        for s in (a, b):
            api.dsa_pages_reserve(s.pg, s.table, s.refs, 12, s.arrays, 8, KP, workspace=s.ws)
        for _ in range(9):
            new = tuple(a._rand((4, w), torch.bfloat16) for w in (IHD, IHD, KVL))
            a._call(a.caches, a.pg, a.lens, new, row_ctx=a.ctx)
            b._call(b.caches, b.pg, b.lens, new, row_ctx=b.ctx, refs=b.refs, status=b.status)
        assert int(b.status) == 0 and torch.equal(a.lens, b.lens) and torch.equal(a.ctx, b.ctx)
        for n in a.widths:
            assert torch.equal(a.caches[n].view(torch.uint8), b.caches[n].view(torch.uint8)), (fmt, n)


@pytest.mark.parametrize("kw", [{}, {"latent_fp8": True}, {"latent_fp4": True}], ids=FORMATS)
def test_layer_out_of_pages(kw):
    """A layer whose pool is full after a fork: captured steps leave both holders and their
    pages as they are, and go on when pages are free again."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=128, heads=8,
                   hidden=256)
    wl = W.make_workload("full-pool", 51, g, [300, 517, 130], block_size=64, max_seq_len=1024,
                         invalid_per_seq=0)
    lay = DsaDecodeLayer(wl, keep_olat=True, decode_from=np.array([200, 260, 60]),
                         manage_pages=True, **kw)
    lay.compress()
    for t in (lay.qidx, lay.w, lay.qlat):
        t.copy_(t[:1].expand_as(t).clone())
    lay.fork_sequences([0], [2])
    free = lay.refs == 0
    lay.refs[free] = 1  # everything else belongs to somebody
    lay.stage(0)
    lay.capture_append()
    page = int(lay.block_table[0, 200 // 64])
    held = [c[page].clone() for c in lay._paged]
    for _ in range(3):
        lay.append_graph.replay()
    torch.cuda.synchronize()
    assert int(lay.status) == _lib.DSA_STATUS_NO_PAGES
    assert lay.seq_lens.tolist() == [200, 263, 200] and lay.row_ctx.tolist() == [200, 263, 200]
    assert torch.equal(lay.block_table[0], lay.block_table[2]) and int(lay.refs[page]) == 2
    for c, h in zip(lay._paged, held):
        assert torch.equal(c[page].view(torch.uint8), h.view(torch.uint8))
    lay.status.zero_()
    lay.refs[free] = 0
    k, gt, c = lay.staged_rows(1)
    for dst, src in ((lay.k_new, k), (lay.gate_new, gt), (lay.ckv_new, c)):
        dst.copy_(src[:1].expand_as(src).to(dst.device))
    for _ in range(2):
        lay.append_graph.replay()
    torch.cuda.synchronize()
    assert int(lay.status) == 0 and lay.seq_lens.tolist() == [202, 265, 202]
    assert int(lay.block_table[0, 3]) != int(lay.block_table[2, 3])
    for name in ("scores", "token_ids", "olat", "y"):
        assert torch.equal(getattr(lay, name)[0], getattr(lay, name)[2]), name


def test_pages_serve():
    """The list against plain loops: padding, repeats, entries out of range, fork's pairs."""
    B = 600
    serving, status = torch.arange(B, dtype=torch.int32, device="cuda"), _i32([0])
    want = np.arange(B)
    api.dsa_pages_serve(_i32([3, -1, 3, 599, 0]), serving, False, status=status)
    want[[3, 599, 0]] = -1
    assert serving.tolist() == want.tolist() and int(status) == 0
    api.dsa_pages_serve(_i32([0, 5]), serving, status=status)
    want[0] = 0
    api.dsa_pages_serve(_i32([]), serving, False, status=status)
    assert serving.tolist() == want.tolist() and int(status) == 0
    api.dsa_pages_serve(_i32([600, -2, 7]), serving, False, status=status)
    want[7] = -1
    assert serving.tolist() == want.tolist() and int(status) == _lib.DSA_STATUS_BAD_SEQ
    for parents, children, on in [([1, 2], [3, 599], [3, 599]), ([1, -1], [3, 7], [3]),
                                  ([1, 3], [3, 7], [3]), ([7], [7], []), ([1, 2], [3, 3], [3]),
                                  ([1, 700, 1], [-1, 3, 7], [7])]:
        want[[3, 7, 599]] = -1
        api.dsa_pages_serve(_i32([3, 7, 599]), serving, False)
        status.zero_()
        api.dsa_pages_serve(_i32(children), serving, True, _i32(parents), status)
        want[on] = on
        assert serving.tolist() == want.tolist(), (parents, children)
        bad = len(on) < sum(c != -1 for c in children)
        assert int(status) == (_lib.DSA_STATUS_BAD_SEQ if bad else 0)


@pytest.mark.parametrize("kw", [{}, {"latent_fp8": True}, {"latent_fp4": True}], ids=FORMATS)
def test_layer_ended_and_paused_sequences(kw):
    """Through captured steps an ended sequence stays ended and a paused one keeps its
    tokens, pages and results; forked over and resumed they grow."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=128, heads=8,
                   hidden=256)
    wl = W.make_workload("ended", 52, g, [300, 517, 130, 260], block_size=64, max_seq_len=1024,
                         invalid_per_seq=0)
    lay = DsaDecodeLayer(wl, keep_olat=True, decode_from=np.array([200, 260, 60, 190]),
                         manage_pages=True, **kw)
    lay.compress()
    lay.stage(0)
    lay.capture_append()
    lay.step()
    paused = lay.olat[1].clone()
    gone = lay.block_table[3][lay.block_table[3] >= 0].long()
    lay.free_sequences([3])
    lay.pause_sequences([1])
    live = int((lay.refs > 0).sum())
    for _ in range(70):  # past a page's end
        lay.append_graph.replay()
    torch.cuda.synchronize()
    assert int(lay.status) == 0
    assert lay.seq_lens.tolist() == [270, 260, 130, 0] == lay.row_ctx.tolist()
    assert (lay.block_table[3] == -1).all() and (lay.olat[3] == 0).all()
    assert torch.equal(lay.olat[1], paused)
    assert int((lay.refs > 0).sum()) == live + 3  # sequence 0: token 256; 2: 64 and 128
    lay.fork_sequences([1], [3])
    lay.resume_sequences([1, -1])
    lay.append_graph.replay()
    torch.cuda.synchronize()
    assert int(lay.status) == 0 and lay.seq_lens.tolist() == [271, 261, 131, 261]
    lay.free_sequences([2, 3])
    lay.resume_sequences([3])
    for _ in range(2):
        lay.append_graph.replay()
    torch.cuda.synchronize()
    assert int(lay.status) == 0 and lay.seq_lens.tolist() == [273, 263, 0, 2]
    assert int((lay.block_table[3] >= 0).sum()) == 1 and len(gone) == 3
    lay.fork_sequences([7], [2])  # a refused pair starts nothing
    lay.append_graph.replay()
    assert int(lay.status) == _lib.DSA_STATUS_BAD_SEQ and int(lay.seq_lens[2]) == 0


def test_descriptors_of_another_device_are_refused():
    """A descriptor whose tensors live on another device than the call's (its note of the
    device is changed here; nothing is launched)."""
    p = Shared("fp4", [20, 16], 8, 6, 0)
    c, new = p.caches, tuple(p._rand((2, w), torch.bfloat16) for w in (IHD, IHD, KVL))
    before = p.refs.clone()

    def calls():
        yield lambda: p._call(c, p.pg, p.lens, new)
        yield lambda: p._call(c, p.pg, p.lens, new, refs=p.refs)
        yield lambda: api.dsa_pages_free(_i32([0]), p.pg, p.table, p.lens, p.refs)
        yield lambda: api.dsa_pages_fork(_i32([0]), _i32([1]), p.pg, p.table, p.lens, p.refs)
        for f in reserve, compact:
            yield f
        q = torch.zeros((2, 8, KVL), dtype=torch.bfloat16, device="cuda")
        yield lambda: api.dsa_sparse_mla_decode_fp4(q, None, c["codes"], c["scales"], -8, p.pg,
                                                    p.table, 1.0, olat=q)

    def reserve():
        api.dsa_pages_reserve(p.pg, p.table, p.refs, 1, p.arrays, workspace=p.ws)

    def compact():
        api.dsa_pages_compact(p.pg, p.table, p.refs, p.arrays, workspace=p.ws)

    assert p.pg.device == p.arrays.device == 0
    p.pg.device = 1
    for f in calls():
        with pytest.raises(ValueError, match="pg describes tensors on cuda:1"):
            f()
    p.pg.device, p.arrays.device = 0, 1
    for f in reserve, compact:
        with pytest.raises(ValueError, match="arrays describes tensors on cuda:1"):
            f()
    torch.cuda.synchronize()
    assert torch.equal(p.refs, before) and p.lens.tolist() == [20, 16]
    with pytest.raises(ValueError, match="cache 1 must be a CUDA tensor|cache 1 is on"):
        api.page_arrays([p.refs, p.refs.cpu()], len(p.refs))
    with pytest.raises(ValueError, match="block_table"):
        api.paging(p.lens, 64, p.table.cpu(), BS, 4)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_serving_list_contiguous(fmt):
    """A contiguous cache, where there are no counts: the list alone, on a stream of its own."""
    p = Shared(fmt, [20, 16, 3], 2, 0, 0)
    c = {n: torch.stack([o[n] for o in p.own]) for n in p.widths}
    plain = {n: t.clone() for n, t in c.items()}
    lens, want = _i32([20, 16, 3]), _i32([20, 16, 3])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for serving in ([0, -1, 2], [-1, 1, -1], [-1, -1, -1]):
            new = tuple(p._rand((3, w), torch.bfloat16) for w in (IHD, IHD, KVL))
            p._call(c, api.paging(lens, p.cap), lens, new, serving=_i32(serving), status=status)
            for b in range(3):
                if serving[b] >= 0:
                    p._call({n: t[b:b + 1] for n, t in plain.items()},
                            api.paging(want[b:b + 1], p.cap), want[b:b + 1],
                            tuple(x[b:b + 1] for x in new))
        assert int(status) == 0 and lens.tolist() == want.tolist() == [21, 17, 4]
        for n in c:
            assert torch.equal(c[n].view(torch.uint8), plain[n].view(torch.uint8)), n
    s.synchronize()
