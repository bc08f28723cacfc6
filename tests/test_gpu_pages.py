"""Page operators on the GPU: every table entry, length, count and cache byte against the
oracle's plain loops, and a decode layer that forks, grows, frees and compacts."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from sparse_attention_decode_kpool_gb300 import api, workloads as W
from sparse_attention_decode_kpool_gb300 import _lib
from sparse_attention_decode_kpool_gb300.pipeline import DsaDecodeLayer

pytestmark = pytest.mark.gpu

FLAGS = {"seq": _lib.DSA_STATUS_BAD_SEQ, "block": _lib.DSA_STATUS_BAD_BLOCK,
         "full": _lib.DSA_STATUS_CACHE_FULL, "pages": _lib.DSA_STATUS_NO_PAGES}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Pool:
    """A pool on the device beside the oracle's."""

    def __init__(self, seed, lens, block, max_blocks, spare, widths=(32, 5, 48), extra_rows=0):
        rng = np.random.default_rng(seed)
        B = len(lens)
        need = [-(-int(n) // block) for n in lens]
        num = sum(need) + spare
        perm = rng.permutation(num)
        table = np.full((B, max_blocks), -1)
        k = 0
        for b in range(B):
            table[b, :need[b]] = perm[k:k + need[b]]
            k += need[b]
        caches = [rng.integers(0, 256, (num, w), dtype=np.uint8) for w in widths]
        self.ref = O.PagePool(table, lens, num, block, caches)
        self.upload()

    def upload(self):
        r = self.ref
        self.table, self.lens, self.refs = _i32(r.table), _i32(r.lens), _i32(r.refs)
        self.caches = [torch.from_numpy(c.copy()).cuda() for c in r.caches]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pg = api.paging(self.lens, r.table.shape[1] * r.bs, self.table, r.bs, r.n)
        self.arrays = api.page_arrays(self.caches, r.n)
        self.ws = torch.full((api.dsa_pages_workspace(r.n, len(r.lens)),), 0x7E, dtype=torch.uint8,
                             device="cuda")

    def free(self, seqs, **kw):
        self.ref.free(seqs)
        api.dsa_pages_free(_i32(seqs), self.pg, self.table, self.lens, self.refs, self.status, **kw)

    def fork(self, parents, children, **kw):
        self.ref.fork(parents, children)
        api.dsa_pages_fork(_i32(parents), _i32(children), self.pg, self.table, self.lens, self.refs,
                           self.status, **kw)

    def reserve(self, new, first_key=0, kpool=0, seqs=None, **kw):
        self.ref.reserve(new, first_key, kpool, seqs)
        api.dsa_pages_reserve(self.pg, self.table, self.refs, new, self.arrays, first_key, kpool,
                              None if seqs is None else _i32(seqs), self.status, self.ws, **kw)

    def compact(self):
        n, remap = self.ref.compact()
        live, got = _i32([-7]), torch.full((self.ref.n,), -7, dtype=torch.int32, device="cuda")
        api.dsa_pages_compact(self.pg, self.table, self.refs, self.arrays, got, live, self.status,
                              self.ws)
        assert int(live) == n
        np.testing.assert_array_equal(got.cpu().numpy(), remap)

    def append(self, k=1):
        """What an append does to the lengths."""
        self.ref.lens += k
        self.lens += k

    def check(self, what=""):
        torch.cuda.synchronize()
        r = self.ref
        np.testing.assert_array_equal(self.table.cpu().numpy(), r.table, err_msg=f"{what} table")
        np.testing.assert_array_equal(self.lens.cpu().numpy(), r.lens, err_msg=f"{what} lens")
        np.testing.assert_array_equal(self.refs.cpu().numpy(), r.refs, err_msg=f"{what} refs")
        for i, (c, w) in enumerate(zip(self.caches, r.caches)):
            np.testing.assert_array_equal(c.cpu().numpy(), w, err_msg=f"{what} cache {i}")
        assert int(self.status) == sum(FLAGS[b] for b in r.bad), (what, int(self.status), r.bad)


def test_pages_free():
    p = Pool(1, [5, 0, 64, 1, 33, 17], 16, 6, 4)
    p.free([2])
    p.check("one")
    p.free([0, -1, 0, 5, 1])  # padding, twice, an empty sequence
    p.check("several")
    p.free([0, 2])  # already free
    p.check("again")
    assert not p.ref.bad
    p.free([6])
    p.free([-2, 3])
    p.check("bad")
    assert p.ref.bad == {"seq"}


def test_pages_free_flags_corrupt_rows():
    p = Pool(2, [40, 40], 16, 4, 2)
    p.ref.table[0, 1] = p.ref.n        # outside the pool
    p.ref.table[1, 0] = -3
    p.ref.refs[p.ref.table[1, 2]] = 0  # held by nobody
    p.upload()
    p.free([0, 1])
    p.check()
    assert p.ref.bad == {"block"}


def test_pages_fork():
    p = Pool(3, [5, 0, 64, 1, 33, 17, 0, 0], 16, 6, 8)
    p.fork([2, 4, 2], [6, 7, 0])  # one parent twice; child 0 held a page
    p.check("fork")
    p.fork([1], [2])  # an empty parent empties the child
    p.check("empty")
    p.fork([6, 0], [-1, 3])
    p.check("padding")
    assert not p.ref.bad


@pytest.mark.parametrize("parents,children", [
    ([0, 1], [3, 3]),      # a child twice: the first counts
    ([0, 3], [3, 2]),      # a parent that the call overwrites
    ([0], [0]),
    ([7, 0], [1, 2]), ([0, 1], [9, 2]), ([-1], [2]),
])
def test_pages_fork_skips(parents, children):
    p = Pool(4, [40, 20, 3, 100], 16, 8, 4)
    p.fork(parents, children)
    p.check()
    assert p.ref.bad == {"seq"}


def test_pages_fork_long_rows():
    """Rows of several chunks of table entries, many children."""
    p = Pool(5, [5000, 2500, 1] + [0] * 9, 2, 2600, 8, widths=())
    p.fork([0, 1, 0, 0, 1, 2, 0], [3, 4, 5, 6, 7, 8, 9])
    p.check("fork")
    p.free(list(range(12)))
    p.check("free")
    assert (p.ref.refs == 0).all()


def test_pages_reserved_pages_are_not_shared():
    p = Pool(6, [16, 3], 16, 6, 6)
    p.reserve(40)
    p.check("reserve")
    p.fork([0], [1])
    p.check("fork")
    p.append()
    p.fork([0], [1])
    p.check("fork again")


@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 40, 100])
def test_pages_reserve(new):
    p = Pool(7, [5, 0, 64, 1, 33, 16, 31], 16, 16, 64)
    p.fork([2, 4], [0, 1])
    p.reserve(new)
    p.check("shared")
    p.append(new)
    p.reserve(new)
    p.check("grown")
    p.reserve(new)
    p.check("again")  # nothing left to do
    # 200 more tokens than 64 exceed neither the pool's 64 spare pages nor the rows' 16
    # below a window of 100
    assert bool(p.ref.bad) == (new == 100)


@pytest.mark.parametrize("first_key", [0, 4, 16, 36])
@pytest.mark.parametrize("new", [1, 3, 9])
def test_pages_reserve_pooled_keys(first_key, new):
    """With first_key > 0 a pooled key is written to a page that is already full of tokens:
    it is copied when shared."""
    p = Pool(8, [63, 64, 43, 1, 51, 40, 3, 0], 16, 12, 80)
    p.fork([0, 1, 4, 2], [7, 6, 3, 5])
    for i in range(6):
        p.reserve(new, first_key, 4)
        p.check(f"step {i}")
        p.append(new)
    assert not p.ref.bad


def test_pages_reserve_lists():
    p = Pool(9, [16, 32, 5, 48, 0], 16, 8, 6)
    p.reserve(1, seqs=[3, -1, 0, 3, 4])
    p.check("list")
    assert not p.ref.bad
    p.reserve(1, seqs=[])
    p.check("empty list")
    p.reserve(1, seqs=[5, 1, -2])
    p.check("bad entries")
    assert p.ref.bad == {"seq"}


def test_pages_reserve_runs_out():
    """Too few pages: sequences in list order, all of a sequence's pages or none."""
    p = Pool(10, [16, 16, 16, 5], 16, 8, 3)
    p.reserve(17, seqs=[1, 0, 2, 3])  # two pages each; the second does not fit any more
    p.check("out")
    assert p.ref.bad == {"pages"}
    q = Pool(11, [16, 20, 16, 16], 16, 8, 0)
    q.fork([1], [0])
    q.reserve(1)
    q.check("freed by the fork")


def test_pages_reserve_full_rows_and_holes():
    p = Pool(12, [32, 31, 64, 10], 16, 4, 20)
    p.ref.table[3, 0] = -1  # a page that should hold tokens
    p.upload()
    p.reserve(1)
    p.check()
    assert p.ref.bad == {"full", "block"}


def test_pages_reserve_huge_window():
    """A prompt's pages: a warp per sequence."""
    p = Pool(13, [0, 100, 16, 7], 4, 700, 2400)
    p.fork([1], [2])
    p.reserve(2300)
    p.check("prompt")
    p.append(2300)
    p.fork([0], [1])
    p.reserve(333, 8, 2)
    p.check("forked prompt")
    assert not p.ref.bad


@pytest.mark.parametrize("n_seq,num", [(3, 40), (40, 5000), (2000, 30000)])
def test_pages_random_life(n_seq, num):
    """Many turns of fork, free, reserve, append and compact."""
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 60, n_seq)
    p = Pool(14, lens, 8, 40, num - int((-(-lens // 8)).sum()) if n_seq < 2000 else 15000)
    for turn in range(8):
        order = rng.permutation(n_seq)
        k = max(1, n_seq // 4)
        p.free(order[:k // 2 + 1])
        p.fork(rng.choice(order[k:], k), order[:k])
        p.check(f"turn {turn} fork")
        p.reserve(int(rng.integers(1, 12)), 8 * int(rng.integers(0, 3)), 4)
        p.check(f"turn {turn} reserve")
        grow = (p.ref.lens >= 0) & (rng.random(n_seq) < 0.8)
        # only sequences whose next token's page is mapped and private grow
        for b in range(n_seq):
            j = int(p.ref.lens[b]) // 8
            ok = j < 40 and p.ref.table[b, j] >= 0 and p.ref.refs[p.ref.table[b, j]] == 1
            grow[b] &= ok
        p.ref.lens += grow
        p.lens += torch.from_numpy(grow).cuda()
        if turn % 3 == 2:
            p.compact()
            p.check(f"turn {turn} compact")


@pytest.mark.parametrize("keep", [[], [0], [5], [0, 1, 2, 3, 4, 5], [1, 3]])
def test_pages_compact(keep):
    p = Pool(15, [40, 100, 3, 64, 0, 17], 16, 8, 9, widths=(4096 + 16, 7, 9000, 16))
    p.free([b for b in range(6) if b not in keep])
    p.compact()
    p.check("compact")
    p.compact()
    p.check("again")
    live = int((p.ref.refs > 0).sum())
    assert (p.ref.refs[:live] > 0).all()


def test_pages_compact_keeps_shared_pages():
    p = Pool(16, [40, 100, 3, 64, 0, 17], 16, 8, 9)
    p.fork([1, 3], [4, 2])
    p.free([0, 1])
    p.compact()
    p.check("one holder each")
    p.fork([4], [0])
    p.compact()
    p.check("two holders")
    assert p.ref.refs.max() == 2


def test_pages_compact_flags_entries_nobody_holds():
    """A table entry at or above the live count that names a free page stays and is flagged."""
    p = Pool(17, [40, 20], 16, 8, 9)
    p.free([0])
    p.ref.table[1, 5] = int(np.flatnonzero(p.ref.refs == 0)[-1])
    p.upload()
    p.compact()
    p.check()
    assert p.ref.bad == {"block"}


def test_pages_without_arrays_and_unaligned_counts():
    """No caches to copy, and counts at an address that is not 16-byte aligned."""
    p = Pool(18, [40, 100, 3], 16, 8, 9, widths=())
    buf = torch.zeros(p.ref.n + 1, dtype=torch.int32, device="cuda")
    buf[1:] = p.refs
    p.refs = buf[1:]
    p.arrays = None
    p.fork([1], [2])
    p.reserve(1)
    p.check("reserve")
    p.free([0])
    p.compact()
    p.check("compact")


def test_pages_graph_replay_and_streams():
    """A captured turn replayed: the decisions are taken from the state at replay."""
    p = Pool(19, [16, 5, 31, 0, 0, 47], 16, 12, 40)
    parents, kids, ended = _i32([0, 5]), _i32([3, 4]), _i32([1, -1])

    def turn():
        api.dsa_pages_free(ended, p.pg, p.table, p.lens, p.refs, p.status)
        api.dsa_pages_fork(parents, kids, p.pg, p.table, p.lens, p.refs, p.status)
        api.dsa_pages_reserve(p.pg, p.table, p.refs, 1, p.arrays, 0, 4, None, p.status, p.ws)

    def ref_turn(e, pa, k):
        p.ref.free(e)
        p.ref.fork(pa, k)
        p.ref.reserve(1, 0, 4)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        turn()
    torch.cuda.current_stream().wait_stream(s)
    ref_turn([1], [0, 5], [3, 4])
    p.check("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        turn()
    for e, pa, k in [([0, -1], [3, 2], [5, 1]), ([4, 4], [1, 1], [0, 3]), ([-1, -1], [2, 2], [-1, 4])]:
        ended.copy_(_i32(e))
        parents.copy_(_i32(pa))
        kids.copy_(_i32(k))
        p.append()
        g.replay()
        ref_turn(e, pa, k)
        p.check(str((e, pa, k)))
    assert not p.ref.bad


def test_pages_on_a_stream_of_their_own():
    """Lists made on the stream that reads them, calls ordered on it."""
    p = Pool(23, [40, 100, 3, 64, 0, 17], 16, 10, 30)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.fork([1, 3], [4, 2])
    p.reserve(5, stream=s)
    with torch.cuda.stream(s):
        p.free([0])
    s.synchronize()
    p.check()


def test_pages_layer_life():
    """A decode layer with the FP4 cache and managed pages: forked sequences fed the same
    tokens give the parent's bits at every step, wherever their pages are."""
    g = W.Geometry(index_kpool=4, index_heads=32, index_head_dim=128, index_topk=128, heads=8,
                   hidden=256)
    wl = W.make_workload("fp4-pages", 47, g, [300, 517, 130, 260], block_size=64,
                         max_seq_len=1024, invalid_per_seq=0)
    # queries and staged tokens equal for all rows, so that rows with equal caches agree
    L0 = np.array([250, 400, 60, 200])
    lay = DsaDecodeLayer(wl, keep_olat=True, decode_from=L0, latent_fp4=True, manage_pages=True)
    lay.compress()
    for t in (lay.qidx, lay.w, lay.qlat):
        t.copy_(t[:1].expand_as(t).clone())
    lay.fork_sequences([0, 1], [2, 3])

    def stage(i):
        k, gt, c = lay.staged_rows(i)
        for dst, src in ((lay.k_new, k), (lay.gate_new, gt), (lay.ckv_new, c)):
            dst.copy_(src[:1].expand_as(src).to(dst.device))

    def same(a, b, what):
        torch.cuda.synchronize()
        assert int(lay.status.item()) == 0, what
        for k in ("scores", "token_ids", "olat", "y"):
            assert torch.equal(getattr(lay, k)[a], getattr(lay, k)[b]), (what, k)

    for i in range(10):  # crosses a page's end (250 -> 260)
        stage(i)
        if i < 2:
            lay.append_step()
        else:
            if lay.append_graph is None:
                lay.capture_append()
            lay.append_graph.replay()
        same(0, 2, f"step {i}")
        same(1, 3, f"step {i}")
    assert not torch.equal(lay.olat[0], lay.olat[1])
    tables = lay.block_table.cpu().numpy()
    held = int(lay.seq_lens[0])
    full = held // 64
    assert (tables[0, :full - 1] == tables[2, :full - 1]).all()  # still shared
    assert tables[0, full] != tables[2, full]                     # written apart
    before = lay.olat.clone()
    lay.free_sequences([3])
    lay.compact_pages()
    lay.step()
    torch.cuda.synchronize()
    assert int(lay.status.item()) == 0
    live = int(lay.pages_live)
    assert live == int((lay.refs > 0).sum()) and (lay.refs[:live] > 0).all()
    assert int(lay.block_table.max()) < live
    for r in (0, 1, 2):
        assert torch.equal(lay.olat[r], before[r])
    # divergence: different tokens from here on
    lay.fork_sequences([0], [3])
    lay.step()  # the child sees the parent's context before any append
    same(0, 3, "at the fork")
    stage(10)
    lay.ckv_new[3] = lay.ckv_new[3].flip(0)
    lay.k_new[3] = lay.k_new[3].flip(0)
    for i in range(4):
        lay.append_step()
    torch.cuda.synchronize()
    same(0, 2, "after the fork")
    assert not torch.equal(lay.olat[0], lay.olat[3])
