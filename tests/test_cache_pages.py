"""Fork, free, copy and compaction of pages against the oracle's plain loops: books and
pages are equal to the last bit."""
import numpy as np
import pytest
import torch

from mla_decode_attention_15_b200 import _build, binding as bd, cache as ca
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    return torch.device("cuda:0")


class World:
    """A pool and its books, on the GPU and as the oracle's numpy copy."""

    def __init__(self, lens, nb, dev, q8=True, rows=None, width=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        rows = rows or len(lens)
        width = width or max(oc.pages_of(n) for n in lens) + 1
        ids = torch.randperm(nb, generator=g).int()
        bt = torch.full((rows, width), -7, dtype=torch.int32)  # unused entries are nobody's
        k = 0
        for b, n in enumerate(lens):
            bt[b, :oc.pages_of(n)] = ids[k:k + oc.pages_of(n)]
            k += oc.pages_of(n)
        assert k <= nb
        full = torch.zeros(rows, dtype=torch.int32)
        full[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
        refs = torch.zeros(nb, dtype=torch.int32)
        refs[ids[:k].long()] = 1
        pool = torch.randint(0, 256, (nb, 64, 1, 576 * (1 if q8 else 2)), generator=g, dtype=torch.uint8)
        self.scales = torch.randn(nb, 1, generator=g) if q8 else None
        self.np = dict(bt=bt.numpy().copy(), lens=full.numpy().copy(), refs=refs.numpy().copy(), pool=pool.numpy().copy(),
                       scales=self.scales.numpy().copy() if q8 else None)
        self.bt, self.lens, self.refs = bt.to(dev), full.to(dev), refs.to(dev)
        self.pool = pool.to(dev).view(torch.float8_e4m3fn if q8 else torch.bfloat16)
        self.scales = self.scales.to(dev) if q8 else None
        self.status, self.dev = torch.zeros(1, dtype=torch.int32, device=dev), dev

    def t(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.dev)

    def moved(self, copies):
        old = self.np["pool"].copy(), None if self.scales is None else self.np["scales"].copy()
        for s, d in copies:
            self.np["pool"][d] = old[0][s]
            if self.scales is not None:
                self.np["scales"][d] = old[1][s]

    def fork(self, parents, children, stream=None):
        ca.cache_fork(self.t(parents), self.t(children), self.bt, self.lens, self.refs, self.pool, self.scales, status=self.status,
                      stream=stream)
        self.moved(oc.fork(parents, children, self.np["bt"], self.np["lens"], self.np["refs"]))

    def free(self, rows):
        ca.cache_free(self.t(rows), self.bt, self.lens, self.refs, status=self.status)
        oc.free(rows, self.np["bt"], self.np["lens"], self.np["refs"])

    def compact(self, workspace=None):
        ca.cache_compact(self.bt, self.lens, self.refs, self.pool, self.scales, workspace=workspace, status=self.status)
        self.moved(oc.compact(self.np["bt"], self.np["lens"], self.np["refs"]))

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status) == status
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.np["lens"])
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.np["refs"])
        np.testing.assert_array_equal(self.bt.cpu().numpy(), self.np["bt"])
        np.testing.assert_array_equal(self.pool.view(torch.uint8).cpu().numpy(), self.np["pool"])
        if self.scales is not None:
            np.testing.assert_array_equal(self.scales.cpu().numpy(), self.np["scales"])


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("lens,times", [([1], 1), ([64], 2), ([65, 128, 63, 0], 2), ([1000, 77, 640, 5], 3)])
def test_fork(dev, lens, times, q8):
    n = len(lens) * times
    w = World(lens, sum(oc.pages_of(x) for x in lens) + n, dev, q8, rows=len(lens) + n, seed=n)
    w.fork([i % len(lens) for i in range(n)], list(range(len(lens) + n - 1, len(lens) - 1, -1)))
    w.check()


def test_fork_of_many_rows_and_of_forks(dev):
    w = World([100] * 10, 1200, dev, rows=1034, seed=4)
    w.fork([i % 10 for i in range(1024)], list(range(10, 1034)))
    w.check()
    w = World([200, 64], 40, dev, rows=8, seed=5)
    w.fork([0, 0], [2, 3])
    w.fork([2, 3, 1], [4, 5, 6])
    w.free([0, 2])
    w.fork([4], [0])
    w.check()


def test_fork_takes_parents_as_they_were(dev):
    w = World([200, 64], 40, dev, rows=6, seed=9)
    w.fork([0, 2, 1, 2], [2, 3, 4, 5])
    w.check()
    assert w.lens.tolist() == [200, 64, 200, 0, 64, 0]


def test_fork_refusals(dev):
    """Rows outside the batch, a child in use, a child named twice, itself: left out. The rest goes on."""
    w = World([100, 200, 30], 40, dev, rows=8, seed=6)
    w.fork([0, 9, -1, 1, 1, 2, 0, 0], [3, 4, 4, 2, 5, 5, 8, 0])
    w.check(ca.MLA_STATUS_BAD_ROW)
    assert w.lens.tolist() == [100, 200, 30, 100, 0, 200, 0, 0]
    # a pool without room: the first forks that need a page get the last ones; those that need none go on
    w = World([100, 128, 30], 2 + 2 + 1 + 1, dev, rows=8, seed=7)
    w.fork([0, 2, 1, 0], [3, 4, 5, 6])
    w.check(ca.MLA_STATUS_NO_FREE_PAGE)
    assert w.lens.tolist() == [100, 128, 30, 100, 0, 128, 0, 0]
    # bad entries of the parent: in the last page, and among the full ones
    w = World([100, 200], 40, dev, rows=4, seed=8)
    w.bt[0, 1] = 40
    w.bt[1, 0] = -2
    ca.cache_fork(w.t([0, 1]), w.t([2, 3]), w.bt, w.lens, w.refs, w.pool, w.scales, status=w.status)
    torch.cuda.synchronize()
    assert int(w.status) == bd.MLA_STATUS_BAD_BLOCK_TABLE and w.lens.tolist() == [100, 200, 0, 200]
    assert int(w.bt[3, 0]) == -2
    # a parent's length past its table
    w = World([100], 40, dev, rows=2, seed=8)
    w.lens[0] = 64 * w.bt.shape[1] + 1
    ca.cache_fork(w.t([0]), w.t([1]), w.bt, w.lens, w.refs, w.pool, w.scales, status=w.status)
    torch.cuda.synchronize()
    assert int(w.status) == ca.MLA_STATUS_BAD_ROW and int(w.lens[1]) == 0


def test_free(dev):
    w = World([100, 200, 30, 0, 64], 20, dev, seed=9)
    w.free([1, 1, 3, 4])
    w.check()
    w.free([-1, 5, 0])
    w.check(ca.MLA_STATUS_BAD_ROW)
    w = World([100, 200], 20, dev, seed=9)
    w.refs[w.bt[0, 1].long()] = 0
    w.bt[1, 2] = 999
    ca.cache_free(w.t([0, 1]), w.bt, w.lens, w.refs, status=w.status)
    torch.cuda.synchronize()
    assert int(w.status) == ca.MLA_STATUS_BAD_REF_COUNT | bd.MLA_STATUS_BAD_BLOCK_TABLE
    assert int(w.refs.sum()) == 1 and int(w.refs.min()) == 0  # the page whose entry was lost stays counted


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("lens,gone,extra", [([64], [], 0), ([64], [0], 3), ([300, 64, 1000, 5], [0], 0), ([300, 64, 1000, 5], [2, 1], 7),
                                             ([640] * 12, [0, 3, 5, 6, 11], 200)])
def test_free_then_compact(dev, lens, gone, extra, q8):
    w = World(lens, sum(oc.pages_of(x) for x in lens) + extra, dev, q8, seed=len(lens) + extra)
    if gone:
        w.free(gone)
    ws = ca.cache_compact_workspace(w.pool.shape[0], dev)
    w.compact(ws)
    w.check()
    live = int((w.np["refs"] > 0).sum())
    assert int(ws.view(torch.int32)[0]) == live and not w.refs[live:].any()
    w.compact(ws)  # packed already: nothing moves
    w.check()


def test_compact_shared_pages_and_large_books(dev):
    w = World([500, 200, 70], 300, dev, rows=9, seed=12)
    w.fork([0, 0, 1, 2], [3, 4, 5, 6])
    w.free([0, 2])
    w.compact()
    w.check()
    # more pages than one pass of the planning block, with holes everywhere
    nb = 9001
    pool = torch.zeros(nb, 64, 1, 576, dtype=torch.uint8, device=dev)
    pool[:, 0, 0, :4] = torch.arange(nb, dtype=torch.int32, device=dev).view(torch.uint8).view(nb, 4)
    refs = torch.from_numpy((np.random.RandomState(3).rand(nb) < 0.4).astype(np.int32))
    held = torch.nonzero(refs)[:, 0].int()
    bt = held[torch.randperm(len(held), generator=torch.Generator().manual_seed(1))][None].contiguous()
    lens = torch.tensor([64 * len(held)], dtype=torch.int32)
    n_bt, n_refs = bt.numpy().copy(), refs.numpy().copy()
    g = [x.to(dev) for x in (bt, lens, refs)]
    scales = torch.arange(nb, dtype=torch.float32, device=dev)[:, None].contiguous()
    ca.cache_compact(*g, pool.view(torch.float8_e4m3fn), scales)
    torch.cuda.synchronize()
    oc.compact(n_bt, lens.numpy(), n_refs)
    np.testing.assert_array_equal(g[0].cpu().numpy(), n_bt)
    np.testing.assert_array_equal(g[2].cpu().numpy(), n_refs)
    # each row entry still leads to the page it had, and so does its scale
    at = g[0][0].long()
    assert torch.equal(pool[at, 0, 0, :4].contiguous().view(torch.int32)[:, 0].cpu(), bt[0])
    assert torch.equal(scales[at, 0].cpu(), bt[0].float())


def test_compact_reports_bad_books(dev):
    w = World([300, 64], 20, dev, seed=13)
    w.bt[0, 0] = 20
    w.refs[w.bt[1, 0].long()] = 0
    ca.cache_compact(w.bt, w.lens, w.refs, w.pool, w.scales, status=w.status)
    torch.cuda.synchronize()
    got = int(w.status)
    assert got & bd.MLA_STATUS_BAD_BLOCK_TABLE and got & ~(bd.MLA_STATUS_BAD_BLOCK_TABLE | ca.MLA_STATUS_BAD_REF_COUNT) == 0


@pytest.mark.parametrize("q8", [True, False])
def test_copy_pages(dev, q8):
    w = World([64 * 10], 30, dev, q8, seed=14)
    src, dst = [0, 5, 5, -1, 29], [10, 11, 12, 13, 14]
    ca.cache_copy_pages(w.t(src), w.t(dst), w.pool, w.scales, status=w.status)
    w.moved([(s, d) for s, d in zip(src, dst) if s >= 0])
    w.check()
    ca.cache_copy_pages(w.t([30, 1, 2]), w.t([20, 30, -1]), w.pool, w.scales, status=w.status)
    w.check(bd.MLA_STATUS_BAD_BLOCK_TABLE)


def test_pages_stream_and_graph(dev):
    w = World([100, 300], 40, dev, rows=6, seed=15)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w.fork([0, 1], [2, 3], stream=s)
    s.synchronize()
    w.check()
    ws = torch.empty(4096, dtype=torch.uint8, device=dev)
    a = [w.t([2]), w.t([4])]
    graph = torch.cuda.CUDAGraph()
    books = [x.clone() for x in (w.bt, w.lens, w.refs)]
    with torch.cuda.graph(graph):
        ca.cache_fork(*a, w.bt, w.lens, w.refs, w.pool, w.scales, status=w.status, workspace=ws)
    for x, y in zip((w.bt, w.lens, w.refs), books):
        assert torch.equal(x, y)
    graph.replay()
    w.moved(oc.fork([2], [4], w.np["bt"], w.np["lens"], w.np["refs"]))
    w.check()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("extra", [0, 3])
def test_compact_keeps_pages_whose_count_was_lost(dev, extra, q8):
    """Held pages with a count of 0 (or below), before and behind the border: reported, and kept with their
    bytes, entries and scales like the others."""
    lens = [300, 64, 1000, 5, 640]
    nb = sum(oc.pages_of(n) for n in lens) + 4 + extra
    w = World(lens, nb, dev, q8, rows=7, seed=31 + extra)
    w.fork([0, 2], [5, 6])
    w.free([1, 4])
    live = int((w.np["refs"] > 0).sum())
    held = sorted({int(w.np["bt"][b, j]) for b in range(7) for j in range(oc.pages_of(int(w.np["lens"][b])))})
    assert len(held) == live
    lost = [held[0], held[2], held[-1]]
    for value in (0, -3):
        if value == 0:
            assert lost[0] < live <= lost[-1]
        w.refs[torch.tensor(lost, device=dev)] = value
        w.np["refs"][lost] = 1
        copies = dict(oc.compact(w.np["bt"], w.np["lens"], w.np["refs"]))
        w.moved(copies.items())
        lost = [copies.get(p, p) for p in lost]
        w.np["refs"][lost] = 0
        w.status.zero_()
        ws = ca.cache_compact_workspace(w.pool.shape[0], dev)
        ca.cache_compact(w.bt, w.lens, w.refs, w.pool, w.scales, workspace=ws, status=w.status)
        w.check(ca.MLA_STATUS_BAD_REF_COUNT)
        assert int(ws.view(torch.int32)[0]) == live


def test_compact_reports_lengths_past_the_table(dev):
    for bad in (-1, 64 * 9):
        w = World([300, 64, 200], 20, dev, seed=17, width=8)
        w.free([1])
        w.bt[0, 5:] = w.np["bt"][0, 5:] = -1
        w.lens[0] = bad
        w.np["lens"][0] = 0 if bad < 0 else 300
        # (the pages of a row without a length are counted, and move; its entries are nobody's)
        w.moved(oc.compact(w.np["bt"], w.np["lens"], w.np["refs"]))
        w.np["lens"][0] = bad
        ca.cache_compact(w.bt, w.lens, w.refs, w.pool, w.scales, status=w.status)
        w.check(bd.MLA_STATUS_BAD_SEQLEN | (bd.MLA_STATUS_BAD_BLOCK_TABLE if bad > 0 else 0))


def test_compact_keeps_lost_pages_of_large_books(dev):
    """More pages than the plan holds in registers: it reads the counts, and the marks, a second time."""
    nb = 66_000
    pool = torch.zeros(nb, 64, 1, 576, dtype=torch.uint8, device=dev)
    pool[:, 0, 0, :4] = torch.arange(nb, dtype=torch.int32, device=dev).view(torch.uint8).view(nb, 4)
    g = torch.Generator().manual_seed(5)
    held = torch.randperm(nb, generator=g)[:3000].int()
    bt, lens = held.view(3, 1000).to(dev), torch.full((3,), 64_000, dtype=torch.int32, device=dev)
    refs = torch.zeros(nb, dtype=torch.int32)
    refs[held.long()] = 1
    lost = held[::7].long()
    n_bt, n_refs = bt.cpu().numpy().copy(), refs.numpy().copy()
    refs[lost] = 0
    copies = dict(oc.compact(n_bt, [64_000] * 3, n_refs))
    n_refs[[copies.get(int(p), int(p)) for p in lost]] = 0
    refs, status = refs.to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    scales = torch.arange(nb, dtype=torch.float32, device=dev)[:, None].contiguous()
    ca.cache_compact(bt, lens, refs, pool.view(torch.float8_e4m3fn), scales, status=status)
    torch.cuda.synchronize()
    assert int(status) == ca.MLA_STATUS_BAD_REF_COUNT
    np.testing.assert_array_equal(bt.cpu().numpy(), n_bt)
    np.testing.assert_array_equal(refs.cpu().numpy(), n_refs)
    at = bt.view(-1).long()
    assert torch.equal(pool[at, 0, 0, :4].contiguous().view(torch.int32)[:, 0].cpu(), held)
    assert torch.equal(scales[at, 0].cpu(), held.float())


@pytest.mark.parametrize("q8", [True, False])
def test_fork_looks_at_the_counts_of_its_parents(dev, q8):
    """A parent's last page that is free by its count is not copied, nor given out to another fork, not even where
    no other page is free; a full page without a count is shared with a word."""
    w = World([100, 200, 300, 70], 17, dev, q8, rows=12, seed=41)
    parents, children = [0, 1, 2, 0, 3], [4, 5, 6, 7, 8]
    lost = [int(w.np["bt"][0, 1]), int(w.np["bt"][2, 4])]
    for value in (0, -2):
        v = World([100, 200, 300, 70], 17, dev, q8, rows=12, seed=41)
        v.refs[torch.tensor(lost, device=dev)] = value
        ca.cache_fork(v.t(parents), v.t(children), v.bt, v.lens, v.refs, v.pool, v.scales, status=v.status)
        v.moved(oc.fork([1, 3], [5, 8], v.np["bt"], v.np["lens"], v.np["refs"]))
        v.np["refs"][lost] = value
        v.check(ca.MLA_STATUS_BAD_REF_COUNT)
    # a pool whose only page with a count of 0 is a parent's own
    v = World([100, 200], 6, dev, q8, rows=4, seed=42)
    page = int(v.np["bt"][0, 1])
    v.refs[page] = 0
    ca.cache_fork(v.t([0, 1]), v.t([2, 3]), v.bt, v.lens, v.refs, v.pool, v.scales, status=v.status)
    v.np["refs"][page] = 0
    v.check(ca.MLA_STATUS_BAD_REF_COUNT | ca.MLA_STATUS_NO_FREE_PAGE)
    # among the full pages
    v = World([128, 64], 8, dev, q8, rows=4, seed=43)
    page = int(v.np["bt"][0, 1])
    v.refs[page] = v.np["refs"][page] = 0
    ca.cache_fork(v.t([0, 1]), v.t([2, 3]), v.bt, v.lens, v.refs, v.pool, v.scales, status=v.status)
    v.moved(oc.fork([0, 1], [2, 3], v.np["bt"], v.np["lens"], v.np["refs"]))
    v.check(ca.MLA_STATUS_BAD_REF_COUNT)


@pytest.mark.parametrize("rows", [1, 5, 1500])
def test_compact_finds_lost_pages_far_into_a_row(dev, rows):
    """Rows of several thousand entries, alone and among more rows than the device has room for."""
    nb, n, width = 4600, 2200, 5000
    g = torch.Generator().manual_seed(rows)
    held = torch.randperm(nb, generator=g)[:2 * n].int().view(2, n)
    bt = torch.full((rows, width), -1, dtype=torch.int32)
    lens = torch.zeros(rows, dtype=torch.int32)
    at = [rows // 2, rows - 1][:min(rows, 2)]
    for i, b in enumerate(at):
        bt[b, :n], lens[b] = held[i], 64 * n - 13
    held = held[:len(at)].flatten()
    refs = torch.zeros(nb, dtype=torch.int32)
    refs[held.long()] = 1
    lost = held[[0, 1023, 1024, 2047, 2048, n - 1, len(held) - 1]].long()
    n_bt, n_refs = bt.numpy().copy(), refs.numpy().copy()
    refs[lost] = 0
    copies = dict(oc.compact(n_bt, lens.tolist(), n_refs))
    n_refs[[copies.get(int(p), int(p)) for p in lost]] = 0
    pool = torch.zeros(nb, 64, 1, 576, dtype=torch.uint8, device=dev)
    pool[:, 0, 0, :4] = torch.arange(nb, dtype=torch.int32, device=dev).view(torch.uint8).view(nb, 4)
    scales, status = torch.arange(nb, dtype=torch.float32, device=dev)[:, None].contiguous(), torch.zeros(1, dtype=torch.int32, device=dev)
    bt, refs = bt.to(dev), refs.to(dev)
    ca.cache_compact(bt, lens.to(dev), refs, pool.view(torch.float8_e4m3fn), scales, status=status)
    torch.cuda.synchronize()
    assert int(status) == ca.MLA_STATUS_BAD_REF_COUNT
    np.testing.assert_array_equal(bt.cpu().numpy(), n_bt)
    np.testing.assert_array_equal(refs.cpu().numpy(), n_refs)
    now = torch.cat([bt[b, :n] for b in at]).long()
    assert torch.equal(pool[now, 0, 0, :4].contiguous().view(torch.int32)[:, 0].cpu(), held)
    assert torch.equal(scales[now, 0].cpu(), held.float())
