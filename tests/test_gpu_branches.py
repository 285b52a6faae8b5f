"""Accepting drafts, keeping their rows, and the pages of branching sequences, against plain Python."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import loader, synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu

pytestmark = pytest.mark.gpu

WID = 162


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def ints(x):
    return gu.dev(np.array(x, np.int32))


def full(shape, v=77):
    import torch
    return torch.full(shape, v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------------------ accept
def run_accept(parents, drafts, chosen, starts, width):
    batch = len(starts) - 1
    path, counts, nxt = full((batch, width)), full((batch,)), full((batch,))
    thinmx.tt_draft_accept(ints(parents), ints(drafts), ints(chosen), ints(starts), batch, len(parents), width, path,
                           counts, nxt)
    return gu.host(path).tolist(), gu.host(counts).tolist(), gu.host(nxt).tolist()


@pytest.mark.parametrize("width", [1, 3, 70])
@pytest.mark.parametrize("vocab", [2, 5, 1000])
def test_accept(width, vocab):
    """A small vocabulary makes many children match: the lowest is taken."""
    r = synth.rng(WID, width, vocab)
    new = [1, 0, 40, 7, 64, 150, 300, 33]
    parents = [p for i, n in enumerate(new) for p in br.parents_of(r, n, chain=i == 5)]
    starts = np.cumsum([0] + new).tolist()
    drafts, chosen = (r.integers(0, vocab, len(parents)).tolist() for _ in range(2))
    for i in range(starts[5], starts[6] - 1):  # the chain is accepted whole
        chosen[i] = drafts[i + 1]
    got = run_accept(parents, drafts, chosen, starts, width)
    assert got == br.accept(parents, drafts, chosen, starts, width)


def test_accept_of_nothing_and_of_parents_that_are_no_tree():
    path, counts, nxt = full((2, 3)), full((2,)), full((2,))
    thinmx.tt_draft_accept(None, None, None, ints([0, 0, 0]), 2, 0, 3, path, counts, nxt)
    assert gu.host(path).tolist() == [[-1] * 3] * 2 and gu.host(counts).tolist() == [0, 0]
    assert gu.host(nxt).tolist() == [-1, -1]
    # parents that point at themselves or ahead are no children of those
    got = run_accept([0, 5, 2, 0, 3], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1], [0, 5], 5)
    assert got == ([[0, 3, 4, -1, -1]], [3], [1])


# ------------------------------------------------------------------------------------------------------------- pools
class Pools:
    """Layers of one table on the device, and their contents on the host."""

    def __init__(self, seed, table, lens, pages, page, kvh=2, d=64, fp8=False, layers=2):
        import torch
        r = synth.rng(WID, seed, 1)
        self.page, self.pages, self.fp8 = page, pages, fp8
        shape = (layers, pages, kvh, page, d)
        kind = np.uint8 if fp8 else np.int16
        info = np.iinfo(kind)
        self.host = [r.integers(info.min, info.max, shape, dtype=kind, endpoint=True) for _ in range(2)]
        if fp8:
            self.host += [r.standard_normal(shape[:4]).astype(np.float32) for _ in range(2)]
        self.dev = [gu.dev(x) for x in self.host]
        self.table, self.lens = ints(table), ints(lens)
        self.kvs = [loader.paged_kv(self.dev[0][i], self.dev[1][i], self.table, self.lens,
                                    *((self.dev[2][i], self.dev[3][i]) if fp8 else ())) for i in range(layers)]
        self.layers, self.n = loader.paged_layers(self.kvs), layers
        nb = thinmx.tt_paged_pages_workspace_bytes(self.kvs[0])
        self.ws = (torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda"), nb)

    def outs(self, in_place):
        return (self.table, self.lens) if in_place else (full(tuple(self.table.shape)), full(tuple(self.lens.shape)))

    def check(self, pages=None):
        """Contents as on the host, in the pages asked for."""
        for got, want in zip(self.dev, self.host):
            g = gu.host(got)
            at = slice(None) if pages is None else sorted(pages)
            assert np.array_equal(g[:, at], want[:, at])


def deal(r, lens, page, pages, width, spare=0):
    """A table of distinct pages, in any order; `spare` pages reserved past each sequence's length."""
    order = iter(r.permutation(pages).tolist())
    table = []
    for n in lens:
        need = -(-n // page) + (spare if n else 0)
        table.append([next(order) for _ in range(need)] + [-1] * (width - need))
    return table


# -------------------------------------------------------------------------------------------------------------- keep
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp8,d,page", [(False, 64, 16), (True, 64, 32), (False, 128, 16), (True, 128, 128)])
def test_keep(fp8, d, page, in_place):
    r = synth.rng(WID, page, d)
    new, past = [1, 0, 9, 40, 3, 64, 20], [30, 0, 15, 100, 0, 7, 60]
    lens = [n + p for n, p in zip(new, past)]
    table = deal(r, lens, page, 60, 10)
    table[6][60 // page] = -1  # moves from and to the hole are dropped
    p = Pools(1, table, lens, 60, page, d=d, fp8=fp8, layers=3)
    starts = np.cumsum([0] + new).tolist()
    width = 12
    paths = [sorted(r.choice(n, min(n, int(r.integers(1, width + 1))), replace=False).tolist()) for n in new]
    paths[2] = [0, 1, 2, 3]  # nothing to move
    paths[5] = list(range(1, 13))  # every row moves onto the one before
    counts = [len(w) for w in paths]
    out = p.outs(in_place)[1]
    thinmx.tt_paged_keep(p.layers, p.n, ints(starts), ints([w + [-1] * (width - len(w)) for w in paths]), width,
                         ints(counts), out)
    old = [x.copy() for x in p.host]
    for b, way in enumerate(paths):
        for j, i in enumerate(way):
            (p0, r0), (p1, r1) = ((table[b][(past[b] + t) // page], (past[b] + t) % page) for t in (i, j))
            if p0 >= 0 and p1 >= 0:
                for x, y in zip(p.host, old):
                    x[:, p1, :, r1] = y[:, p0, :, r0]
    p.check()
    assert gu.host(out).tolist() == [a + c for a, c in zip(past, counts)]
    assert gu.device_error() == 0


def test_keep_many_rows():
    """More rows than are looked up at a time."""
    r = synth.rng(WID, 3, 3)
    n, past, page = 700, 20, 16
    table = deal(r, [n + past], page, 50, 46)
    p = Pools(2, table, [n + past], 50, page)
    way = sorted(r.choice(n, 600, replace=False).tolist())
    out = p.outs(False)[1]
    thinmx.tt_paged_keep(p.layers, p.n, ints([0, n]), ints([way]), 600, ints([600]), out)
    old = [x.copy() for x in p.host]
    for j, i in enumerate(way):
        (p0, r0), (p1, r1) = ((table[0][(past + t) // page], (past + t) % page) for t in (i, j))
        for x, y in zip(p.host, old):
            x[:, p1, :, r1] = y[:, p0, :, r0]
    p.check()
    assert gu.host(out).tolist() == [620]


def test_keep_reports_what_is_no_path():
    page, lens = 16, [20, 20, 20, 20, 3]
    table = deal(synth.rng(WID, 4, 4), lens, page, 12, 2)
    p = Pools(3, table, lens, 12, page)
    paths = [[0, 2, 2, 3], [0, 1, 9, 3], [1, 0, 2, 3], [0, 2, 3, 4], [0, 1, 4, -1]]
    out = p.outs(False)[1]
    thinmx.tt_paged_keep(p.layers, p.n, ints([0, 8, 16, 24, 32, 37]), ints(paths), 4, ints([4, 4, -1, 9, 3]), out)
    assert gu.device_error() == 2
    # the good beginnings of the paths are kept; the last sequence has two tokens without a place
    assert gu.host(out).tolist() == [12 + 2, 12 + 2, 12, 12 + 4, 1]
    for b, way in ((0, [0, 2]), (3, [0, 2, 3, 4]), (4, [0, 1, 4])):
        past = [12, 12, 12, 12, -2][b]
        old = [x.copy() for x in p.host]
        for j, i in enumerate(way):
            if past + j >= 0:
                (p0, r0), (p1, r1) = ((table[b][(past + t) // page], (past + t) % page) for t in (i, j))
                for x, y in zip(p.host, old):
                    x[:, p1, :, r1] = y[:, p0, :, r0]
    p.check()


# ------------------------------------------------------------------------------------------------------------- pages
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pages", [(1, 3, 9), (5, 9, 40), (40, 70, 3000), (3, 300, 1000)])
def test_resize(batch, width, pages, in_place):
    r = synth.rng(WID, batch, width)
    page = 16
    lens = r.integers(0, max(1, min(width * page, pages * page // (2 * batch))), batch).tolist()
    table = deal(r, lens, page, pages, width)
    if batch > 2:
        table[1][0] = -1          # a hole below the length stays one
        lens[1] = max(lens[1], 17)
        table[2][width - 1] = table[0][0]  # a page named twice, past the length
    want = [int(w) for w in r.integers(-1, width * page + 1, batch)]
    held = np.zeros(pages, np.uint8)
    held[r.choice(pages, pages // 8, replace=False)] = 1
    for use_held in (False, True):
        p = Pools(4, table, lens, pages, page, layers=1)
        t, n = p.outs(in_place)
        left = full((1,))
        thinmx.tt_paged_resize(p.kvs[0], ints(want), gu.dev(held) if use_held else None, t, n, left, *p.ws)
        a, b, c = br.resize(table, lens, want, pages, page, np.flatnonzero(held).tolist() if use_held else ())
        assert gu.host(t).tolist() == a and gu.host(n).tolist() == b and gu.host(left).tolist() == [c]
        assert gu.device_error() == (8 if c < 0 else 0)


def test_resize_past_the_table_and_to_nothing():
    p = Pools(5, [[0, 1, -1], [2, 3, 4]], [20, 40], 9, 16, layers=1)
    t, n = p.outs(False)
    thinmx.tt_paged_resize(p.kvs[0], ints([1000, 0]), None, t, n, None, *p.ws)
    assert gu.device_error() == 2
    assert gu.host(t).tolist() == [[0, 1, 2], [-1, -1, -1]] and gu.host(n).tolist() == [20, 0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp8,page,d", [(False, 16, 64), (True, 64, 64), (True, 128, 128), (False, 32, 128)])
@pytest.mark.parametrize("batch", [2, 9, 70])
def test_fork(batch, fp8, page, d, in_place):
    r = synth.rng(WID, batch, page)
    width, most = 6, 4 * page
    lens = [int(n) for n in r.integers(0, most, batch)]
    lens[0] = 2 * page  # no part page
    pages = sum(-(-n // page) + 1 for n in lens) + batch + 4
    table = deal(r, lens, page, pages, width, spare=1)
    held = np.zeros(pages, np.uint8)
    held[r.choice(pages, 3, replace=False)] = 1
    for come in ([int(a) for a in r.integers(-1, batch, batch)],          # anything
                 [b - b % 2 for b in range(batch)], [-1] * batch, list(range(batch)),
                 [(b + 1) % batch for b in range(batch)],                 # all change places: nothing is copied
                 [batch - 1] * batch):
        p = Pools(6, table, lens, pages, page, d=d, fp8=fp8)
        t, n = p.outs(in_place)
        left = full((1,))
        thinmx.tt_paged_fork(p.layers, p.n, ints(come), gu.dev(held), t, n, left, *p.ws)
        a, b, c, copies = br.fork(table, lens, come, pages, page, np.flatnonzero(held).tolist())
        assert gu.host(t).tolist() == a and gu.host(n).tolist() == b and gu.host(left).tolist() == [c]
        assert gu.device_error() == (8 if c < 0 else 0)
        for src, dst, rows in copies:
            for x in p.host:
                x[:, dst, :, :rows] = x[:, src, :, :rows]
        p.check()


def test_fork_without_pages_and_from_nowhere():
    table = [[0, 1], [2, -1], [3, 4]]
    p = Pools(7, table, [20, 3, 30], 5, 16)
    t, n = p.outs(False)
    left = full((1,))
    thinmx.tt_paged_fork(p.layers, p.n, ints([0, 0, 3]), None, t, n, left, *p.ws)  # page 2 is let go, and taken
    assert gu.device_error() == 2  # (3 is no sequence: it stays)
    assert gu.host(t).tolist() == [[0, 1], [0, 2], [3, 4]] and gu.host(left).tolist() == [0]
    thinmx.tt_paged_fork(p.layers, p.n, ints([2, 2, 2]), gu.dev(np.array([1, 1, 0, 0, 0], np.uint8)), t, n, left, *p.ws)
    assert gu.device_error() == 8  # one of two pages
    assert gu.host(t).tolist() == [[3, 2], [3, -1], [3, 4]] and gu.host(left).tolist() == [-1]
    assert gu.host(n).tolist() == [30, 30, 30]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp8,page,d,pages", [(False, 16, 64, 33), (True, 64, 128, 100), (True, 16, 64, 2500),
                                              (False, 128, 128, 40)])
def test_compact(fp8, page, d, pages, in_place):
    r = synth.rng(WID, page, pages)
    batch = 7
    for fill in (0.0, 0.1, 0.5, 1.0):
        lens = [int(fill * pages * page / batch)] * batch
        width = max(1, -(-lens[0] // page)) + 1
        table = deal(r, [max(0, n - page + 1) for n in lens], page, pages, width)
        table[3][-1] = table[0][0]  # a shared page
        held = np.zeros(pages, np.uint8)
        held[r.choice(pages, pages // 5, replace=False)] = 1
        for use_held in (False, True):
            p = Pools(8, table, lens, pages, page, d=d, fp8=fp8)
            t, _ = p.outs(in_place)
            span = full((1,))
            thinmx.tt_paged_compact(p.layers, p.n, gu.dev(held) if use_held else None, t, span, *p.ws)
            a, top, copies = br.compact(table, pages, np.flatnonzero(held).tolist() if use_held else ())
            assert gu.host(t).tolist() == a and gu.host(span).tolist() == [top]
            for src, dst in copies:
                for x in p.host:
                    x[:, dst] = x[:, src]
            p.check({q for row in a for q in row if q >= 0})
            assert gu.device_error() == 0


def test_pools_of_more_pages_than_shared_memory_has_bits_for():
    import torch
    pages, page = 1_400_000, 16
    kv = torch.zeros((pages, 1, page, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((pages, 1, page), device="cuda")
    far = [1_399_999, 7, 1_310_720, 64]
    for i, q in enumerate(far):
        kv[q] = i + 1
        scales[q] = i + 1.0
    t = ints([far])
    h = loader.paged_kv(kv, kv, t, ints([60]), scales, scales)
    nb = thinmx.tt_paged_pages_workspace_bytes(h)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    span = full((1,))
    thinmx.tt_paged_compact(h, 1, None, t, span, ws, nb)
    assert gu.host(t).tolist() == [[3, 0, 2, 1]]  # in the order of their numbers
    assert gu.host(span).tolist() == [4]
    assert [int(kv[q].max()) for q in gu.host(t)[0]] == [1, 2, 3, 4]
    assert [float(scales[q].min()) for q in gu.host(t)[0]] == [1.0, 2.0, 3.0, 4.0]
    assert gu.device_error() == 0


def test_a_page_number_past_the_pool():
    table = [[0, 9], [8, -1]]
    for call in ("resize", "fork", "compact"):
        p = Pools(9, table, [20, 10], 9, 16, layers=1)
        t, n = p.outs(False)
        if call == "resize":
            thinmx.tt_paged_resize(p.kvs[0], ints([-1, 20]), None, t, n, None, *p.ws)
            assert gu.host(t).tolist() == [[0, 9], [8, 1]]
        elif call == "fork":
            thinmx.tt_paged_fork(p.layers, 1, ints([0, 0]), None, t, n, None, *p.ws)
            assert gu.host(t).tolist() == [[0, 9], [0, 9]]  # no page to copy
        else:
            thinmx.tt_paged_compact(p.layers, 1, None, t, None, *p.ws)
            assert gu.host(t).tolist() == [[0, 9], [1, -1]]
        assert gu.device_error() == 2


def test_graph_of_a_beam_step():
    """Fork and resize in place, captured once and replayed with other choices: as the same calls on the host."""
    import torch
    r = synth.rng(WID, 30, 0)
    batch, page, pages, width = 6, 16, 80, 10
    lens = [33, 0, 16, 50, 47, 1]
    table = deal(r, lens, page, pages, width)
    p = Pools(10, table, lens, pages, page)
    come, want, left = full((batch,), -1), full((batch,), -1), full((1,))
    come.copy_(torch.arange(batch, dtype=torch.int32))

    def step():
        thinmx.tt_paged_fork(p.layers, p.n, come, None, p.table, p.lens, left, *p.ws)
        torch.add(p.lens, 1, out=want)
        thinmx.tt_paged_resize(p.kvs[0], want, None, p.table, p.lens, left, *p.ws)
        torch.add(p.lens, (p.lens > 0).int(), out=p.lens)

    step()
    torch.cuda.synchronize()
    p.table.copy_(ints(table))
    p.lens.copy_(ints(lens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(12):
        choice = [int(a) for a in r.integers(0, batch, batch)]
        come.copy_(ints(choice))
        graph.replay()
        table, lens, _, copies = br.fork(table, lens, choice, pages, page)
        for src, dst, rows in copies:
            for x in p.host:
                x[:, dst, :, :rows] = x[:, src, :, :rows]
        table, lens, n = br.resize(table, lens, [a + 1 for a in lens], pages, page)
        lens = [a + (a > 0) for a in lens]
        assert gu.host(p.table).tolist() == table and gu.host(p.lens).tolist() == lens
        assert gu.host(left).tolist() == [n] and n >= 0
        p.check({q for row in table for q in row if q >= 0})
    assert gu.device_error() == 0
