"""Cuts into pages that other sequences name, and the error word of each page call."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu
from .test_gpu_branches import Pools, deal, full, ints
from .test_gpu_shared_pages import SIZES, fork, shared_tables

pytestmark = pytest.mark.gpu

WID = 191


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def resize(table, lens, want, pages, page, held=()):
    """(table, lens, left, cuts that end inside a page which another entry names): branch_ref's, with the number of
    those cuts, which are reported."""
    new, out, left = br.resize(table, lens, want, pages, page, held)
    names = [q for b, row in enumerate(table) for e, q in enumerate(row) if want[b] < 0 or e < -(-want[b] // page)]
    shared = 0
    for b, (n, w) in enumerate(zip(lens, want)):
        if 0 <= w < n and w % page:
            q = table[b][w // page]
            shared += 0 <= q < pages and names.count(q) > 1
    return new, out, left, shared


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pages", SIZES)
def test_cuts_into_shared_pages(batch, width, pages, in_place):
    r = synth.rng(WID, batch, width + 1)
    page, met, alone = 16, 0, 0
    for i in range(4):
        table, lens = shared_tables(r, batch, width, pages, page)
        want = [-1 if r.random() < 0.2 else int(r.integers(0, n + page)) for n in lens]
        p = Pools(2, table, lens, pages, page, kvh=1, layers=1)
        t, n = p.outs(in_place)
        left = full((1,))
        thinmx.tt_paged_resize(p.kvs[0], ints(want), None, t, n, left, *p.ws)
        a, b, c, shared = resize(table, lens, want, pages, page)
        assert gu.host(t).tolist() == a and gu.host(n).tolist() == b and gu.host(left).tolist() == [c]
        assert gu.device_error() == (8 if shared or c < 0 else 0)
        met += shared
        # the others alone, which are cut into pages of their own
        cut = [-1 if 0 <= w < x and w % page else w for w, x in zip(want, lens)]
        p = Pools(2, table, lens, pages, page, kvh=1, layers=1)
        thinmx.tt_paged_resize(p.kvs[0], ints(cut), None, t, n, left, *p.ws)
        a, b, c, shared = resize(table, lens, cut, pages, page)
        assert gu.host(t).tolist() == a and gu.host(n).tolist() == b
        assert shared == 0 and gu.device_error() == (8 if c < 0 else 0)
        alone += c >= 0
    assert met > 0 and alone > 0


def test_a_pool_whose_bits_lie_in_the_workspace():
    """More pages than shared memory has bits for."""
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    pages, page = 1_400_000, 16
    k, v = (torch.zeros((pages, 1, page, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = torch.zeros((pages, 1, page), device="cuda")
    last = pages - 1
    table, lens = ints([[5, last], [5, last], [6, -1]]), ints([30, 30, 9])
    kv = loader.paged_kv(k, v, table, lens, scales, scales)
    nb = thinmx.tt_paged_pages_workspace_bytes(kv)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    for want, code in (([-1, -1, 4], 0), ([-1, 20, 4], 8), ([0, 18, -1], 0)):
        thinmx.tt_paged_resize(kv, ints(want), None, table, lens, None, ws, nb)
        assert gu.device_error() == code
    assert gu.host(lens).tolist() == [0, 18, 4]
    assert gu.host(table).tolist() == [[-1, -1], [5, last], [6, -1]]


@pytest.mark.parametrize("fp8", [False, True])
def test_a_cut_that_is_reported_and_separated(fp8):
    """Two branches of 32 tokens in shared pages, one of them cut to 20: reported, since both name the page; after a
    fork that gives it one of its own it is cut again, without a report."""
    page, d, kvh = 16, 64, 2
    p = Pools(3, [[4, 1, -1], [4, 1, -1]], [32, 32], 9, page, kvh=kvh, d=d, fp8=fp8)
    left = full((1,))
    thinmx.tt_paged_resize(p.kvs[0], ints([-1, 20]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.lens).tolist() == [32, 20] and gu.device_error() == 8
    thinmx.tt_paged_fork(p.layers, p.n, ints([0, 1]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.table).tolist() == [[4, 1, -1], [4, 0, -1]]
    for x in p.host:
        x[:, 0, :, :4] = x[:, 1, :, :4]
    p.check()
    thinmx.tt_paged_resize(p.kvs[0], ints([-1, 18]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.lens).tolist() == [32, 18] and gu.device_error() == 0


def test_one_of_two_goes_on():
    """A cut into a page whose other name the same call lets go is not reported."""
    p = Pools(4, [[4, 1], [4, 1], [2, 3]], [32, 32, 32], 9, 16, layers=1)
    t, n = p.outs(False)
    thinmx.tt_paged_resize(p.kvs[0], ints([20, 16, 0]), None, t, n, None, *p.ws)
    assert gu.host(t).tolist() == [[4, 1], [4, -1], [-1, -1]] and gu.host(n).tolist() == [20, 16, 0]
    assert gu.device_error() == 0
    # both cut: both would write the page
    thinmx.tt_paged_resize(p.kvs[0], ints([20, 25, -1]), None, t, n, None, *p.ws)
    assert gu.host(t).tolist() == [[4, 1], [4, 1], [2, 3]] and gu.host(n).tolist() == [20, 25, 32]
    assert gu.device_error() == 8
