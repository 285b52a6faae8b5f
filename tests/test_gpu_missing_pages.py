"""The error word of each page call on the largest batch, by its own free pages."""
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import gpu_util as gu
from .test_gpu_branches import Pools, deal, full, ints
from .test_gpu_page_cuts import resize
from .test_gpu_shared_pages import fork

pytestmark = pytest.mark.gpu

WID = 191


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


@pytest.mark.parametrize("few", [False, True])
def test_missing_pages_are_reported_by_the_call_that_lacks_them(few):
    """1024 sequences: after the fork, which finds its pages, and after the resize, which may not."""
    r = synth.rng(WID, 2, few)
    batch, page, width = 1024, 16, 5
    lens = [int(n) for n in r.integers(0, 50, batch)]
    pages = sum(-(-n // page) for n in lens) + (100 if few else 4000)
    table = deal(r, lens, page, pages, width)
    p = Pools(5, table, lens, pages, page, kvh=1, layers=1)
    come = [b if r.random() < 0.5 else int(r.integers(0, batch)) for b in range(batch)]
    left = full((1,))
    thinmx.tt_paged_fork(p.layers, 1, ints(come), None, p.table, p.lens, left, *p.ws)
    a, b, free, _ = fork(table, lens, come, pages, page)
    assert gu.host(p.table).tolist() == a and gu.host(p.lens).tolist() == b and gu.host(left).tolist() == [free]
    assert free >= 0 and gu.device_error() == 0
    want = [-1 if r.random() < 0.1 else page * width for _ in range(batch)]
    thinmx.tt_paged_resize(p.kvs[0], ints(want), None, p.table, p.lens, left, *p.ws)
    a, b, free, shared = resize(a, b, want, pages, page)
    assert gu.host(p.table).tolist() == a and gu.host(p.lens).tolist() == b and gu.host(left).tolist() == [free]
    assert shared == 0 and (free < 0) == few and gu.device_error() == (8 if few else 0)
