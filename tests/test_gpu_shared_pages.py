"""Sequences that share pages: a last page that is not full has one sequence that writes it, whatever the table was and
however the sequences were forked and cut."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu
from .test_gpu_branches import Pools, deal, full, ints

pytestmark = pytest.mark.gpu

WID = 191


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def fork(table, lens, come, pages, page, held=()):
    """(table, lens, left, copies [(from page, to page, rows)]).  A part page that the new table names elsewhere than as
    a part page is nobody's; else it is the first sequence's of those that stay and end in it, or the first one's."""
    batch, width = len(table), len(table[0])
    new, out, ends = [], [], {}
    for b, a in enumerate(come):
        n = int(lens[a]) if a >= 0 else 0
        row = [-1] * width if a < 0 else list(map(int, table[a]))
        if a >= 0 and a != b:
            row[-(-n // page):] = [-1] * (width - -(-n // page))
        if n % page and 0 <= row[n // page] < pages:
            ends.setdefault(row[n // page], []).append(b)
            row[n // page] = -1
        new.append(row)
        out.append(n)
    named = {q for row in new for q in row}
    keeps = {}
    for q, who in ends.items():
        if q not in named:
            keeps[min(who, key=lambda b: (come[b] != b, b))] = q
    copies = [(b, q) for q, who in ends.items() for b in who if b not in keeps]
    for b, q in keeps.items():
        new[b][out[b] // page] = q
    free = br.lowest_free(new, pages, held)
    copies.sort()
    done = []
    for (b, q), to in zip(copies, free):
        new[b][out[b] // page] = to
        done.append((q, to, out[b] % page))
    return new, out, len(free) - len(copies), done


def shared_tables(r, batch, width, pages, page):
    """Tables of sequences that begin with pages of one another, of any length: whole and part pages named often."""
    lens = [int(n) for n in r.integers(0, (width - 1) * page, batch)]
    table = deal(r, lens, page, pages, width)
    for b in range(batch):
        for _ in range(2):
            a = int(r.integers(0, batch))
            if a != b and r.random() < 0.6:
                k = int(r.integers(0, min(-(-lens[a] // page), -(-lens[b] // page)) + 1))
                table[b][:k] = table[a][:k]
    return table, lens


SIZES = [(2, 4, 60), (9, 6, 90), (70, 9, 1000), (1024, 5, 9000)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pages", SIZES)
def test_fork_of_sequences_that_share(batch, width, pages, in_place):
    r = synth.rng(WID, batch, width)
    page, apart = 16, 0
    for i in range(3):
        table, lens = shared_tables(r, batch, width, pages, page)
        for come in (list(range(batch)), [int(a) for a in r.integers(-1, batch, batch)],
                     [b if r.random() < 0.7 else int(r.integers(0, batch)) for b in range(batch)]):
            p = Pools(1, table, lens, pages, page, kvh=1, layers=1 if batch > 100 else 2)
            t, n = p.outs(in_place)
            left = full((1,))
            thinmx.tt_paged_fork(p.layers, p.n, ints(come), None, t, n, left, *p.ws)
            a, b, c, copies = fork(table, lens, come, pages, page)
            assert gu.host(t).tolist() == a and gu.host(n).tolist() == b and gu.host(left).tolist() == [c]
            assert gu.device_error() == (8 if c < 0 else 0)
            for src, dst, rows in copies:
                for x in p.host:
                    x[:, dst, :, :rows] = x[:, src, :, :rows]
            p.check({q for row in a for q in row if q >= 0})
            apart += come == list(range(batch)) and len(copies)
            # each part page is named once
            names = [q for row in a for q in row if q >= 0]
            assert all(names.count(a[s][b[s] // page]) == 1 for s in range(min(batch, 70))
                       if b[s] % page and a[s][b[s] // page] >= 0)
    assert apart > 0  # sequences that stay were given pages of their own


def test_a_pool_whose_bits_lie_in_the_workspace():
    """More pages than shared memory has bits for: two sequences that end in one page."""
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    pages, page = 1_400_000, 16
    k, v = (torch.zeros((pages, 1, page, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, other = (torch.zeros((pages, 1, page), device="cuda") for _ in range(2))
    last = pages - 1
    k[last], v[last], scales[last] = 7, 9, 3.0
    table, lens = ints([[5, last], [5, last], [6, -1]]), ints([30, 20, 4])
    layers = loader.paged_layers([loader.paged_kv(k, v, table, lens, scales, other)])
    nb = thinmx.tt_paged_pages_workspace_bytes(layers[0])
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    thinmx.tt_paged_fork(layers, 1, ints([0, 1, 2]), None, table, lens, full((1,)), ws, nb)
    assert gu.host(table).tolist() == [[5, last], [5, 0], [6, -1]]
    assert (k[0, 0, :4] == 7).all() and (v[0, 0, :4] == 9).all() and (scales[0, 0, :4] == 3.0).all()
    assert not k[0, 0, 4:].any() and gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_branch_that_is_cut_leaves_the_other_as_it_was(fp8):
    """Two branches of 32 tokens in shared pages, one of them cut to 20 and grown again: a fork gives it a page of its
    own, and the other keeps its rows."""
    import torch
    page, d, kvh = 16, 64, 2
    p = Pools(3, [[4, 1, -1], [-1] * 3], [32, 0], 9, page, kvh=kvh, d=d, fp8=fp8)
    left = full((1,))
    thinmx.tt_paged_fork(p.layers, p.n, ints([0, 0]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.table).tolist() == [[4, 1, -1]] * 2
    r = synth.rng(WID, 7, fp8)
    new = gu.dev(synth.f32_to_bf16_bits(r.standard_normal((2, 2, kvh, d)).astype(np.float32)))

    def grow(step):  # one token of the second branch, in every layer
        want = p.lens.clone()
        want[1] += 1
        thinmx.tt_paged_resize(p.kvs[0], ints([-1, int(want[1])]), None, p.table, p.lens, left, *p.ws)
        p.lens.copy_(want)
        for kv in p.kvs:
            thinmx.tt_paged_rope_append(kv, None, new[step, 0], new[step, 1], 0, kvh * d, 1, ints([0, 0, 1]), 0, None, 64,
                                        False, None, 1, None, None)
        torch.cuda.synchronize()

    p.lens[1] = 20
    thinmx.tt_paged_fork(p.layers, p.n, ints([0, 1]), None, p.table, p.lens, left, *p.ws)
    thinmx.tt_paged_resize(p.kvs[0], ints([-1, 20]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.lens).tolist() == [32, 20] and gu.device_error() == 0
    assert gu.host(p.table).tolist() == [[4, 1, -1], [4, 0, -1]]
    for x in p.host:
        x[:, 0, :, :4] = x[:, 1, :, :4]
    grow(0)
    for got, want in zip(p.dev, p.host):
        g = gu.host(got)
        assert np.array_equal(g[:, [1, 4]], want[:, [1, 4]])              # the first branch
        assert np.array_equal(g[:, 0, :, :4], want[:, 0, :, :4])          # the second one's copied rows
        assert not np.array_equal(g[:, 0, :, 4], want[:, 0, :, 4])        # its new one
    # alone in its page, it is cut without a report
    thinmx.tt_paged_resize(p.kvs[0], ints([-1, 18]), None, p.table, p.lens, left, *p.ws)
    assert gu.host(p.lens).tolist() == [32, 18] and gu.device_error() == 0
