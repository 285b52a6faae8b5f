"""Drafted trees, pages and log probabilities at the ends of their ranges: pools and logits past 2^32 bytes, the largest
batches, two captured graphs on one workspace, a whole drafted step in a graph."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import loader, synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu
from . import paged_ref as ref
from .test_gpu_branches import full, ints
from .test_gpu_paged import _handle
from .test_gpu_tree import EPS, attend, check, queries, setup

pytestmark = pytest.mark.gpu

WID = 181


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def far_pool(cache, pages, rows):
    """The cache's pages at places of a pool of `pages` pages: (k, v, scales or None, table)."""
    import torch
    places = synth.rng(WID, rows, 0).permutation(cache.pages) * (pages // cache.pages) + pages - 1 - (
        cache.pages - 1) * (pages // cache.pages)
    kind = torch.uint8 if cache.fp8 else torch.int16
    at = torch.from_numpy(places.astype(np.int64)).cuda()
    pools = []
    for x in (cache.k, cache.v):
        p = torch.zeros((pages,) + x.shape[1:], dtype=kind, device="cuda")
        p[at] = gu.dev(x)
        pools.append(p)
    scales = []
    for x in (cache.k_scales, cache.v_scales) if cache.fp8 else ():
        p = torch.zeros((pages,) + x.shape[1:], device="cuda")
        p[at] = gu.dev(x)
        scales.append(p)
    table = np.where(cache.table >= 0, places[np.maximum(cache.table, 0)], -1).astype(np.int32)
    assert places.max() == pages - 1 and places.min() >= 0
    return pools, scales, gu.dev(table), table


@pytest.mark.parametrize("fp8", [False, True])
def test_pools_past_4_gb(fp8):
    """Pages whose rows lie past 2^32 bytes are attended, copied by a fork, kept, and moved together."""
    import torch
    page, kvh, d, new, past = 128, 4, 128, [20, 9], [300, 150]
    cache, starts, masks, words, q = setup(40, (16, kvh, d), page, fp8, new, past)
    pages = 70001 if fp8 else 35003
    pools, scales, t, table = far_pool(cache, pages, 1)
    assert pools[0].numel() * pools[0].element_size() > 2 ** 32
    lens = gu.dev(cache.lens)
    kv = loader.paged_kv(pools[0], pools[1], t, lens, *scales)
    want = br.tree_attention(cache, q, starts, masks, words, 0.1)
    ref.check_attention(*attend(kv, q, starts, masks, words, 0.1), want, EPS, "far pages")
    layers = loader.paged_layers([kv])
    nb = thinmx.tt_paged_pages_workspace_bytes(kv)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")

    def rows(b, upto):
        tab, i = gu.host(t)[b], np.arange(upto)
        at = torch.from_numpy(tab[i // page].astype(np.int64)).cuda(), torch.from_numpy(i % page).cuda()
        return [x[at[0], :, at[1]].cpu().numpy() for x in pools + scales]

    # kept: nodes 0, 3 and 7 of the first tree, 0 of the second
    before = rows(0, past[0] + new[0])
    path, counts = ints([[0, 3, 7], [0, -1, -1]]), ints([3, 1])
    thinmx.tt_paged_keep(layers, 1, ints(starts.tolist()), path, 3, counts, lens)
    assert gu.host(lens).tolist() == [past[0] + 3, past[1] + 1]
    for got, old in zip(rows(0, past[0] + 3), before):
        assert np.array_equal(got[:past[0]], old[:past[0]])
        assert np.array_equal(got[past[0]:], old[[past[0], past[0] + 3, past[0] + 7]])
    # moved together: all pages lie at the front, with the same rows
    kept = [rows(b, n) for b, n in ((0, past[0] + 3), (1, past[1] + 1))]
    span, left = full((1,)), full((1,))
    thinmx.tt_paged_compact(layers, 1, None, t, span, ws, nb)
    used = int((table >= 0).sum())
    assert gu.host(span).tolist() == [used] and gu.host(t).max() == used - 1
    for b, want in enumerate(kept):
        assert all(np.array_equal(x, y) for x, y in zip(rows(b, len(want[0])), want))
    # forked with all but the last pages held: the part page's copy goes to the pool's end
    held = torch.ones(pages, dtype=torch.uint8, device="cuda")
    held[-1] = 0
    thinmx.tt_paged_fork(layers, 1, ints([0, 0]), held, t, lens, left, ws, nb)
    assert gu.host(t)[1, (past[0] + 3) // page] == pages - 1 and gu.host(left).tolist() == [0]
    assert all(np.array_equal(x, y) for x, y in zip(rows(1, past[0] + 3), kept[0]))
    assert gu.device_error() == 0


def test_tree_attention_of_the_largest_batch():
    """1024 sequences, most of them without new tokens or short."""
    r = synth.rng(WID, 1, 0)
    new = [int(n) for n in np.where(r.random(1024) < 0.6, 0, r.integers(1, 5, 1024))]
    past = [int(n) for n in r.integers(0, 40, 1024)]
    new[1023], past[1023], new[0], past[0] = 40, 300, 0, 0
    check(41, (8, 8, 64), 16, False, new, past, "1024 sequences")


def test_pages_of_the_largest_batch():
    """Fork and resize of 1024 sequences, some of which end, and whose pages others take."""
    import torch
    r = synth.rng(WID, 2, 0)
    batch, page, pages, width = 1024, 16, 4000, 5
    order = iter(r.permutation(pages).tolist())
    lens = [int(n) for n in r.integers(0, 50, batch)]
    table = [[next(order) for _ in range(-(-n // page))] for n in lens]
    table = [t + [-1] * (width - len(t)) for t in table]
    k, v = (torch.zeros((pages, 1, page, 64), dtype=torch.int16, device="cuda") for _ in range(2))
    k += torch.arange(pages, dtype=torch.int16, device="cuda").view(-1, 1, 1, 1)
    t, n, left = ints(table), ints(lens), full((1,))
    kv = loader.paged_kv(k, v, t, n)
    nb = thinmx.tt_paged_pages_workspace_bytes(kv)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    come = [int(a) for a in np.where(r.random(batch) < 0.5, np.arange(batch), r.integers(-1, batch, batch))]
    thinmx.tt_paged_fork(loader.paged_layers([kv]), 1, ints(come), None, t, n, left, ws, nb)
    want, lens, free, copies = br.fork(table, lens, come, pages, page)
    assert gu.host(t).tolist() == want and gu.host(n).tolist() == lens and gu.host(left).tolist() == [free]
    got, was = gu.host(k)[:, 0, :, 0], np.repeat(np.arange(pages)[:, None], page, 1).astype(np.int16)
    for src, dst, rows in copies:
        was[dst, :rows] = was[src, :rows]
    in_use = sorted({q for row in want for q in row if q >= 0})
    assert np.array_equal(got[in_use], was[in_use])
    more = [int(a) for a in r.integers(-1, page * width + 1, batch)]
    thinmx.tt_paged_resize(kv, ints(more), None, t, n, left, ws, nb)
    want, lens, free = br.resize(want, lens, more, pages, page)
    assert gu.host(t).tolist() == want and gu.host(n).tolist() == lens and gu.host(left).tolist() == [free]
    assert gu.device_error() in (0, 8)


@pytest.mark.parametrize("bf16", [True, False])
def test_logits_past_4_gb(bf16):
    """Rows whose offsets pass 2^32 bytes, and 2^32 elements in bf16; many rows of few logits."""
    import torch
    stride, rows, vocab = (2_000_000_011 if bf16 else 700_000_003), 4, 5003
    kind = torch.int16 if bf16 else torch.float32
    big = torch.empty(stride * (rows - 1) + vocab, dtype=kind, device="cuda")
    x = (synth.rng(WID, 3, 0).standard_normal((rows, vocab)) * 3).astype(np.float32)
    bits = synth.f32_to_bf16_bits(x) if bf16 else x
    for r in range(rows):
        big[r * stride:r * stride + vocab] = gu.dev(bits[r])
    small = gu.dev(bits)
    got = []
    for logits, apart in ((big, stride), (small, vocab)):
        logp, ent, tops = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros((rows, 7), device="cuda")
        ids = full((rows, 7))
        nb = thinmx.tt_token_logprobs_workspace_bytes(rows, vocab, 7)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        thinmx.tt_token_logprobs(logits, thinmx.TT_LOGITS_BF16 if bf16 else thinmx.TT_LOGITS_F32, rows, vocab, apart, 1.0,
                                 ints([1, 2, 3, 5002]), 7, logp, ent, ids, tops, ws, nb)
        got.append([gu.host(a) for a in (logp, ent, ids, tops)])
    assert np.array_equal(got[0][2], got[1][2])
    # sums in another order, where a row begins elsewhere from a 16-byte boundary: a chain of at most 104 additions and
    # the logarithm's argument, half a step each, twice
    for a, b in zip(got[0][:2] + got[0][3:], got[1][:2] + got[1][3:]):
        assert np.abs(a - b).max() <= 2 * (104 + 8) * 2.0 ** -24 * (1 + np.abs(b).max())
    assert gu.device_error() == 0


def test_many_rows_of_few_logits():
    import torch
    rows, vocab = 150_001, 33
    x = torch.randn((rows, vocab), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    logp, ent = (torch.zeros(rows, device="cuda") for _ in range(2))
    ids = torch.zeros((rows, 3), dtype=torch.int32, device="cuda")
    t = torch.randint(0, vocab, (rows,), device="cuda", dtype=torch.int32)
    nb = thinmx.tt_token_logprobs_workspace_bytes(rows, vocab, 3)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    thinmx.tt_token_logprobs(x, thinmx.TT_LOGITS_F32, rows, vocab, vocab, 1.0, t, 3, logp, ent, ids, None, ws, nb)
    want = torch.log_softmax(x.double(), 1)
    # half steps: 33 + 8 in the sum, |x| <= 6 and its difference in an exponential's argument
    assert float((logp.double() - want.gather(1, t.long()[:, None])[:, 0]).abs().max()) <= (41 + 8 * 12) * 2.0 ** -24
    assert float((ent.double() + (want.exp() * want).sum(1)).abs().max()) <= 12 * (41 + 8 * 12) * 2.0 ** -24
    assert torch.equal(ids.long(), torch.sort(x, dim=1, descending=True, stable=True)[1][:, :3])
    assert gu.device_error() == 0


def test_two_graphs_on_one_workspace():
    """Captured apart, replayed in turn on one stream."""
    import torch
    nb = thinmx.tt_paged_tree_workspace_bytes(16, 4, 128)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    cases, graphs = [], []
    for seed, new, past in ((50, [9], [2500]), (51, [4, 30, 1], [20, 900, 40])):
        cache, starts, masks, words, q = setup(seed, (16, 4, 128), 16, False, new, past)
        alone = attend(_handle(cache), q, starts, masks, words, 0.1)
        kv, qd, st = _handle(cache), gu.dev(q), ints(starts.tolist())
        mk = gu.dev(br.words_of(masks, words).view(np.int32))
        out, lse = torch.zeros(q.shape, dtype=torch.int16, device="cuda"), torch.zeros(q.shape[:2], device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            thinmx.tt_paged_tree_attention(kv, qd, 16 * 128, st, len(q), 16, 0.1, 0.0, 0, None, None, mk, words, out, lse,
                                           ws, nb)
        cases.append((alone, out, lse, kv, qd, st, mk))
        graphs.append(graph)
    for _ in range(4):
        for g in graphs:
            g.replay()
    for g, (alone, out, lse, *_) in zip(reversed(graphs), reversed(cases)):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(gu.host(out, np.uint16), alone[0]) and np.array_equal(gu.host(lse), alone[1])
    assert gu.device_error() == 0


def test_a_drafted_step_in_a_graph():
    """Masks, attention, choices, walk, kept rows and new pages, captured together and replayed on new drafts: as the same
    calls one by one on a second cache."""
    import torch
    r = synth.rng(WID, 4, 0)
    heads, kvh, d, page, batch, n, width, vocab = 16, 4, 64, 16, 3, 6, 12, 3
    starts = ints([0, n, 2 * n, 3 * n])
    head = torch.randn((heads * d, vocab), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")

    class Side:
        def __init__(self):
            seed = torch.Generator(device="cuda").manual_seed(2)
            self.k, self.v = (torch.randn((60, kvh, page, d), generator=seed, device="cuda").bfloat16() for _ in range(2))
            self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
            self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
            self.kv = loader.paged_kv(self.k, self.v, self.table, self.lens)
            self.layers = loader.paged_layers([self.kv])
            self.parents, self.drafts = full((batch * n,), -1), full((batch * n,), 0)
            self.q, self.out = (torch.zeros((batch * n, heads, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            nb = thinmx.tt_paged_tree_workspace_bytes(heads, kvh, d)
            self.ws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
            nb = thinmx.tt_paged_pages_workspace_bytes(self.kv)
            self.pws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
            nb = thinmx.tt_token_logprobs_workspace_bytes(batch * n, vocab, 1)
            self.lws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
            self.masks, self.positions = full((batch * n, 1)), full((batch * n,))
            self.ids, self.path, self.counts, self.next = full((batch * n, 1)), full((batch, n)), full((batch,)), full((batch,))
            self.left, self.want = full((1,)), full((batch,))

        def step(self):
            torch.add(self.lens, n, out=self.want)
            thinmx.tt_paged_resize(self.kv, self.want, None, self.table, self.lens, self.left, *self.pws)
            self.lens.copy_(self.want)
            thinmx.tt_draft_tree(self.parents, starts, self.lens, batch, batch * n, 1, self.masks, self.positions)
            thinmx.tt_paged_tree_attention(self.kv, self.q, heads * d, starts, batch * n, heads, 0.125, 0.0, 0, None, None,
                                           self.masks, 1, self.out, None, *self.ws)
            logits = (self.out.float().reshape(batch * n, -1, 1) * head).sum(1)
            thinmx.tt_token_logprobs(logits, thinmx.TT_LOGITS_F32, batch * n, vocab, vocab, 1.0, None, 1, None, None, self.ids,
                                     None, *self.lws)
            thinmx.tt_draft_accept(self.parents, self.drafts, self.ids, starts, batch, batch * n, n, self.path, self.counts,
                                   self.next)
            thinmx.tt_paged_keep(self.layers, 1, starts, self.path, n, self.counts, self.lens)

        def seen(self):
            return [gu.host(x) for x in (self.table, self.lens, self.ids, self.path, self.counts, self.next, self.left,
                                         self.masks, self.positions, self.out.view(torch.int16), self.k.view(torch.int16),
                                         self.v.view(torch.int16))]

    a, b = Side(), Side()
    a.step()  # first uses outside of a capture
    torch.cuda.synchronize()
    a = Side()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    accepted = 0
    for i in range(10):
        parents = [p for _ in range(batch) for p in br.parents_of(r, n)]
        drafts = [int(x) for x in r.integers(0, vocab, batch * n)]
        q = synth.f32_to_bf16_bits(r.standard_normal((batch * n, heads, d)).astype(np.float32))
        for s in (a, b):
            s.parents.copy_(ints(parents))
            s.q.view(torch.int16).copy_(gu.dev(q))
            s.drafts.copy_(ints(drafts))
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert all(np.array_equal(x, y) for x, y in zip(a.seen(), b.seen())), i
        accepted += int(gu.host(a.counts).sum())
    assert accepted > 10 * batch and gu.device_error() == 0
