"""Attention of drafted trees over the paged cache, and the trees' masks, against 64-bit references."""
import math

import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64
from .test_gpu_paged import _dev, _handle, _options

pytestmark = pytest.mark.gpu

WID = 161
# weights are rounded to bf16 before their product with the values (half a step, relative)
EPS = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def _workspace(heads, kvh, d):
    import torch
    nb = thinmx.tt_paged_tree_workspace_bytes(heads, kvh, d)
    return torch.full((max(nb, 16),), 0xA5, dtype=torch.uint8, device="cuda"), nb  # no initial contents needed


def attend(kv, q, starts, masks, words, scale, softcap=0.0, window=0, slopes=None, sinks=None, stride=None, ws=None,
           lse=True):
    import torch
    tokens, heads, d = q.shape
    ws = ws or _workspace(heads, kv.kv_heads, d)
    stride = stride or heads * d
    wide = np.full((tokens, stride), 0x7FC0, np.uint16)
    wide[:, :heads * d] = q.reshape(tokens, -1)
    out = torch.full((tokens, heads, d), 0x7FC0, dtype=torch.int16, device="cuda")
    lse = torch.full((tokens, heads), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    thinmx.tt_paged_tree_attention(kv, gu.dev(wide), stride, _dev(np.asarray(starts, np.int32)), tokens, heads, scale,
                                   softcap, window, _dev(slopes), _dev(sinks),
                                   _dev(br.words_of(masks, words).view(np.int32)), words, out, lse, ws[0], ws[1])
    torch.cuda.synchronize()
    return gu.host(out, np.uint16), None if lse is None else gu.host(lse)


def queries(seed, tokens, heads, d):
    return synth.f32_to_bf16_bits(synth.rng(WID, seed, 1).standard_normal((tokens, heads, d)).astype(np.float32))


def setup(seed, layout, page, fp8, new, past, words=None, chain=False, roots=False):
    heads, kvh, d = layout
    r = synth.rng(WID, seed, 2)
    cache = ref.Cache(seed, [n + p for n, p in zip(new, past)], kvh, d, page, fp8=fp8)
    starts = np.cumsum([0] + list(new))
    parents = [br.parents_of(r, n, chain, roots) for n in new]
    masks = [m for p in parents for m in br.masks_of(p)]
    return cache, starts, masks, words or max(1, -(-max(new) // 32)), queries(seed, int(starts[-1]), heads, d)


def check(seed, layout, page, fp8, new, past, what, words=None, chain=False, roots=False, stride=None, **opt):
    cache, starts, masks, words, q = setup(seed, layout, page, fp8, new, past, words, chain, roots)
    opt = _options(layout[0], seed, **opt)
    scale = 1.0 / math.sqrt(layout[2])
    got = attend(_handle(cache), q, starts, masks, words, scale, stride=stride, **opt)
    ref.check_attention(*got, br.tree_attention(cache, q, starts, masks, words, scale, **opt), EPS, what)
    assert gu.device_error() == 0


LAYOUTS = [(16, 4, 128), (64, 8, 64), (28, 4, 128), (8, 8, 64), (12, 1, 64), (16, 1, 128), (40, 10, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_layouts(layout, fp8):
    check(1, layout, 16, fp8, [7, 1, 12], [140, 3, 300], f"{layout} fp8={fp8}")


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [1]), ([2], [0]), ([64], [0]), ([5], [127]), ([5], [128]),
                                      ([5], [125]), ([33], [95]), ([64, 0, 3], [200, 0, 1000]),
                                      ([0, 1, 0], [0, 255, 0])], ids=str)
def test_tile_and_page_ends(page, new, past):
    for fp8 in (False, True):
        check(2, (8, 2, 64), page, fp8, new, past, f"{new} {past} page {page} fp8={fp8}", roots=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("opt", [dict(sinks=True), dict(alibi=True), dict(softcap=30.0), dict(softcap=1000.0),
                                 dict(window=3), dict(window=64), dict(window=300, alibi=True, sinks=True),
                                 dict(window=1)], ids=str)
def test_options(opt, fp8):
    check(3, (16, 4, 128), 32, fp8, [20, 9, 1], [300, 0, 77], f"{opt} fp8={fp8}", **opt)
    check(4, (8, 1, 64), 16, fp8, [40, 2], [90, 600], f"{opt} fp8={fp8}", chain=True, **opt)


@pytest.mark.parametrize("n,words", [(100, 4), (256, 8), (130, 5), (40, 1), (300, 8)])
def test_large_trees_and_masks_of_fewer_words(n, words):
    """New tokens past the mask's words are seen by none, and see what their row names."""
    check(5, (8, 2, 64), 16, False, [n, 3], [50, 700], f"{n} nodes, {words} words", words=words)
    check(6, (8, 1, 128), 64, True, [n, 3], [50, 700], f"{n} nodes, {words} words", words=words, alibi=True, window=40)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_context_is_split(fp8):
    check(7, (16, 4, 128), 64, fp8, [8], [9000], "one long sequence", sinks=True)
    check(8, (64, 8, 64), 16, fp8, [24, 2, 9], [5000, 11, 2600], "ragged")


def test_query_stride():
    check(9, (8, 2, 64), 16, False, [9, 4], [40, 400], "stride", stride=8 * 64 + 2 * 2 * 64)


def test_any_mask():
    """Masks that are no tree: empty rows, rows that do not name themselves, keys after the token."""
    heads, kvh, d = 8, 2, 64
    for fp8 in (False, True):
        r = synth.rng(WID, 10, 3)
        cache = ref.Cache(10, [60, 40, 20], kvh, d, 16, fp8=fp8)
        starts = [0, 20, 60, 80]
        masks = [int(r.integers(0, 1 << 40)) for _ in range(80)]
        masks[3] = masks[25] = masks[61] = 0
        q = queries(10, 80, heads, d)
        for opt in (dict(), dict(window=4, alibi=True), dict(sinks=True)):
            opt = _options(heads, 10, **opt)
            got = attend(_handle(cache), q, starts, masks, 2, 0.125, **opt)
            want = br.tree_attention(cache, q, starts, masks, 2, 0.125, **opt)
            ref.check_attention(*got, want, EPS, f"any mask {opt} fp8={fp8}")
        # the second sequence is new altogether, and this row of it sees nothing
        out, lse = attend(_handle(cache), q, starts, masks, 2, 0.125)
        assert not out[25].any() and np.isneginf(lse[25]).all()


def test_holes_and_rows_of_no_sequence():
    heads, kvh, d = 8, 2, 64
    for fp8 in (False, True):
        cache, starts, masks, words, q = setup(11, (heads, kvh, d), 16, fp8, [12, 6], [300, 100])
        cache.table[0, 3] = cache.table[0, 19] = cache.table[1, 0] = -1  # (page 19 has new tokens)
        q = np.concatenate((q, queries(12, 3, heads, d)))
        got = attend(_handle(cache), q, starts, masks + [0] * 3, words, 0.125)
        want = br.tree_attention(cache, q[:-3], starts, masks, words, 0.125)
        ref.check_attention(got[0][:-3], got[1][:-3], want, EPS, f"holes fp8={fp8}")
        assert (got[0][-3:] == 0x7FC0).all() and np.isnan(got[1][-3:]).all()  # left as they were
        # a page past the pool is an error, and a hole
        cache.table[0, 3] = cache.pages
        again = attend(_handle(cache), q, starts, masks + [0] * 3, words, 0.125)
        assert gu.device_error() == 2
        assert np.array_equal(got[0], again[0])


def test_fewer_cached_than_new():
    """lens < new tokens: those without a place see nothing and are seen by none."""
    heads, kvh, d = 4, 2, 64
    cache = ref.Cache(13, [5, 70], kvh, d, 16)
    starts, masks = [0, 9, 12], [(1 << (i + 1)) - 1 for i in range(9)] + [1, 3, 7]
    q = queries(13, 12, heads, d)
    got = attend(_handle(cache), q, starts, masks, 1, 0.125)
    # the last five of the nine have rows 0 .. 4; depths count the masks' bits
    want = br.tree_attention(cache, q[4:], [0, 5, 8], [m >> 4 for m in masks[4:9]] + masks[9:], 1, 0.125)
    ref.check_attention(got[0][4:], got[1][4:], want, EPS, "rows with a place")
    assert not got[0][:4].any() and np.isneginf(got[1][:4]).all()


def test_values_that_are_not_finite():
    """A NaN or infinity in a value row that a token does not see does not reach it; one that it sees does."""
    heads, kvh, d = 8, 2, 64
    for fp8 in (False, True):
        cache, starts, masks, words, q = setup(14, (heads, kvh, d), 16, fp8, [6], [200])
        masks = br.masks_of([-1, 0, 0, 1, 1, 2])
        at = cache.table[0, 203 // 16], 0, 203 % 16, 5  # node 3's value, kv head 0
        cache.v[at] = 0x7F if fp8 else 0x7F80
        out, lse = attend(_handle(cache), q, starts, masks, words, 0.125)
        y = bf16_to_f64(out).reshape(out.shape)
        bad = ~np.isfinite(y)
        assert bad[3, :4, 5].all() and bad.sum() == 4
        assert np.isfinite(lse).all()
        cache.v[at] = 0
        clean = attend(_handle(cache), q, starts, masks, words, 0.125)[0]
        assert np.array_equal(out[[0, 1, 2, 4, 5]], clean[[0, 1, 2, 4, 5]])


def test_same_workspace_streams_and_graphs():
    """Calls of several sizes on one workspace, on a stream of their own, captured and replayed with other lengths."""
    import torch
    layout = (16, 4, 128)
    ws = _workspace(*layout)
    cases = [setup(15, layout, 16, False, [9], [3000]), setup(16, layout, 16, False, [4, 30], [20, 500])]
    alone = [attend(_handle(c), q, st, m, w, 0.1) for c, st, m, w, q in cases]
    for i in (0, 1, 0, 1):
        c, st, m, w, q = cases[i]
        got = attend(_handle(c), q, st, m, w, 0.1, ws=ws)
        assert all(np.array_equal(x, y) for x, y in zip(got, alone[i]))
    c, st, m, w, q = cases[0]
    kv = _handle(c)
    qd, starts, masks = gu.dev(q), _dev(st.astype(np.int32)), _dev(br.words_of(m, w).view(np.int32))
    out = torch.zeros(q.shape, dtype=torch.int16, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    call = lambda: thinmx.tt_paged_tree_attention(kv, qd, 16 * 128, starts, 9, 16, 0.1, 0.0, 0, None, None, masks, w,  # noqa: E731
                                                  out, lse, ws[0], ws[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert np.array_equal(gu.host(out, np.uint16), alone[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (3009, 109, 9, 2048):
        kv.tensors[3].fill_(n)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.lens[0] = n
        ref.check_attention(gu.host(out, np.uint16), gu.host(lse), br.tree_attention(c, q, st, m, w, 0.1), EPS,
                            f"replayed at {n}")


@pytest.mark.parametrize("words", [1, 2, 8])
def test_draft_tree(words):
    import torch
    r = synth.rng(WID, 20, words)
    new = [min(n, 32 * words) for n in (1, 0, 32, 7, 64, 250)]
    trees = [br.parents_of(r, n, chain=i == 2, roots=i % 2 == 0) for i, n in enumerate(new)]
    starts = np.cumsum([0] + new).astype(np.int32)
    lens = np.array([n + 10 * i for i, n in enumerate(new)], np.int32)
    tokens = int(starts[-1]) + 2
    masks = torch.full((tokens, words), 77, dtype=torch.int32, device="cuda")
    positions = torch.full((tokens,), 77, dtype=torch.int32, device="cuda")
    flat = gu.dev(np.array([p for t in trees for p in t] + [0, 0], np.int32))
    thinmx.tt_draft_tree(flat, gu.dev(starts), gu.dev(lens), len(new), tokens, words, masks, positions)
    want = [m for t in trees for m in br.masks_of(t)]
    got = gu.host(masks).view(np.uint32)
    assert np.array_equal(got[:-2], br.words_of(want, words)) and (got[-2:] == 77).all()
    depth = [bin(m).count("1") - 1 for m in want]
    past = np.repeat(lens - np.array(new), new)
    assert np.array_equal(gu.host(positions), list(past + depth) + [77, 77])
    assert gu.device_error() == 0


def test_draft_tree_reports_what_is_no_tree():
    import torch
    masks, positions = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((40, 1), (40,)))
    starts, lens = gu.dev(np.array([0, 4, 40], np.int32)), gu.dev(np.array([9, 40], np.int32))
    parents = np.full(40, -1, np.int32)
    parents[:4] = [0, -2, 3, 1]  # its own parent, below -1, a later one; then a good one
    thinmx.tt_draft_tree(gu.dev(parents), starts, lens, 2, 40, 1, masks, positions)
    assert gu.device_error() == 2
    got = gu.host(masks)[:, 0].view(np.uint32)
    assert list(got[:4]) == [1, 2, 4, 8 | 2]
    assert list(got[4:36]) == [1 << i for i in range(32)] and list(got[36:]) == [0] * 4  # 36 nodes, 32 bits
    assert list(gu.host(positions)[:5]) == [5, 5, 5, 6, 4] and list(gu.host(positions)[36:]) == [4] * 4


def test_every_code_of_an_fp8_cache():
    """Keys and values of all 256 codes, subnormal ones and NaN too: with one token to see, its value row is the
    output and its score the log of the sum."""
    from . import paged_ref
    d, kvh, batch = 64, 4, 4
    cache = ref.Cache(21, [1] * batch, kvh, d, 16, fp8=True)
    codes = np.arange(256, dtype=np.uint8).reshape(kvh, d)
    for b in range(batch):
        at = cache.table[b, 0], slice(None), 0
        cache.k[at] = cache.v[at] = codes
        cache.k_scales[at] = cache.v_scales[at] = 1.0
    q = np.zeros((batch, 16 * kvh, d), np.uint16)
    for b in range(batch):
        for h in range(16 * kvh):
            q[b, h, 16 * b + h % 16] = 0x3F80  # picks one element of the key
    want = paged_ref.e4m3_to_f64(codes)
    # NaN in a key poisons only products with it; 0 * NaN is NaN as well: leave those keys to one row each
    for b in range(batch):
        cache.k[cache.table[b, 0], :, 0][np.isnan(want)] = 0
    out, lse = attend(_handle(cache), q, list(range(batch + 1)), [1] * batch, 1, 1.0)
    y = bf16_to_f64(out).reshape(batch, kvh, 16, d)
    assert np.array_equal(y, np.broadcast_to(want[None, :, None], y.shape), equal_nan=True)
    for b in range(batch):
        z = np.where(np.isnan(want), 0.0, want)[:, 16 * b:16 * b + 16].ravel()
        assert np.abs(lse[b] - z).max() <= 2.0 ** -22 * 448
