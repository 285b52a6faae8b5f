"""Host-side checks of the drafted-tree, page and log-probability entry points: sizes and refusals, all before any
launch."""
import ctypes

import pytest

from bit_weight_only_mxfp4_gb300 import loader, thinmx

from .test_paged_abi import A, BAD_CACHES, kv, lib, status  # noqa: F401

BIG = 1 << 40


def tree(parents=A, starts=A, lens=A, batch=2, tokens=7, words=2, masks=A, positions=A):
    return status(thinmx.tt_draft_tree, parents, starts, lens, batch, tokens, words, masks, positions)


def accept(parents=A, drafts=A, chosen=A, starts=A, batch=2, tokens=7, width=4, path=A, counts=A, next=A):
    return status(thinmx.tt_draft_accept, parents, drafts, chosen, starts, batch, tokens, width, path, counts, next)


def attend(c, q=A, q_stride=2048, starts=A, tokens=7, heads=16, scale=0.1, softcap=0.0, window=0, slopes=None,
           sinks=None, masks=A, words=2, out=A, lse=None, ws=A, wsb=BIG):
    return status(thinmx.tt_paged_tree_attention, c, q, q_stride, starts, tokens, heads, scale, softcap, window, slopes,
                  sinks, masks, words, out, lse, ws, wsb)


def keep(layers, n=1, starts=A, path=A, width=4, counts=A, lens=A):
    return status(thinmx.tt_paged_keep, layers, n, starts, path, width, counts, lens)


def resize(c, want=A, held=None, table=A, lens=A, left=None, ws=A, wsb=BIG):
    return status(thinmx.tt_paged_resize, c, want, held, table, lens, left, ws, wsb)


def fork(layers, n=1, come=A, held=None, table=A, lens=A, left=None, ws=A, wsb=BIG):
    return status(thinmx.tt_paged_fork, layers, n, come, held, table, lens, left, ws, wsb)


def compact(layers, n=1, held=None, table=A, span=None, ws=A, wsb=BIG):
    return status(thinmx.tt_paged_compact, layers, n, held, table, span, ws, wsb)


def logprobs(logits=A, kind=1, rows=3, vocab=1000, stride=1000, scale=1.0, targets=A, top=5, logp=A, entropy=A, ids=A,
             tops=A, ws=A, wsb=BIG):
    return status(thinmx.tt_token_logprobs, logits, kind, rows, vocab, stride, scale, targets, top, logp, entropy, ids,
                  tops, ws, wsb)


@pytest.mark.parametrize("bad,want", BAD_CACHES, ids=lambda x: str(x).replace(" ", ""))
def test_bad_caches_are_refused_by_every_call(lib, bad, want):
    for call in (attend, keep, resize, fork, compact):
        assert call(kv(**bad)) == want
    assert thinmx.tt_paged_pages_workspace_bytes(kv(**bad)) == 0


def test_no_cache(lib):
    for call in (attend, keep, resize, fork, compact):
        assert call(None) == 1
    assert thinmx.tt_paged_pages_workspace_bytes(None) == 0


def test_draft_tree_refusals(lib):
    assert tree(batch=0) == tree(tokens=-1) == tree(tokens=1 << 31) == tree(words=0) == 2
    assert tree(batch=1025) == tree(words=9) == 5
    for name in ("parents", "starts", "lens", "masks", "positions"):
        assert tree(**{name: None}) == 1
        assert tree(**{name: A + 2}) == 3
    thinmx.tt_draft_tree(A, A, A, 2, 0, 2, A, A, stream=0)  # no tokens: nothing to do


def test_draft_accept_refusals(lib):
    assert accept(batch=0) == accept(tokens=-1) == accept(tokens=1 << 31) == accept(width=0) == 2
    assert accept(batch=1025) == 5
    for name in ("parents", "drafts", "chosen", "starts", "path", "counts", "next"):
        assert accept(**{name: None}) == 1
        assert accept(**{name: A + 1}) == 3


def test_tree_attention_refusals(lib):
    c = kv()
    assert attend(c, heads=0) == attend(c, heads=18) == 2
    assert attend(c, heads=68, q_stride=68 * 128) == 5
    assert attend(c, scale=float("nan")) == attend(c, softcap=float("inf")) == 4
    assert attend(c, softcap=-1.0) == attend(c, window=-1) == attend(c, q_stride=2040) == attend(c, q_stride=2052) == 2
    assert attend(c, tokens=-1) == attend(c, tokens=1 << 31) == 2
    assert attend(c, words=0) == 2
    assert attend(c, words=9) == 5
    # 2^17 tiles of keys for each of some 2^24 tiles of rows
    assert attend(kv(pages_per_seq=1 << 20, page_size=16), tokens=1 << 26) == 5
    for name in ("q", "starts", "masks", "out", "ws"):
        assert attend(c, **{name: None}) == 1
    assert attend(c, q=A + 8) == attend(c, out=A + 2) == attend(c, ws=A + 8) == attend(c, starts=A + 2) == 3
    for name in ("lse", "slopes", "sinks", "masks"):
        assert attend(c, **{name: A + 2}) == 3
    need = thinmx.tt_paged_tree_workspace_bytes(16, 4, 128)
    if need:
        assert attend(c, wsb=need - 1) == 8
    thinmx.tt_paged_tree_attention(c, A, 2048, A, 0, 16, 0.1, 0.0, 0, None, None, A, 2, A, None, A, BIG, stream=0)
    assert thinmx.tt_paged_tree_workspace_bytes(16, 3, 128) == 0
    assert thinmx.tt_paged_tree_workspace_bytes(16, 4, 96) == 0
    assert thinmx.tt_paged_tree_workspace_bytes(64, 2, 128) == 0


def test_layers_have_to_agree(lib):
    for call in (keep, fork, compact):
        assert call(kv(), n=0) == call(kv(), n=129) == 2
        for other in (dict(page_table=A + 64), dict(lens=A + 64), dict(num_pages=99), dict(page_size=32),
                      dict(kv_heads=8), dict(head_dim=64), dict(batch=1), dict(pages_per_seq=9),
                      dict(type=1, k_scales=A, v_scales=A)):
            assert call(loader.paged_layers([kv(), kv(**other)]), n=2) == 2
        assert call(loader.paged_layers([kv(), kv(k=A + 8)]), n=2) == 3
        assert call(loader.paged_layers([kv(), kv(v=None)]), n=2) == 1
    layers = loader.paged_layers([kv(k=A + 16 * i) for i in range(3)])
    assert isinstance(layers, ctypes.Array) and layers[2].k == A + 32


def test_keep_refusals(lib):
    assert keep(kv(), width=0) == 2
    for name in ("starts", "path", "counts", "lens"):
        assert keep(kv(), **{name: None}) == 1
        assert keep(kv(), **{name: A + 2}) == 3


def test_page_refusals(lib):
    c = kv()
    need = thinmx.tt_paged_pages_workspace_bytes(c)
    assert need > 0
    for call, counter in ((resize, "left"), (fork, "left"), (compact, "span")):
        assert call(c, table=None) == call(c, ws=None) == 1
        assert call(c, table=A + 2) == call(c, ws=A + 8) == call(c, **{counter: A + 2}) == 3
        assert call(c, wsb=need - 1) == 8
    assert resize(c, want=None) == resize(c, lens=None) == fork(c, come=None) == fork(c, lens=None) == 1
    assert resize(c, want=A + 2) == resize(c, lens=A + 1) == fork(c, come=A + 2) == fork(c, lens=A + 3) == 3


def test_logprobs_refusals(lib):
    assert logprobs(kind=2) == logprobs(kind=-1) == logprobs(rows=-1) == logprobs(rows=1 << 31) == 2
    assert logprobs(vocab=0) == logprobs(stride=999) == logprobs(top=-1) == logprobs(vocab=4, top=5) == 2
    assert logprobs(vocab=(1 << 30) + 1, stride=1 << 31) == logprobs(top=33) == 5
    assert logprobs(scale=0.0) == logprobs(scale=-1.0) == logprobs(scale=2.0 ** -101) == logprobs(scale=2.0 ** 101) == 2
    assert logprobs(scale=float("inf")) == logprobs(scale=float("nan")) == 4
    assert logprobs(targets=None) == logprobs(logits=None) == logprobs(ids=None) == 1
    assert logprobs(logits=A + 1) == logprobs(kind=0, logits=A + 2) == 3
    for name in ("targets", "logp", "entropy", "ids", "tops"):
        assert logprobs(**{name: A + 2}) == 3
    need = thinmx.tt_token_logprobs_workspace_bytes(3, 1000, 5)
    if need:
        assert logprobs(ws=None) == 1
        assert logprobs(ws=A + 8) == 3
        assert logprobs(wsb=need - 1) == 8
    thinmx.tt_token_logprobs(None, 1, 0, 1000, 1000, 1.0, None, 0, None, None, None, None, None, 0, stream=0)
    for bad in ((0, 1000, 5), (3, 0, 0), (3, 1000, -1), (3, 1000, 33)):
        assert thinmx.tt_token_logprobs_workspace_bytes(*bad) == 0


def test_more_layers_than_there_are(lib):
    two = loader.paged_layers([kv(), kv()])
    for call in (keep, fork, compact):
        with pytest.raises(ValueError):
            call(two, n=3)
        with pytest.raises(ValueError):
            call(kv(), n=2)
