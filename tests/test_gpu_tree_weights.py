"""The weights of the tree attention keep 16 bits before their product with the values, as the decode attention's of a
bf16 cache do, and an infinite value that is seen gives that infinity."""
import math

import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth

from . import branch_ref as br
from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64
from .test_gpu_paged import _handle, _options
from .test_gpu_tree import attend, queries

pytestmark = pytest.mark.gpu

WID = 192
# a weight is a bf16 part below it and the rest, which lies below 2^-7 of the weight's power of two and is rounded to
# bf16: half a step of that is 2^-8 of 2^-8
EPS = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def setup(seed, layout, page, fp8, new, past):
    """Keys of small size: many weights of about the same size, and scores of small errors."""
    heads, kvh, d = layout
    r = synth.rng(WID, seed, 1)
    cache = ref.Cache(seed, [n + p for n, p in zip(new, past)], kvh, d, page, fp8=fp8, k_std=0.1)
    starts = np.cumsum([0] + list(new))
    masks = [m for n in new for m in br.masks_of(br.parents_of(r, n))]
    return cache, starts, masks, max(1, -(-max(new) // 32)), queries(seed, int(starts[-1]), heads, d)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("opt", [dict(), dict(sinks=True), dict(softcap=30.0), dict(softcap=1000.0),
                                 dict(window=40, alibi=True)], ids=str)
@pytest.mark.parametrize("layout", [(16, 4, 128), (64, 8, 64), (8, 8, 64), (28, 4, 128)], ids=str)
def test_weights(layout, opt, fp8):
    cache, starts, masks, words, q = setup(1, layout, 16, fp8, [9, 1, 6, 20], [3, 11, 150, 700])
    opt = _options(layout[0], 1, **opt)
    scale = 1.0 / math.sqrt(layout[2])
    got = attend(_handle(cache), q, starts, masks, words, scale, **opt)
    want = br.tree_attention(cache, q, starts, masks, words, scale, **opt)
    ref.check_attention(*got, want, EPS, f"{layout} {opt} fp8={fp8}")
    assert gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_in_parts(fp8):
    """Sequences whose row tiles are joined from parts."""
    for layout in ((16, 4, 128), (64, 8, 64)):
        cache, starts, masks, words, q = setup(2, layout, 64, fp8, [8], [9000])
        got = attend(_handle(cache), q, starts, masks, words, 0.1, sinks=np.full(layout[0], 1.0, np.float32))
        want = br.tree_attention(cache, q, starts, masks, words, 0.1, sinks=np.full(layout[0], 1.0, np.float32))
        ref.check_attention(*got, want, EPS, f"{layout} fp8={fp8}")
    assert gu.device_error() == 0


@pytest.mark.parametrize("past", [1, 90, 9000])
@pytest.mark.parametrize("layout", [(16, 4, 128), (8, 2, 64)], ids=str)
def test_infinite_values(layout, past):
    """Infinities in cached tokens and in new ones that some tokens see, with weights of about the same
    size, or of exactly 1: a token that sees one of them has it, one that sees both has no number."""
    heads, kvh, d = layout
    cache, starts, masks, words, q = setup(3, layout, 16, False, [6], [past])
    masks = br.masks_of([-1, 0, 0, 1, 1, 2])
    if past == 1:  # (equal scores: weights of exactly 1)
        cache.k[:] = 0
    put = lambda t, j, e, bits: cache.v.__setitem__((cache.table[0, t // 16], j, t % 16, e), bits)  # noqa: E731
    put(0, 0, 5, 0x7F80)             # all see it
    put(past // 2, 1, 3, 0xFF80)     # so they do this one
    put(past + 3, 1, 3, 0x7F80)      # and node 3 its own
    put(past + 4, 0, 7, 0xFF80)      # node 4 alone sees it
    out, lse = attend(_handle(cache), q, starts, masks, words, 0.125)
    y = bf16_to_f64(out).reshape(out.shape)
    want = np.zeros(out.shape)
    g = heads // kvh
    want[:, :g, 5] = np.inf
    want[:, g:2 * g, 3] = -np.inf
    want[3, g:2 * g, 3] = np.nan
    want[4, :g, 7] = -np.inf
    got = np.where(np.isfinite(y), 0.0, y)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isfinite(lse).all() and gu.device_error() == 0
