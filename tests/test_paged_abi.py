"""Host-side checks of the paged cache entry points: sizes and refusals, all before any launch."""
import ctypes

import pytest

from bit_weight_only_mxfp4_gb300 import build as tt_build
from bit_weight_only_mxfp4_gb300 import thinmx

A = 1 << 20  # an aligned address that is never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    tt_build.build()
    return thinmx.load()


def kv(**kw):
    f = dict(k=A, v=A, k_scales=None, v_scales=None, page_table=A, lens=A, num_pages=100, type=0, page_size=16,
             kv_heads=4, head_dim=128, batch=2, pages_per_seq=10)
    f.update(kw)
    return thinmx.tt_paged_kv(**f)


BAD_CACHES = [
    (dict(type=2), 2), (dict(num_pages=0), 2), (dict(kv_heads=0), 2), (dict(batch=0), 2), (dict(pages_per_seq=0), 2),
    (dict(head_dim=0), 2), (dict(page_size=0), 2), (dict(page_size=24), 5), (dict(page_size=256), 5),
    (dict(page_size=8), 5), (dict(head_dim=96), 5), (dict(kv_heads=65), 5), (dict(batch=1025), 5),
    (dict(num_pages=(1 << 31) // 64), 5), (dict(pages_per_seq=1 << 28), 5), (dict(k=None), 1), (dict(v=None), 1),
    (dict(page_table=None), 1), (dict(lens=None), 1), (dict(type=1), 1), (dict(type=1, k_scales=A), 1),
    (dict(k=A + 8), 3), (dict(v=A + 2), 3), (dict(page_table=A + 2), 3), (dict(lens=A + 1), 3),
    (dict(type=1, k_scales=A + 4, v_scales=A), 3),
]


def status(fn, *a):
    with pytest.raises(thinmx.ThinmxError) as e:
        fn(*a, stream=0)
    return e.value.status


def append(c, q=A, k=A, v=A, q_stride=2048, kv_stride=512, tokens=2, starts=None, heads=16, turns=A, rot=128,
           interleaved=0, positions=None, axes=1, pair_axis=None, q_out=A):
    return status(thinmx.tt_paged_rope_append, c, q, k, v, q_stride, kv_stride, tokens, starts, heads, turns, rot,
                  interleaved, positions, axes, pair_axis, q_out)


def decode(c, q=A, q_stride=2048, heads=16, scale=0.1, softcap=0.0, window=0, slopes=None, sinks=None, out=A, lse=None,
           ws=A, wsb=1 << 40):
    return status(thinmx.tt_paged_decode_attention, c, q, q_stride, heads, scale, softcap, window, slopes, sinks, out,
                  lse, ws, wsb)


def prefill(c, q=A, q_stride=2048, starts=A, tokens=7, heads=16, scale=0.1, softcap=0.0, window=0, slopes=None,
            sinks=None, prefix=None, out=A, lse=None, ws=A, wsb=1 << 40):
    return status(thinmx.tt_paged_prefill_attention, c, q, q_stride, starts, tokens, heads, scale, softcap, window,
                  slopes, sinks, prefix, out, lse, ws, wsb)


@pytest.mark.parametrize("bad,want", BAD_CACHES, ids=lambda x: str(x).replace(" ", ""))
def test_bad_caches_are_refused_by_every_call(lib, bad, want):
    assert append(kv(**bad)) == want
    assert decode(kv(**bad)) == want
    assert prefill(kv(**bad)) == want


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_of_almost_two_to_the_31_tokens(lib, page):
    """Tokens are counted in 32 bits up to a tile's end and a warp's furthest page: the last 4096 are refused."""
    most = ((1 << 31) - 4096) // page
    for call in (append, decode, prefill):
        for more in (1, 4096 // page - 1):
            assert call(kv(page_size=page, batch=1, pages_per_seq=most + more, num_pages=10)) == 5
        # accepted as a size: the next check refuses it
        assert call(kv(page_size=page, batch=1, pages_per_seq=most, num_pages=10, k=A + 8)) == 3


def test_no_cache(lib):
    assert append(None) == decode(None) == prefill(None) == 1


def test_append_refusals(lib):
    c = kv()
    assert append(c, tokens=3) == 2          # one token per sequence without starts
    assert append(c, tokens=-1) == 2
    assert append(c, heads=-1) == 2
    assert append(c, kv_stride=504) == 2     # less than a row
    assert append(c, kv_stride=516) == 2     # not a multiple of 8
    assert append(c, q_stride=2040) == 2
    assert append(c, rot=24) == 2
    assert append(c, rot=0) == 2
    assert append(c, rot=144) == 2
    assert append(c, axes=0, positions=A) == 2
    assert append(c, axes=5, positions=A) == 2
    assert append(c, axes=3) == 2            # several axes need positions
    assert append(c, q=None) == 1
    assert append(c, k=None) == 1
    assert append(c, v=None) == 1
    assert append(c, q_out=None) == 1
    assert append(c, q=A + 8) == 3
    assert append(c, k=A + 2) == 3
    assert append(c, q_out=A + 4) == 3
    assert append(c, turns=A + 4) == 3
    assert append(c, starts=A + 2, tokens=5) == 3
    assert append(c, positions=A + 1) == 3


def test_attention_refusals(lib):
    c = kv()
    for call in (decode, prefill):
        assert call(c, heads=0) == 2
        assert call(c, heads=18) == 2                      # not a multiple of kv_heads
        assert call(c, heads=68, q_stride=68 * 128) == 5   # 17-wide groups
        assert call(c, scale=float("nan")) == 4
        assert call(c, softcap=float("inf")) == 4
        assert call(c, softcap=-1.0) == 2
        assert call(c, window=-1) == 2
        assert call(c, q_stride=2040) == 2
        assert call(c, q_stride=2052) == 2
        assert call(c, q=None) == 1
        assert call(c, out=None) == 1
        assert call(c, ws=None) == 1
        assert call(c, wsb=thinmx.tt_paged_attention_workspace_bytes(16, 4, 128) - 1) == 8
        assert call(c, q=A + 8) == 3
        assert call(c, out=A + 2) == 3
        assert call(c, ws=A + 8) == 3
        assert call(c, lse=A + 2) == 3
        assert call(c, slopes=A + 1) == 3
        assert call(c, sinks=A + 3) == 3
    # more tiles than 32 bits count
    assert decode(kv(batch=1024, pages_per_seq=(1 << 31) // 16 - 1)) == 5
    assert prefill(c, starts=None) == 1
    assert prefill(c, tokens=-1) == 2
    assert prefill(c, tokens=1 << 31) == 2
    assert prefill(c, starts=A + 2) == 3
    assert prefill(c, prefix=A + 2) == 3


def test_rope_turns_refusals(lib):
    assert status(thinmx.tt_rope_turns, A, 0, A) == 2
    assert status(thinmx.tt_rope_turns, None, 4, A) == 1
    assert status(thinmx.tt_rope_turns, A, 4, A + 4) == 3


def test_workspace_sizes(lib):
    f = thinmx.tt_paged_attention_workspace_bytes
    assert f(16, 4, 128) > 0 and f(64, 8, 64) > 0
    assert f(15, 4, 128) == f(16, 4, 96) == f(68, 4, 64) == f(65, 65, 64) == f(0, 4, 64) == 0


def test_struct_size(lib):
    """The header's struct: six pointers, a 64-bit count and six 32-bit fields."""
    assert ctypes.sizeof(thinmx.tt_paged_kv) == 6 * 8 + 8 + 6 * 4
