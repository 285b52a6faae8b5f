"""The paged cache operators on the GPU against 64-bit references: append
with rotation, attention of one and of several new tokens per sequence."""
import math

import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64

pytestmark = pytest.mark.gpu

WID = 151


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def _dev(a):
    return None if a is None else gu.dev(a)


def _handle(c):
    """The cache on the device, as a tt_paged_kv that holds its tensors."""
    from bit_weight_only_mxfp4_gb300 import loader
    k, v = gu.dev(c.k), gu.dev(c.v)
    ks, vs = (gu.dev(c.k_scales), gu.dev(c.v_scales)) if c.fp8 else (None, None)
    return loader.paged_kv(k, v, gu.dev(c.table), gu.dev(c.lens), ks, vs)


def _workspace(heads, kvh, d):
    import torch
    nb = thinmx.tt_paged_attention_workspace_bytes(heads, kvh, d)
    assert nb > 0
    return torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb


def _attend(kv, q, starts, scale, softcap=0.0, window=0, slopes=None, sinks=None, prefix=None, ws=None, stride=None):
    """Runs decode (starts None) or prefill; (out bits, lse)."""
    import torch
    tokens, heads, d = q.shape
    ws = ws or _workspace(heads, kv.kv_heads, d)
    if stride:
        wide = np.full((tokens, stride), 0x7FC0, np.uint16)
        wide[:, :heads * d] = q.reshape(tokens, -1)
        qd = gu.dev(wide)
    else:
        qd, stride = gu.dev(q), heads * d
    out = torch.full((tokens, heads, d), 0x7FC0, dtype=torch.int16, device="cuda")
    lse = torch.full((tokens, heads), float("nan"), dtype=torch.float32, device="cuda")
    slopes, sinks, prefix, starts = _dev(slopes), _dev(sinks), _dev(prefix), _dev(starts)
    if starts is None:
        thinmx.tt_paged_decode_attention(kv, qd, stride, heads, scale, softcap, window, slopes, sinks, out, lse, ws[0],
                                         ws[1])
    else:
        thinmx.tt_paged_prefill_attention(kv, qd, stride, starts, tokens, heads, scale, softcap, window, slopes, sinks,
                                          prefix, out, lse, ws[0], ws[1])
    torch.cuda.synchronize()
    return gu.host(out, np.uint16), gu.host(lse)


def _options(heads, seed, softcap=0.0, window=0, alibi=False, sinks=False):
    r = synth.rng(WID, seed, 9)
    return dict(softcap=softcap, window=window,
                slopes=(2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32) if alibi else None,
                sinks=r.standard_normal(heads).astype(np.float32) if sinks else None)


# What the weights are rounded to before their product with the values (half a step, relative): in the decode kernel
# two bf16 terms (2^-16), or f16 on an FP8 cache (2^-11; weights far below the largest keep 2^-25 of it, which 2^-11 of
# sum w |v| covers at these sizes); in the prompt kernel bf16 (2^-8).
DECODE_EPS = {False: 2.0 ** -16, True: 2.0 ** -11}
PREFILL_EPS = 2.0 ** -8


def _decode_case(seed, heads, kvh, d, page, fp8, lens, k_std=1.0, cache=None, scale=None, stride=None, **opt):
    c = cache or ref.Cache(seed, lens, kvh, d, page, fp8, k_std)
    q = synth.normal_bf16(synth.rng(WID, seed, 1), (len(c.lens), heads, d), 1.0)
    scale = float(np.float32(1.0 / math.sqrt(d) if scale is None else scale))
    o = _options(heads, seed, **opt)
    got = _attend(_handle(c), q, None, scale, stride=stride, **o)
    ref.check_attention(*got, ref.attention(c, q, None, scale, **o), DECODE_EPS[fp8],
                        f"decode {heads}/{kvh}/{d} page {page} fp8 {fp8}")
    assert gu.device_error() == 0
    return got


HEADS = [(16, 4, 128), (64, 8, 64), (8, 8, 64), (12, 1, 64), (32, 2, 128), (40, 10, 128), (28, 4, 128), (5, 1, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kvh,d", HEADS)
def test_decode_shapes(heads, kvh, d, page, fp8):
    _decode_case(heads + page, heads, kvh, d, page, fp8, [333, 1, 0, 130, 64, 17])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1025])
def test_decode_lengths(n, fp8):
    _decode_case(n, 64, 8, 64, 16, fp8, [n])
    _decode_case(n, 16, 4, 128, 32, fp8, [n])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d,n", [(64, 8, 64, 20001), (16, 4, 128, 9000)])
def test_decode_long(heads, kvh, d, n, fp8):
    _decode_case(7, heads, kvh, d, 64, fp8, [n, 5])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("opt", [
    dict(softcap=30.0), dict(softcap=1.0), dict(window=1), dict(window=16), dict(window=100), dict(window=5000),
    dict(alibi=True), dict(sinks=True), dict(softcap=20.0, window=70, alibi=True, sinks=True)],
    ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()))
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64), (12, 1, 64)])
def test_decode_options(heads, kvh, d, opt, fp8):
    _decode_case(31, heads, kvh, d, 16, fp8, [300, 0, 1, 90, 16, 1500], k_std=3.0, **opt)


def test_decode_of_many_sequences():
    r = synth.rng(WID, 5, 0)
    _decode_case(5, 8, 8, 64, 16, False, r.integers(0, 40, 1024))
    _decode_case(6, 16, 4, 128, 16, True, r.integers(0, 300, 300))


def test_decode_strided_queries():
    _decode_case(8, 16, 4, 128, 16, False, [70, 3, 200], stride=16 * 128 + 1024)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 40])
def test_decode_holes(window, fp8):
    """Holes at the start (pages a window has left behind), in the middle, and everywhere; the pages hold NaN."""
    c = ref.Cache(12, [150, 64, 33, 700], 4, 128, 16, fp8, junk=False)
    for b, pages in ((0, [0, 1, 4]), (1, [0, 1, 2, 3]), (2, [2]), (3, [0, 3, 4, 5, 20, 43])):
        for i in pages:
            gone = c.table[b, i]
            c.table[b, i] = -1
            if fp8:
                c.k[gone] = c.v[gone] = 0x7F
                c.k_scales[gone] = c.v_scales[gone] = np.nan
            else:
                c.k[gone] = c.v[gone] = 0x7FC0
    _decode_case(12, 16, 4, 128, 16, fp8, None, cache=c, window=window)
    _decode_case(12, 16, 4, 128, 16, fp8, None, cache=c, window=window, sinks=True)


@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80, 0xFF7F], ids=["nan", "inf", "-inf", "lowest"])
def test_masked_keys_and_values_do_not_matter(bad):
    """Keys and values before the window and past the length, in pages that are read, hold NaN, infinities or the
    type's lowest value."""
    c = ref.Cache(13, [100, 47], 8, 64, 64, False, junk=False)
    clean = ref.Cache(13, [100, 47], 8, 64, 64, False, junk=False)
    for b in range(2):
        n = int(c.lens[b])
        for t in list(range(n - 20)) + list(range(n, -(-n // 64) * 64)):
            c.k[c.table[b, t // 64], :, t % 64] = bad
            c.v[c.table[b, t // 64], :, t % 64] = bad
    a = _decode_case(13, 64, 8, 64, 64, False, None, cache=clean, window=20)
    q = synth.normal_bf16(synth.rng(WID, 13, 1), (2, 64, 64), 1.0)
    scale = float(np.float32(0.125))
    b = _attend(_handle(c), q, None, scale, window=20)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    starts = np.array([0, 1, 2], np.int32)
    a, b = (_attend(_handle(x), q, starts, scale, window=20) for x in (clean, c))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_peaked_and_flat(fp8):
    _decode_case(14, 64, 8, 64, 16, fp8, [1500, 700], k_std=4.0, scale=0.5)
    _decode_case(14, 64, 8, 64, 16, fp8, [1500, 700], scale=0.0)
    _decode_case(14, 16, 4, 128, 16, fp8, [900], scale=-0.05)


def _scaled_cache(seed):
    """FP8 rows whose scales differ by 2^20, some of them zero rows with scale zero."""
    c = ref.Cache(seed, [400], 4, 128, 16, True)
    r = synth.rng(WID, seed, 3)
    c.v_scales *= np.exp2(r.integers(-10, 11, c.v_scales.shape)).astype(np.float32)
    c.v_scales[:, :, 3] = 0.0
    c.v[:, :, 3] = 0
    c.k_scales[:, :, 5] = 0.0
    c.k[:, :, 5] = 0
    return c


def test_fp8_scales_of_many_sizes():
    c = _scaled_cache(15)
    _decode_case(15, 16, 4, 128, 16, True, None, cache=c)
    q = synth.normal_bf16(synth.rng(WID, 16, 1), (300, 16, 128), 1.0)
    starts = np.array([0, 300], np.int32)
    got = _attend(_handle(c), q, starts, 0.125)
    ref.check_attention(*got, ref.attention(c, q, starts, 0.125), PREFILL_EPS, "scales")


def test_decode_is_deterministic_and_reuses_its_workspace():
    import torch
    nb = max(_workspace(32, 2, 128)[1], _workspace(64, 8, 64)[1])
    ws = (torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb)
    first = {}
    for rep in range(3):
        for i, (heads, kvh, d, lens) in enumerate([(32, 2, 128, [3000]), (64, 8, 64, [700, 0, 5000, 33]),
                                                   (16, 4, 128, [1]), (16, 4, 128, [4000] * 5)]):
            c = ref.Cache(40 + i, lens, kvh, d, 16)
            q = synth.normal_bf16(synth.rng(WID, 40 + i, 1), (len(lens), heads, d), 1.0)
            got = _attend(_handle(c), q, None, 0.125, ws=ws)
            if rep == 0:
                first[i] = got
                ref.check_attention(*got, ref.attention(c, q, None, 0.125), DECODE_EPS[False], f"{i}")
            assert np.array_equal(got[0], first[i][0]) and np.array_equal(got[1], first[i][1])
    assert gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_past_two_to_the_32_elements(fp8):
    """A pool of 2^32 elements and more, read and written in its last pages."""
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    heads, kvh, d, page = 16, 8, 128, 128
    pages = (1 << 32) // (kvh * page * d) + 4
    small = ref.Cache(50, [200], kvh, d, page, fp8, junk=False, spare=0)
    dt = torch.uint8 if fp8 else torch.int16
    k, v = (torch.zeros((pages, kvh, page, d), dtype=dt, device="cuda") for _ in range(2))
    ks = vs = None
    k[-2:], v[-2:] = gu.dev(small.k), gu.dev(small.v)
    if fp8:
        ks, vs = (torch.zeros((pages, kvh, page), dtype=torch.float32, device="cuda") for _ in range(2))
        ks[-2:], vs[-2:] = gu.dev(small.k_scales), gu.dev(small.v_scales)
    kv = loader.paged_kv(k, v, gu.dev(small.table + np.int32(pages - 2)), gu.dev(small.lens), ks, vs)
    q = synth.normal_bf16(synth.rng(WID, 50, 1), (1, heads, d), 1.0)
    want = ref.attention(small, q, None, 0.0625)
    ref.check_attention(*_attend(kv, q, None, 0.0625), want, DECODE_EPS[fp8], "far pages")
    ref.check_attention(*_attend(kv, q, np.array([0, 1], np.int32), 0.0625), want, PREFILL_EPS, "far pages, prompt")
    x = synth.normal_bf16(synth.rng(WID, 51, 1), (1, 2 * kvh * d), 1.0)
    xd = gu.dev(x)
    thinmx.tt_paged_rope_append(kv, None, xd, xd.data_ptr() + 2 * kvh * d, 0, 2 * kvh * d, 1, None, 0, None, 0, 0, None,
                                1, None, None)
    torch.cuda.synchronize()
    at = int(small.table[0, 1]) + pages - 2
    for c, s, rows in ((k, ks, x[0, :kvh * d]), (v, vs, x[0, kvh * d:])):
        rows = rows.reshape(kvh, d)
        if fp8:
            y = ref.e4m3_to_f64(gu.host(c[at, :, 199 % page])) * gu.host(s[at, :, 199 % page]).astype(np.float64)[:, None]
            r = bf16_to_f64(rows).reshape(kvh, d)
            assert np.all(np.abs(y - r) <= 2.0 ** -4 * np.abs(r) + 2.0 ** -9 * np.abs(r).max(1)[:, None] / 448)
        else:
            assert np.array_equal(gu.host(c[at, :, 199 % page], np.uint16), rows)
    assert gu.device_error() == 0


def test_page_numbers_and_lengths_outside_are_reported_and_masked():
    """The kernels check every page number and length: a bad one is a hole, and the error word says so."""
    import torch
    lens = [100, 40]
    q = synth.normal_bf16(synth.rng(WID, 60, 1), (2, 16, 128), 1.0)
    both = ((None, DECODE_EPS[False]), (np.array([0, 1, 2], np.int32), PREFILL_EPS))
    for bad in (0, 2 ** 31 - 1):
        c, want = (ref.Cache(60, lens, 4, 128, 16) for _ in range(2))
        want.table[0, 2] = -1
        c.table[0, 2] = bad or c.pages  # one past the pool, or far past it
        for starts, eps in both:
            got = _attend(_handle(c), q, starts, 0.125)
            assert gu.device_error() == 2
            ref.check_attention(*got, ref.attention(want, q, None, 0.125), eps, "bad page")
    c = ref.Cache(60, lens, 4, 128, 16)
    c.lens = np.array([100000, -3], np.int32)  # clamped to the table's 112 rows, and to none
    for starts, _ in both:
        got = _attend(_handle(c), q, starts, 0.125)
        assert gu.device_error() == 2
        assert np.isneginf(got[1][1]).all() and not bf16_to_f64(got[0][1]).any()
    x = gu.dev(synth.normal_bf16(synth.rng(WID, 61, 1), (2, 8 * 128), 1.0))
    kv = _handle(c)
    before = gu.host(kv.tensors[0]).copy()
    thinmx.tt_paged_rope_append(kv, None, x, x.data_ptr() + 2 * 4 * 128, 0, 8 * 128, 2, None, 0, None, 0, 0, None, 1,
                                None, None)
    torch.cuda.synchronize()
    assert gu.device_error() == 2
    changed = np.argwhere((before != gu.host(kv.tensors[0])).any((1, 3)))
    assert [list(r) for r in changed] == [[c.table[0, 6], 15]]  # the clamped length's last row


# ------------------------------------------------------------------------------------------------------------ prompts
def _prefill_case(seed, heads, kvh, d, page, fp8, new, past, k_std=1.0, prefix=None, stride=None, extra=0, **opt):
    c = ref.Cache(seed, [n + p for n, p in zip(new, past)], kvh, d, page, fp8, k_std)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tokens = int(starts[-1])
    q = synth.normal_bf16(synth.rng(WID, seed, 2), (tokens + extra, heads, d), 1.0)
    scale = float(np.float32(1.0 / math.sqrt(d)))
    o = _options(heads, seed, **opt)
    pre = None if prefix is None else np.asarray(prefix, np.int32)
    got = _attend(_handle(c), q, starts, scale, prefix=pre, stride=stride, **o)
    want = ref.attention(c, q[:tokens], starts, scale, prefix=pre, **o)
    ref.check_attention(got[0][:tokens], got[1][:tokens], want, PREFILL_EPS, f"prefill {heads}/{kvh}/{d} {new} {past}")
    assert (got[0][tokens:] == 0x7FC0).all() and np.isnan(got[1][tokens:]).all()  # rows of no sequence stay
    assert gu.device_error() == 0
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kvh,d", HEADS)
def test_prefill_shapes(heads, kvh, d, page, fp8):
    _prefill_case(heads + page, heads, kvh, d, page, fp8, [70, 1, 0, 33, 5], [0, 200, 30, 64, 131])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 127, 128, 129, 200, 257])
def test_prefill_lengths(n, fp8):
    _prefill_case(n, 4, 4, 64, 16, fp8, [n], [0])
    _prefill_case(n, 16, 4, 128, 64, fp8, [n], [77])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("opt", [
    dict(softcap=30.0), dict(softcap=1.0), dict(window=1), dict(window=16), dict(window=100), dict(window=5000),
    dict(alibi=True), dict(sinks=True), dict(prefix=[50, 0, 300, 0]), dict(prefix=[400, 1, 260, 1], window=70),
    dict(softcap=20.0, window=70, alibi=True, sinks=True, prefix=[120, 0, 9, 1])],
    ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()).replace(" ", ""))
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64), (12, 1, 64)])
def test_prefill_options(heads, kvh, d, opt, fp8):
    _prefill_case(33, heads, kvh, d, 16, fp8, [140, 0, 60, 1], [160, 0, 250, 0], k_std=3.0, **opt)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_long(fp8):
    _prefill_case(34, 16, 4, 128, 64, fp8, [600, 300], [0, 1100])
    _prefill_case(35, 8, 1, 64, 128, fp8, [900], [2000])


def test_prefill_strides_and_rows_of_no_sequence():
    _prefill_case(36, 16, 4, 128, 16, False, [70, 20], [3, 0], stride=16 * 128 + 512, extra=9)


def test_prefill_more_new_tokens_than_length():
    """lens[b] < n_b: the first tokens have no place and see nothing."""
    c = ref.Cache(37, [20, 0, 50], 4, 128, 16)
    starts = np.array([0, 30, 36, 50], np.int32)
    q = synth.normal_bf16(synth.rng(WID, 37, 2), (50, 16, 128), 1.0)
    got = _attend(_handle(c), q, starts, 0.125)
    ref.check_attention(*got, ref.attention(c, q, starts, 0.125), PREFILL_EPS, "short")
    assert np.isneginf(got[1][:10]).all() and np.isneginf(got[1][30:36]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_holes(fp8):
    c = ref.Cache(38, [150, 64], 4, 128, 16, fp8)
    c.table[0, 0] = c.table[0, 3] = c.table[0, 9] = -1
    c.table[1, :] = -1
    starts = np.array([0, 140, 180], np.int32)
    q = synth.normal_bf16(synth.rng(WID, 38, 2), (180, 16, 128), 1.0)
    got = _attend(_handle(c), q, starts, 0.125)
    ref.check_attention(*got, ref.attention(c, q, starts, 0.125), PREFILL_EPS, "holes")


def test_prefill_is_deterministic_and_reuses_its_workspace():
    ws = _workspace(32, 2, 128)
    first = {}
    for rep in range(2):
        for i, (heads, kvh, d, new, past) in enumerate([(32, 2, 128, [100], [3000]), (16, 4, 128, [300, 5], [0, 900]),
                                                        (16, 4, 64, [1], [0])]):
            c = ref.Cache(70 + i, [a + b for a, b in zip(new, past)], kvh, d, 16)
            starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            q = synth.normal_bf16(synth.rng(WID, 70 + i, 1), (int(starts[-1]), heads, d), 1.0)
            got = _attend(_handle(c), q, starts, 0.125, ws=ws)
            if rep == 0:
                first[i] = got
                ref.check_attention(*got, ref.attention(c, q, starts, 0.125), PREFILL_EPS, f"{i}")
            assert np.array_equal(got[0], first[i][0]) and np.array_equal(got[1], first[i][1])


# ------------------------------------------------------------------------------------------------------------- append
def _append_case(seed, heads, kvh, d, page, fp8, lens, new=None, rot=None, interleaved=False, axes=1, far=0, extra=0,
                 edit=None, in_place=False):
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    c = ref.Cache(seed, lens, kvh, d, page, fp8, junk=False)
    r = synth.rng(WID, seed, 4)
    starts = None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tokens = len(lens) if new is None else int(starts[-1])
    row = (heads + 2 * kvh) * d + extra
    x = synth.normal_bf16(r, (tokens, row), 1.0)
    if edit:
        edit(x, heads, kvh, d)
    rot = d if rot is None else rot
    pos = pair_axis = None
    if axes > 1 or far:
        pos = r.integers(-5, far or 5000, (axes, tokens)).astype(np.int32)
        pos[:, -1] = far - 1 if far else 7
    if axes > 1:
        pair_axis = r.integers(0, axes, rot // 2).astype(np.uint8)
    inv = 1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))
    kv = _handle(c)
    xd, starts_d, pos_d, axis_d = gu.dev(x), _dev(starts), _dev(pos), _dev(pair_axis)
    turns = loader.rope_turns(torch.from_numpy(inv).cuda()) if rot else None
    q_out = torch.full((tokens, heads, d), 0x7FC0, dtype=torch.int16, device="cuda")
    base = xd.data_ptr()
    qp, q_stride = base, row
    if in_place:
        q_out.copy_(xd[:, :heads * d].reshape(tokens, heads, d))
        qp, q_stride = q_out.data_ptr(), heads * d
    thinmx.tt_paged_rope_append(kv, qp, base + 2 * heads * d, base + 2 * (heads + kvh) * d, q_stride, row, tokens,
                                starts_d, heads, turns, rot, interleaved, pos_d, axes, axis_d, q_out)
    torch.cuda.synchronize()
    # the reference
    xf = bf16_to_f64(x).reshape(tokens, row)[:, :row - extra].reshape(tokens, heads + 2 * kvh, d)
    seq = np.arange(tokens) if new is None else np.repeat(np.arange(len(lens)), new)
    n_b = np.ones(len(lens), int) if new is None else np.asarray(new)
    first = np.arange(len(lens)) if new is None else starts[:-1]
    place = np.asarray(lens)[seq] - n_b[seq] + (np.arange(tokens) - first[seq])
    y, slack = xf.copy(), np.zeros_like(xf)
    if rot:
        which = np.zeros(rot // 2, int) if pair_axis is None else pair_axis
        p = (place[:, None] if pos is None else pos[which].T).astype(np.float64)
        turned = xf[:, :heads + kvh, :rot]
        y[:, :heads + kvh, :rot] = ref.rotate(turned, p[:, None], inv, interleaved)
        # sine and cosine off by 2^-22 (the argument's rounding, pi 2^-25 rad, and the function's own), two products
        # and a sum in 32 bits; and the 64-bit reference's own angle, off by 2^-51 of it
        slack[:, :heads + kvh, :rot] = (2.0 ** -21 + np.abs(p).max() * inv.max() * 2.0 ** -51) * (
            2 * np.abs(np.where(np.isfinite(turned), turned, 0.0)).max(-1)[..., None])
    q = bf16_to_f64(gu.host(q_out, np.uint16)).reshape(tokens, heads, d)
    here = place >= 0
    want = np.where(here[:, None, None], y[:, :heads], 0.0)
    assert np.all(np.abs(q - want) <= 2.0 ** -8 * np.abs(want) + slack[:, :heads]), "q"
    # the cache: the appended rows, and nothing else
    names = ["k", "v"] + (["k_scales", "v_scales"] if fp8 else [])
    now = {n: gu.host(t, getattr(c, n).dtype) for n, t in zip(["k", "v", None, None, "k_scales", "v_scales"], kv.tensors)
           if n in names}
    new_rows = np.zeros((c.pages, page), bool)
    for t in np.flatnonzero(here):
        at = (c.table[seq[t], place[t] // page], slice(None), place[t] % page)
        new_rows[at[0], at[2]] = True
        for name, o in (("k", heads), ("v", heads + kvh)):
            want, s = y[t, o:o + kvh], slack[t, o:o + kvh]
            if not fp8:
                g = bf16_to_f64(now[name][at]).reshape(kvh, d)
                assert np.all(np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + s), f"{name} token {t}"
                continue
            code, sc = now[name][at], now[name + "_scales"][at].astype(np.float64)
            ok = np.isfinite(want).all(1)
            assert np.isnan(sc[~ok]).all() and not code[~ok].any()
            want, s, code, sc = want[ok], s[ok], code[ok], sc[ok]
            amax = np.abs(want).max(1)
            assert np.all(np.abs(sc - amax / 448) <= 2.0 ** -23 * amax / 448 + s.max(1) / 448 + 2.0 ** -149)
            g = ref.e4m3_to_f64(code) * sc[:, None]
            # half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below 2^-6), the quotient's rounding, and
            # saturation where the scale was rounded down
            tol = 2.0 ** -4 * np.abs(want) + (2.0 ** -10 + 448 * 2.0 ** -22) * sc[:, None] + 2 * s + 448 * 2.0 ** -149
            assert np.all(np.abs(g - want) <= tol), f"{name} token {t}"
    for name in names:
        old = getattr(c, name)
        same = (old.reshape(c.pages, kvh, page, -1) == now[name].reshape(c.pages, kvh, page, -1)).all((1, 3))
        assert same[~new_rows].all(), f"{name}: other rows changed"
    assert gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("heads,kvh,d", HEADS)
def test_append_one_token_each(heads, kvh, d, page, fp8):
    _append_case(heads + page, heads, kvh, d, page, fp8, [1, 16, 17, 0, 128, 129, 300])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rot,interleaved,axes", [(None, False, 1), (None, True, 1), (32, False, 1), (16, True, 3),
                                                  (None, False, 3), (48, False, 4), (0, False, 1)])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64), (5, 1, 128)])
def test_append_prompts(heads, kvh, d, rot, interleaved, axes, fp8):
    if rot == 0:
        axes = 1
    _append_case(81, heads, kvh, d, 16, fp8, [40, 0, 1, 77, 9], [40, 0, 1, 30, 2], rot, interleaved, axes)


def test_append_far_positions():
    for far in (1 << 20, (1 << 31) - 1):
        _append_case(82, 16, 4, 128, 16, False, [20, 5], [20, 3], far=far)
        _append_case(82, 16, 4, 128, 16, True, [20, 5], [20, 3], axes=3, far=far)


def test_append_strides_and_places():
    _append_case(83, 16, 4, 128, 32, False, [50, 3], [50, 3], extra=64)
    _append_case(84, 16, 4, 128, 32, False, [50, 3], [50, 3], in_place=True)
    _append_case(85, 16, 4, 128, 32, False, [5, 3, 0], [9, 3, 2])  # more new tokens than the length


def test_append_fp8_rows_of_zero_and_not_finite():
    def edit(x, heads, kvh, d):
        x[0, heads * d:(heads + 1) * d] = 0  # a zero key row
        x[1, (heads + kvh) * d:(heads + kvh + 1) * d] = 0
        x[2, (heads + 1) * d + 105] = 0x7FC0  # NaN
        x[3, (heads + kvh + 2) * d + 100] = 0xFF80  # -inf
        x[4, (heads + 1) * d:(heads + 2) * d] = 0x0001  # subnormal
    _append_case(86, 16, 4, 128, 16, True, [30], [8], rot=32, edit=edit)


def test_append_holes():
    import torch
    c = ref.Cache(87, [40, 33], 4, 128, 16, junk=False)
    c.table[0, 2] = -1
    kv = _handle(c)
    x = gu.dev(synth.normal_bf16(synth.rng(WID, 87, 4), (2, 8 * 128), 1.0))
    thinmx.tt_paged_rope_append(kv, None, x, x.data_ptr() + 2 * 4 * 128, 0, 8 * 128, 2, None, 0, None, 0, 0, None, 1,
                                None, None)
    torch.cuda.synchronize()
    changed = np.argwhere((gu.host(kv.tensors[0], np.uint16) != c.k).any((1, 3)))
    assert [list(r) for r in changed] == [[c.table[1, 2], 0]]
    assert gu.device_error() == 0


# ----------------------------------------------------------------------------------------------- together, as in a step
def test_steps_in_a_graph_on_another_stream():
    """A step's append and attention, captured once on a side stream and replayed while the lengths grow in place: the
    same as eager calls, and as the reference's."""
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    heads, kvh, d, page, steps = 16, 4, 128, 16, 5
    lens0 = [30, 14, 0, 100]
    c = ref.Cache(90, [n + steps for n in lens0], kvh, d, page, False, junk=False)
    inv = 1e4 ** (-np.arange(d // 2) / (d // 2))
    turns = loader.rope_turns(torch.from_numpy(inv).cuda())
    kv = _handle(c)
    lens = kv.tensors[3]
    x = synth.normal_bf16(synth.rng(WID, 90, 4), (steps, 4, (heads + 2 * kvh) * d), 1.0)
    xd = gu.dev(x)
    buf = xd[0].clone()
    q, out = (torch.empty((4, heads, d), dtype=torch.int16, device="cuda") for _ in range(2))
    lse = torch.empty((4, heads), dtype=torch.float32, device="cuda")
    ws = _workspace(heads, kvh, d)
    base = buf.data_ptr()

    def step():
        thinmx.tt_paged_rope_append(kv, base, base + 2 * heads * d, base + 2 * (heads + kvh) * d, buf.shape[1],
                                    buf.shape[1], 4, None, heads, turns, d, 0, None, 1, None, q)
        thinmx.tt_paged_decode_attention(kv, q, heads * d, heads, 0.125, 0.0, 0, None, None, out, lse, ws[0], ws[1])

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    lens.copy_(torch.tensor(lens0, dtype=torch.int32))
    torch.cuda.synchronize()
    got = []
    for i in range(steps):
        with torch.cuda.stream(side):
            buf.copy_(xd[i])
            lens += 1
            g.replay()
        torch.cuda.synchronize()
        got.append((gu.host(q, np.uint16).copy(), gu.host(out, np.uint16).copy(), gu.host(lse).copy()))
        c.k, c.v = gu.host(kv.tensors[0], np.uint16), gu.host(kv.tensors[1], np.uint16)
        c.lens = np.array([n + i + 1 for n in lens0], np.int32)
        ref.check_attention(got[i][1], got[i][2], ref.attention(c, got[i][0], None, 0.125), DECODE_EPS[False],
                            f"step {i}")
    lens.copy_(torch.tensor(lens0, dtype=torch.int32))
    for i in range(steps):
        buf.copy_(xd[i])
        lens += 1
        step()
        torch.cuda.synchronize()
        for a, b in zip(got[i], (gu.host(q, np.uint16), gu.host(out, np.uint16), gu.host(lse))):
            assert np.array_equal(a, b)
    assert gu.device_error() == 0


def test_prompt_then_decode_agree():
    """The last token of a prompt attended by the prompt kernel, and by the decode kernel."""
    for fp8 in (False, True):
        c = ref.Cache(91, [333], 8, 64, 16, fp8)
        q = synth.normal_bf16(synth.rng(WID, 91, 1), (20, 64, 64), 1.0)
        a = _attend(_handle(c), q, np.array([0, 20], np.int32), 0.125)
        b = _attend(_handle(c), q[-1:], None, 0.125)
        want = ref.attention(c, q[-1:], None, 0.125)
        ref.check_attention(a[0][-1:], a[1][-1:], want, PREFILL_EPS, "prompt")
        ref.check_attention(*b, want, DECODE_EPS[fp8], "decode")


# ------------------------------------------------------------------------------------------- larger and stranger cases
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d,batch,rot,interleaved", [(5, 1, 128, 3, 128, False), (16, 4, 64, 40, 32, True),
                                                              (8, 8, 128, 31, 64, False), (12, 1, 64, 33, 64, False)])
def test_append_many_tokens(heads, kvh, d, batch, rot, interleaved, fp8):
    """From eight tokens per SM on a CTA takes several tokens; an odd number of them, few and many sequences."""
    r = synth.rng(WID, batch, 6)
    new = r.integers(0, 2 * 1300 // batch, batch)
    new[0] += max(0, 1301 - int(new.sum()))
    if int(new.sum()) % 2 == 0:
        new[0] += 1
    _append_case(92 + batch, heads, kvh, d, 32, fp8, [int(n + r.integers(0, 40)) for n in new], [int(n) for n in new],
                 rot, interleaved)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d,batch,most", [(40, 10, 128, 64, 40), (8, 8, 64, 50, 300), (64, 8, 64, 90, 30)])
def test_prefill_more_pieces_than_sms(heads, kvh, d, batch, most, fp8):
    """Several pieces a CTA, with one and with two row tiles."""
    r = synth.rng(WID, batch, 7)
    new = [int(n) for n in r.integers(0, most, batch)]
    _prefill_case(batch, heads, kvh, d, 16, fp8, new, [int(n) for n in r.integers(0, 60, batch)])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d,new,past,opt", [
    (64, 4, 128, [641], [1300], {}),  # 152 pieces and some: those of the last round in parts
    (64, 4, 64, [641], [1300], {"prefix": [1900], "sinks": True}),
    (64, 4, 64, [700], [900], {"window": 500}),  # the last round's pieces are short
    (64, 4, 128, [300, 1, 0, 260, 200], [100, 1500, 0, 0, 1400], {}),  # taken in order of their lengths
    (64, 4, 64, [300, 30, 0, 260, 200, 300], [1300, 1500, 0, 700, 1400, 1300], {"prefix": [0, 1530, 0, 0, 1500, 900]}),
])
def test_prefill_rounds(heads, kvh, d, new, past, opt, fp8):
    got = _prefill_case(len(new), heads, kvh, d, 64, fp8, new, past, **opt)
    again = _prefill_case(len(new), heads, kvh, d, 64, fp8, new, past, **opt)
    assert (got[0] == again[0]).all() and (got[1] == again[1]).all()


@pytest.mark.parametrize("parts", [True, False])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80], ids=["nan", "inf", "-inf"])
def test_prefill_values_not_finite_reach_only_rows_that_see_them(bad, parts):
    """A value that is not finite makes its dimension so in the rows that see its token, and in no other: causal rows
    before it, rows whose window has left it behind, and every row of another kv head."""
    heads, kvh, d, n = (16, 4, 128, 300) if parts else (64, 16, 64, 1100)
    window, at, dim = 200, (70, 133, 260), 17
    c = ref.Cache(95, [n], kvh, d, 32, False, junk=False)
    for t in at:
        c.v[c.table[0, t // 32], 1, t % 32, dim] = bad
    starts = np.array([0, n], np.int32)
    q = synth.normal_bf16(synth.rng(WID, 95, 2), (n, heads, d), 1.0)
    got = bf16_to_f64(_attend(_handle(c), q, starts, 0.125, window=window)[0]).reshape(n, heads, d)
    clean = ref.Cache(95, [n], kvh, d, 32, False, junk=False)
    want = bf16_to_f64(_attend(_handle(clean), q, starts, 0.125, window=window)[0]).reshape(n, heads, d)
    p = np.arange(n)
    sees = np.zeros(n, bool)
    for t in at:
        sees |= (p >= t) & (p < t + window)
    hit = np.zeros((n, heads, d), bool)
    group = heads // kvh
    hit[sees, group:2 * group, dim] = True
    assert np.array_equal(~np.isfinite(got), hit)
    if bad != 0x7FC0:
        assert (got[hit] == bf16_to_f64(np.uint16(bad))).all()
    assert np.array_equal(got[~hit], want[~hit])


@pytest.mark.parametrize("what", ["code", "scale"])
def test_prefill_fp8_values_not_finite(what):
    """The same for an E4M3 NaN code, and for a row whose scale is NaN (what the append writes for a row that is not
    finite): the whole row of values."""
    n, t = 300, 140
    c, clean = (ref.Cache(96, [n], 4, 128, 32, True, junk=False) for _ in range(2))
    at = (c.table[0, t // 32], 2, t % 32)
    if what == "code":
        c.v[at][5] = 0x7F
    else:
        c.v_scales[at] = np.nan
    starts = np.array([0, n], np.int32)
    q = synth.normal_bf16(synth.rng(WID, 96, 2), (n, 16, 128), 1.0)
    got, want = (bf16_to_f64(_attend(_handle(x), q, starts, 0.125)[0]).reshape(n, 16, 128) for x in (c, clean))
    hit = np.zeros((n, 16, 128), bool)
    hit[t:, 8:12, 5 if what == "code" else slice(None)] = True
    assert np.array_equal(~np.isfinite(got), hit)
    # the scale stands beside all weights of the rows' products, so those rows are the only ones that may differ
    assert np.array_equal(got[~hit], want[~hit])


def test_decode_values_not_finite_in_sight():
    c = ref.Cache(97, [100, 60], 8, 64, 16, False, junk=False)
    c.v[c.table[0, 2], 3, 5, 9] = 0x7F80
    q = synth.normal_bf16(synth.rng(WID, 97, 1), (2, 64, 64), 1.0)
    got = bf16_to_f64(_attend(_handle(c), q, None, 0.125)[0]).reshape(2, 64, 64)
    hit = np.zeros((2, 64, 64), bool)
    hit[0, 24:32, 9] = True
    assert np.array_equal(~np.isfinite(got), hit)


@pytest.mark.parametrize("fp8", [False, True])
def test_example_layer(fp8):
    """A prompt and steps of a layer, decoded in a graph, against one prompt over all tokens.  Between the two lie the
    weights' rounding to bf16 in the prompt kernel (2^-8) and, after it, three bf16 roundings of the rows (2^-8 each)
    that a different last bit can turn the other way, once for each of the two."""
    from examples import paged_layer
    one, whole = paged_layer.serve(fp8, steps=9)
    one, whole = one.double().cpu().numpy(), whole.double().cpu().numpy()
    far = np.linalg.norm(one - whole, axis=-1) / np.linalg.norm(whole, axis=-1)
    assert far.max() <= 7 * 2.0 ** -8, far.max()
