"""The paged cache operators on values at the ends of their ranges, against 64-bit references: sinks that are not
finite, value scales far apart, values that are not finite, large caps, and what such values cost."""
import math

import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64
from .test_gpu_paged import DECODE_EPS, PREFILL_EPS, WID, _attend, _handle, _workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def _queries(seed, tokens, heads, d):
    return synth.normal_bf16(synth.rng(WID, seed, 1), (tokens, heads, d), 1.0)


# -------------------------------------------------------------------------------------------------------------- sinks
def _no_sinks(heads):
    """Every third head without a sink: minus infinity, and the type's lowest value."""
    s = synth.rng(WID, 200, 0).standard_normal(heads).astype(np.float32)
    s[::3] = -np.inf
    s[1::3] = np.finfo(np.float32).min
    return s


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64)])
def test_decode_heads_without_a_sink(heads, kvh, d, window, fp8):
    """A token that sees no key (an empty place, a sequence of holes, a window in holes): out 0, lse = the sink."""
    c = ref.Cache(200, [150, 33, 0, 700, 5000], kvh, d, 16, fp8)
    c.table[1, :] = -1
    c.table[0, 5:] = -1
    c.table[4, :] = -1  # in several parts
    q, sinks = _queries(200, 5, heads, d), _no_sinks(heads)
    got = _attend(_handle(c), q, None, 0.125, window=window, sinks=sinks)
    ref.check_attention(*got, ref.attention(c, q, None, 0.125, window=window, sinks=sinks), DECODE_EPS[fp8], "decode")
    assert np.array_equal(got[1][[1, 2, 4]], np.broadcast_to(sinks, (3, heads)))
    assert gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64)])
@pytest.mark.parametrize("new,lens,holes", [([30, 6, 14], [20, 0, 50], False), ([30, 40], [60, 300], True),
                                            ([20], [3000], True)], ids=["short", "holes", "parts"])
def test_prefill_heads_without_a_sink(heads, kvh, d, new, lens, holes, fp8):
    """The same for tokens of no place, for holes, and for holes in a piece that is split along its tokens."""
    c = ref.Cache(201, lens, kvh, d, 16, fp8)
    if holes:
        c.table[0, :] = -1
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q, sinks = _queries(201, int(starts[-1]), heads, d), _no_sinks(heads)
    got = _attend(_handle(c), q, starts, 0.125, sinks=sinks)
    ref.check_attention(*got, ref.attention(c, q, starts, 0.125, sinks=sinks), PREFILL_EPS, "prefill")
    none = 10 if not holes else new[0]
    assert np.array_equal(got[1][:none], np.broadcast_to(sinks, (none, heads)))
    assert gu.device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_sink_of_infinity_takes_everything(fp8):
    c = ref.Cache(202, [90, 33], 4, 128, 16, fp8)
    c.table[1, :] = -1
    sinks = np.zeros(16, np.float32)
    sinks[::2] = np.inf
    for starts, tokens in ((None, 2), (np.array([0, 20, 25], np.int32), 25)):
        out, lse = _attend(_handle(c), _queries(202, tokens, 16, 128), starts, 0.125, sinks=sinks)
        assert not bf16_to_f64(out[:, ::2]).any() and np.isposinf(lse[:, ::2]).all()
        assert np.isfinite(bf16_to_f64(out)).all() and np.isfinite(lse[:, 1::2]).all()


# ----------------------------------------------------------------------------------- weights times scales, FP8 decode
@pytest.mark.parametrize("ratio", [-16, -20, -30, -60])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64), (12, 1, 64), (32, 2, 128)])
def test_fp8_decode_small_scales_with_all_the_weight(heads, kvh, d, ratio):
    """The last 4 tokens have all the softmax (a steep distance bias) and value scales 2^ratio of those of their
    neighbours, which weigh e^-96 at most.  The bound is relative to what the 4 make: 2^-11, an f16 rounding of each
    weight times scale."""
    lens = [704, 304]
    c = ref.Cache(203, lens, kvh, d, 16, True)
    q = _queries(203, 2, heads, d)
    for b, n in enumerate(lens):
        t = np.arange(n - 4, n)
        at = (c.table[b, t // 16], slice(None), t % 16)
        c.v_scales[at] = (c.v_scales[at] * 2.0 ** ratio).astype(np.float32)
    opt = dict(slopes=np.full(heads, 24.0, np.float32), window=48)
    got = _attend(_handle(c), q, None, 0.125, **opt)
    ref.check_attention(*got, ref.attention(c, q, None, 0.125, **opt), DECODE_EPS[True], f"2^{ratio}")


def _flat_scores(seed, scores, v_scales, kvh, d):
    """Keys and queries of ones: the score of token t is scores[t].  Values of one code and sign, so that an error of
    the weights does not average out."""
    n = len(scores)
    c = ref.Cache(seed, [n], kvh, d, 16, True)
    t = np.arange(n)
    at = (c.table[0, t // 16], slice(None), t % 16)
    c.k[at], c.v[at] = 0x38, 0x3D  # 1, and 1.625
    c.k_scales[at] = np.asarray(scores, np.float32)[:, None]
    c.v_scales[at] = np.asarray(v_scales, np.float32)[:, None]
    return c


@pytest.mark.parametrize("gap", [12.0, 14.3, 16.3, 18.0])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64), (12, 1, 64)])
@pytest.mark.parametrize("where", [0, 200, -1])
def test_fp8_decode_one_heavy_token_of_small_values(heads, kvh, d, where, gap):
    """One token far above the rest whose value row is almost zero (an attention sink): the rest makes the output."""
    n = 700
    scores, vs = np.zeros(n), np.ones(n)
    scores[where], vs[where] = gap, 2.0 ** -40
    c = _flat_scores(204, scores, vs, kvh, d)
    q = np.full((1, heads, d), 0x3F80, np.uint16)
    got = _attend(_handle(c), q, None, 1.0 / d)
    ref.check_attention(*got, ref.attention(c, q, None, 1.0 / d), DECODE_EPS[True], f"gap {gap}")


@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64)])
@pytest.mark.parametrize("big", [100.0, 2.0 ** 20, 2.0 ** 24])
def test_fp8_decode_one_large_scale_of_small_weight(heads, kvh, d, big):
    """One token whose value scale is far above the others', 40 nats below them."""
    n = 100
    scores, vs = np.full(n, 40.0), np.full(n, 1.3)
    vs[5], scores[5] = big, 0.0
    scores[::3] = 37.0  # and others between
    c = _flat_scores(205, scores, vs, kvh, d)
    q = np.full((1, heads, d), 0x3F80, np.uint16)
    got = _attend(_handle(c), q, None, 1.0 / d)
    ref.check_attention(*got, ref.attention(c, q, None, 1.0 / d), DECODE_EPS[True], f"scale {big}")


def test_fp8_decode_heads_of_one_group_with_different_tokens():
    """Two heads of one kv head: one has all its weight on a row of a small scale, the other on one of a large scale."""
    c = ref.Cache(206, [120], 1, 64, 16, True)
    t = np.arange(120)
    at = (c.table[0, t // 16], 0, t % 16)
    c.k[at] = 0
    code = np.where(t < 60, 0x38, 0xB8)[:, None]  # +1 or -1
    c.k[at] = np.broadcast_to(code, (120, 64))
    c.k_scales[at] = 0.5
    c.v[at] = 0x3D
    c.v_scales[at] = np.where(t < 60, 1.0, 2.0 ** -28).astype(np.float32)
    q = np.empty((1, 2, 64), np.uint16)
    q[0, 0], q[0, 1] = 0x3F80, 0xBF80  # the score of a token: +-32
    got = _attend(_handle(c), q, None, 1.0)
    ref.check_attention(*got, ref.attention(c, q, None, 1.0), DECODE_EPS[True], "two heads")


@pytest.mark.parametrize("shift", [-120, -100, 100])
def test_fp8_decode_scales_at_the_ends_of_the_range(shift):
    """All value scales at 2^-120, 2^-100 and 2^100 of the usual ones (those below 2^-126 lose bits in 32 bits too)."""
    c = ref.Cache(207, [700, 33], 4, 128, 16, True)
    c.v_scales = (c.v_scales.astype(np.float64) * 2.0 ** shift).astype(np.float32)
    q = _queries(207, 2, 16, 128)
    out, lse = _attend(_handle(c), q, None, 0.125)
    w_out, w_lse, spread, slack = ref.attention(c, q, None, 0.125)
    y = bf16_to_f64(out).reshape(w_out.shape)
    tol = 2.0 ** -8 * np.abs(w_out) + (2.0 ** -11 + 2 * slack[..., None] + 2.0 ** -16) * spread + 2.0 ** -133
    assert np.isfinite(y).all() and np.all(np.abs(y - w_out) <= tol)


# ------------------------------------------------------------------------------------------------ values in sight
@pytest.mark.parametrize("heads,kvh,d", [(64, 8, 64), (16, 4, 128), (12, 1, 64)])
@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("n,t", [(1, 0), (100, 37), (100, 99), (5000, 4000)])
def test_decode_infinite_values_in_sight(n, t, bad, heads, kvh, d):
    """sum e^z v with v infinite and e^z > 0 is that infinity, whatever the weight's bits are."""
    j, dim = kvh - 1, 9
    c, clean = (ref.Cache(208, [n, 60], kvh, d, 16, False, junk=False) for _ in range(2))
    c.v[c.table[0, t // 16], j, t % 16, dim] = bad
    q = _queries(208, 2, heads, d)
    got = bf16_to_f64(_attend(_handle(c), q, None, 0.125)[0]).reshape(2, heads, d)
    want = bf16_to_f64(_attend(_handle(clean), q, None, 0.125)[0]).reshape(2, heads, d)
    hit = np.zeros((2, heads, d), bool)
    hit[0, j * (heads // kvh):(j + 1) * (heads // kvh), dim] = True
    assert np.array_equal(got[~hit], want[~hit])
    value = bf16_to_f64(np.uint16(bad))
    assert np.isnan(got[hit]).all() if bad == 0x7FC0 else (got[hit] == value).all()


# ---------------------------------------------------------------------------------------------------------------- caps
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kvh,d", [(16, 4, 128), (64, 8, 64)])
@pytest.mark.parametrize("cap", [1e3, 3e4, 1e5, 1e7, 1e20, 3.4e38])
def test_large_caps(cap, heads, kvh, d, fp8):
    """A cap far above the scores hardly bends them: its error must not grow with it.  c tanh(s / c) for |s| < c / 8 is
    s less s^3 / (3 c^2), in 32 bits off by a few 2^-24 |s|, which is below the slack of the scores' own sums (2 d steps
    of 2^-24 of sum |q k|, and |s| <= that sum), so the uncapped scores' slack is the bound, doubled for both."""
    cap = float(np.float32(cap))
    c = ref.Cache(209, [300, 41, 1], kvh, d, 16, fp8, k_std=3.0)
    scale = float(np.float32(1.0 / math.sqrt(d)))
    for starts, tokens, eps in ((None, 3, DECODE_EPS[fp8]), (np.array([0, 30, 41, 42], np.int32), 42, PREFILL_EPS)):
        q = _queries(209, tokens, heads, d)
        out, lse, spread, _ = ref.attention(c, q, starts, scale, softcap=cap)
        slack = 2 * ref.attention(c, q, starts, scale)[3]
        got = _attend(_handle(c), q, starts, scale, softcap=cap)
        ref.check_attention(*got, (out, lse, spread, slack), eps, f"cap {cap}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [1e-40, 1e-30, 1e-3, 0.5, 255.0, 257.0, 1000.0])
def test_caps_that_bend_the_scores(cap, fp8):
    """Scores below, around and above the cap; tiny caps make all weights alike."""
    cap = float(np.float32(cap))
    c = ref.Cache(210, [300, 41], 4, 128, 16, fp8, k_std=min(60.0, 3.0 + cap / 4))
    for starts, tokens, eps in ((None, 2, DECODE_EPS[fp8]), (np.array([0, 30, 41], np.int32), 41, PREFILL_EPS)):
        q = _queries(210, tokens, 16, 128)
        got = _attend(_handle(c), q, starts, 0.25, softcap=cap)
        ref.check_attention(*got, ref.attention(c, q, starts, 0.25, softcap=cap), eps, f"cap {cap}")


# ---------------------------------------------------------------------------------- what a value that is not finite costs
@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_one_value_not_finite_costs_little(fp8):
    """One NaN in a tile that the mask cuts, behind a long past and with a length that ends inside a page: only the
    tiles that were cleaned are read again.  (Read again whole, the past takes a hundred times the call.)"""
    import torch
    heads, kvh, d, new, past = 16, 4, 128, 2500, 17003
    n = new + past
    c = ref.Cache(211, [n], kvh, d, 64, fp8, junk=False)
    kv = _handle(c)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((new, heads, d), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    starts = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    ws = _workspace(heads, kvh, d)

    def call():
        thinmx.tt_paged_prefill_attention(kv, q, heads * d, starts, new, heads, 0.088, 0.0, 0, None, None, None, out, None,
                                          ws[0], ws[1])

    def best():
        call()
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean, want = best(), out.clone()
    t = past + 1201
    kv.tensors[1][int(c.table[0, t // 64]), 2, t % 64, 17] = 0x7F if fp8 else 0x7FC0
    dirty = best()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[t - past:, 8:12, 17] = True
    assert torch.equal(~torch.isfinite(out), hit)
    assert torch.equal(out[~hit], want[~hit])
    assert gu.device_error() == 0
    assert dirty <= 3 * clean, f"{clean:.3f} ms clean, {dirty:.3f} ms with one NaN"


def test_prefill_values_not_finite_between_holes():
    """Holes in tiles that the mask does not cut: values that are not finite are found in those tiles, too."""
    heads, kvh, d, n, new = 16, 4, 128, 1500, 100
    c, clean = (ref.Cache(212, [n], kvh, d, 16, False, junk=False) for _ in range(2))
    for x in (c, clean):
        x.table[0, [3, 20, 21, 60]] = -1  # tokens 48.., 320.., 960..
    at = (40, 330 + 30, 600, 975 + 20, 1450)  # beside holes, in a whole tile, and in a cut one
    for i, t in enumerate(at):
        c.v[c.table[0, t // 16], 1, t % 16, 7 + i] = 0x7F80 if i % 2 else 0x7FC0
    starts = np.array([0, new], np.int32)
    q = _queries(212, new, heads, d)
    got, want = (bf16_to_f64(_attend(_handle(x), q, starts, 0.125)[0]).reshape(new, heads, d) for x in (c, clean))
    hit = np.zeros((new, heads, d), bool)
    p = np.arange(n - new, n)
    for i, t in enumerate(at):
        hit[p >= t, 4:8, 7 + i] = True
        x = got[p >= t, 4:8, 7 + i]
        assert np.isposinf(x).all() if i % 2 else np.isnan(x).all()
    assert np.array_equal(~np.isfinite(got), hit)
    assert np.array_equal(got[~hit], want[~hit])


# ----------------------------------------------------------------------------------------------------------------- types
def test_caches_of_other_types_are_refused():
    import torch
    from bit_weight_only_mxfp4_gb300 import loader
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 4), (2,)))
    scales = torch.ones((8, 2, 16), device="cuda")

    def make(dtype, s=None):
        x = torch.zeros((8, 2, 16, 64), dtype=dtype, device="cuda")
        return loader.paged_kv(x, x.clone(), table, lens, s, s)

    make(torch.bfloat16)
    make(torch.float8_e4m3fn, scales)
    make(torch.uint8, scales)
    for dtype, s in ((torch.float16, None), (torch.float8_e5m2, scales), (torch.float8_e4m3fn, None),
                     (torch.bfloat16, scales), (torch.float32, None)):
        with pytest.raises(AssertionError):
            make(dtype, s)
