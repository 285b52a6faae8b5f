"""The paged cache operators on values at the ends of their ranges, against 64-bit references: sinks that are not
finite, value scales far apart, values that are not finite, large caps, and what such values cost."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth

from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64
from .test_gpu_paged import DECODE_EPS, PREFILL_EPS, WID, _attend, _handle

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
