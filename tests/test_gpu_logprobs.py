"""Log probabilities, entropy and top alternatives against 64 bits."""
import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import synth, thinmx

from . import gpu_util as gu
from .parity import bf16_to_f64

pytestmark = pytest.mark.gpu

WID = 163


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def run(logits, vocab, scale=1.0, targets=None, top=0, shift=0, entropy=True):
    """logits: bf16 bits (uint16) or fp32 [rows][stride]; shift: elements before the first row."""
    import torch
    rows, stride = logits.shape
    bf16 = logits.dtype == np.uint16
    flat = gu.dev(np.concatenate((np.zeros(shift, logits.dtype), logits.ravel())))[shift:]
    logp, ent = (torch.full((rows,), 77.0, device="cuda") for _ in range(2))
    ids = torch.full((rows, top), 77, dtype=torch.int32, device="cuda")
    tops = torch.full((rows, top), 77.0, device="cuda")
    nb = thinmx.tt_token_logprobs_workspace_bytes(rows, vocab, top)
    ws = torch.full((max(nb, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    t = None if targets is None else gu.dev(np.asarray(targets, np.int32))
    thinmx.tt_token_logprobs(flat, thinmx.TT_LOGITS_BF16 if bf16 else thinmx.TT_LOGITS_F32, rows, vocab, stride, scale,
                             t, top, None if t is None else logp, ent if entropy else None, ids if top else None,
                             tops if top else None, ws, nb)
    torch.cuda.synchronize()
    return gu.host(logp), gu.host(ent), gu.host(ids), gu.host(tops)


def values(logits):
    return bf16_to_f64(logits).reshape(logits.shape) if logits.dtype == np.uint16 else logits.astype(np.float64)


def check(logits, vocab, scale=1.0, targets=None, top=0, shift=0, what=""):
    x = values(logits)[:, :vocab]
    rows = len(x)
    got = run(logits, vocab, scale, targets, top, shift)
    z = x * float(np.float32(scale))
    m = z.max(1, keepdims=True)
    y = np.where(np.isneginf(z), 0.0, z - m)
    p = np.where(np.isneginf(z), 0.0, np.exp(y))
    s = p.sum(1)
    lse = np.log(s) + m[:, 0]
    p = p / s[:, None]
    a1, a2 = (p * np.abs(y)).sum(1), (p * y * y).sum(1)
    # What 32-bit arithmetic can be off by.  A weight e^y: the argument is rounded a few times (|y| 2^-22), the
    # exponential 2^-22; a sum of n numbers of one sign in a chain of at most n / 128 + 64 additions 2^-24 each.  So the
    # logarithm of the sum is off by chain + 2^-22 (1 + E|y|); the mean of y by E|y| (2 chain + 2^-21) + 2^-22 E y^2; z
    # and the differences by half a step of each number that is added.
    chain = (vocab / 128 + 64) * 2.0 ** -24
    tol = chain + 2.0 ** -22 * (2 + a1) + 2.0 ** -23 * (np.abs(m[:, 0]) + np.abs(lse))
    if targets is not None:
        t = np.asarray(targets)
        want = np.where(t < 0, 0.0, z[np.arange(rows), np.maximum(t, 0)] - lse)
        both = np.isneginf(want) & np.isneginf(got[0])
        with np.errstate(invalid="ignore"):
            off = np.where(both, 0.0, np.abs(got[0] - want)) - tol - 2.0 ** -22 * np.where(both, 0.0, np.abs(want))
        assert off.max() <= 0, f"{what} logp off by {off.max():.3e} over its bound"
    want = lse - m[:, 0] - (p * y).sum(1)
    off = np.abs(got[1] - want) - tol - a1 * (2 * chain + 2.0 ** -21) - 2.0 ** -22 * a2 - 2.0 ** -22 * np.abs(want)
    assert off.max() <= 0, f"{what} entropy off by {off.max():.3e} over its bound"
    if top:
        order = np.argsort(-x, axis=1, kind="stable")[:, :top]
        assert np.array_equal(got[2], order), what
        want = np.take_along_axis(z, order, 1) - lse[:, None]
        same = np.isneginf(want) & np.isneginf(got[3])
        with np.errstate(invalid="ignore"):
            off = np.where(same, 0.0, np.abs(got[3] - want) - 2.0 ** -22 * np.abs(want)) - tol[:, None]
        assert off.max() <= 0, f"{what} top off by {off.max():.3e} over its bound"
    assert gu.device_error() == 0


def normal(seed, rows, stride, bf16, std=3.0):
    x = (synth.rng(WID, seed, 0).standard_normal((rows, stride)) * std).astype(np.float32)
    return synth.f32_to_bf16_bits(x) if bf16 else x


SIZES = [1, 2, 7, 31, 33, 255, 1000, 1025, 4099, 32000, 50257]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("vocab", SIZES)
def test_sizes(vocab, bf16):
    r = synth.rng(WID, vocab, 1)
    for rows, pad, shift, top in ((1, 0, 0, min(5, vocab)), (3, 1, 1, 1), (2, 5, 3, min(20, vocab)),
                                  (4, 8, 0, min(32, vocab)), (2, 0, 0, 0)):
        targets = r.integers(-1, vocab, rows)
        check(normal(vocab, rows, vocab + pad, bf16), vocab, 1.0, targets, top, shift, f"{vocab} {rows} {pad} {shift}")


@pytest.mark.parametrize("bf16", [True, False])
def test_rows_and_scales(bf16):
    r = synth.rng(WID, 2, 2)
    for rows, vocab, scale in ((200, 2000, 0.5), (700, 515, 2.0), (17, 100352, 1.25), (1, 201088, 0.7), (310, 9000, 1e-3),
                               (5, 3000, 40.0)):
        check(normal(rows, rows, vocab, bf16), vocab, scale, r.integers(0, vocab, rows), 8, what=f"{rows} {vocab} {scale}")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("vocab", [40, 5000, 70001])
def test_ties_and_order(vocab, bf16):
    """Equal logits in falling order go by rising index, wherever they lie; also +0 and -0."""
    r = synth.rng(WID, vocab, 3)
    x = np.stack([np.zeros(vocab), np.where(r.random(vocab) < 0.5, 0.0, -0.0), np.arange(vocab) // 7 * 0.5,
                  -np.arange(vocab) * 0.25, r.integers(-2, 3, vocab), np.full(vocab, -1e4), np.full(vocab, 3e4)])
    x = x.astype(np.float32)
    x = synth.f32_to_bf16_bits(x) if bf16 else x
    for top in (1, 20, 32):
        check(x, vocab, 1.0, r.integers(0, vocab, len(x)), top, what=f"ties {vocab} {top}")


@pytest.mark.parametrize("bf16", [True, False])
def test_all_large_ones_in_one_place(bf16):
    """The top ones side by side, far apart, first, last."""
    for vocab in (6000, 130000):
        x = np.random.default_rng(1).standard_normal((6, vocab)).astype(np.float32)
        big = 50 + np.arange(40)
        x[0, :40], x[1, -40:], x[2, 3000:3040] = big, big, big[::-1]
        x[3, np.arange(40) * (vocab // 40)] = big
        x[4, np.arange(40) * 128] = big
        x[5, np.arange(40) * 8 + 5] = big[::-1]
        check(synth.f32_to_bf16_bits(x) if bf16 else x, vocab, 1.0, [0] * 6, 32, what="large ones")


@pytest.mark.parametrize("bf16", [True, False])
def test_minus_infinity(bf16):
    """Masked logits: probability 0; a row of one."""
    for vocab in (100, 20000):
        r = synth.rng(WID, vocab, 4)
        x = r.standard_normal((4, vocab)).astype(np.float32)
        x[0, r.random(vocab) < 0.9] = -np.inf
        x[1] = -np.inf
        x[1, vocab - 3] = -5.0
        x[2, :vocab // 2] = -np.inf
        x[3, 1:] = -np.inf
        x[0, 7] = -np.inf
        bits = synth.f32_to_bf16_bits(x) if bf16 else x
        check(bits, vocab, 1.0, [7, vocab - 3, vocab - 1, 0], 20, what="masked")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("vocab", [64, 30000])
def test_rows_without_probabilities(vocab, bf16):
    """NaN, +infinity, or nothing above -infinity: NaN everywhere; NaN comes first in the order."""
    x = synth.rng(WID, vocab, 5).standard_normal((4, vocab)).astype(np.float32)
    x[0, 9] = x[0, 40] = np.nan
    x[1, vocab - 1] = np.inf
    x[2] = -np.inf
    bits = synth.f32_to_bf16_bits(x) if bf16 else x
    logp, ent, ids, tops = run(bits, vocab, 1.0, [0, 1, 2, 3], 3)
    assert np.isnan(logp[:3]).all() and np.isnan(ent[:3]).all() and np.isnan(tops[:3]).all()
    assert np.isfinite(logp[3]) and np.isfinite(tops[3]).all()
    rest = np.argsort(-values(bits)[0], kind="stable")
    rest = rest[~np.isin(rest, (9, 40))]
    assert ids[0].tolist() == [9, 40, rest[0]] and ids[1, 0] == vocab - 1 and ids[2].tolist() == [0, 1, 2]
    assert gu.device_error() == 0


def test_no_token_and_a_token_past_the_vocabulary():
    x = normal(6, 3, 500, True)
    logp = run(x, 500, 1.0, [-1, -100, 499])[0]
    assert logp[0] == 0.0 and logp[1] == 0.0 and np.isfinite(logp[2]) and gu.device_error() == 0
    logp = run(x, 499, 1.0, [3, 499, -1])[0]
    assert np.isnan(logp[1]) and np.isfinite(logp[0]) and logp[2] == 0.0
    assert gu.device_error() == 2


def test_outputs_that_are_not_asked_for():
    x = normal(7, 3, 5000, False)
    all_of = run(x, 5000, 1.0, [1, 2, 3], 4)
    logp, ent, _, _ = run(x, 5000, 1.0, [1, 2, 3], 0, entropy=False)
    assert np.array_equal(logp, all_of[0]) and (ent == 77.0).all()
    logp, ent, ids, tops = run(x, 5000, 1.0, None, 4)
    assert (logp == 77.0).all()
    assert np.array_equal(ent, all_of[1]) and np.array_equal(ids, all_of[2]) and np.array_equal(tops, all_of[3])


def test_same_results_each_time_and_in_a_graph():
    import torch
    x = normal(8, 3, 150000, True)
    first = run(x, 150000, 1.0, [5, 6, 7], 20)
    for _ in range(3):
        assert all(np.array_equal(a, b) for a, b in zip(run(x, 150000, 1.0, [5, 6, 7], 20), first))
    d, t = gu.dev(x), gu.dev(np.array([5, 6, 7], np.int32))
    logp, ent = (torch.zeros(3, device="cuda") for _ in range(2))
    ids, tops = torch.zeros((3, 20), dtype=torch.int32, device="cuda"), torch.zeros((3, 20), device="cuda")
    nb = thinmx.tt_token_logprobs_workspace_bytes(3, 150000, 20)
    ws = torch.zeros(max(nb, 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            thinmx.tt_token_logprobs(d, 1, 3, 150000, 150000, 1.0, t, 20, logp, ent, ids, tops, ws, nb)
    for scale in (1, 0):
        d.copy_(gu.dev(x if scale else normal(9, 3, 150000, True)))
        graph.replay()
        torch.cuda.synchronize()
        want = first if scale else run(normal(9, 3, 150000, True), 150000, 1.0, [5, 6, 7], 20)
        assert all(np.array_equal(gu.host(a), b) for a, b in zip((logp, ent, ids, tops), want))


LOWEST = {True: float(np.uint32(0xff7f0000).view(np.float32)), False: float(np.finfo(np.float32).min)}


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("vocab", [50, 9000])
@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-6, 0.3, 1.0, 40.0, 1e4, 2.0 ** 100])
def test_logits_and_scales_of_any_size(scale, vocab, bf16):
    """Large logits beside small ones, the lowest finite logit beside -infinity: what counts is differences."""
    r = synth.rng(WID, vocab, 6)
    x = r.standard_normal((12, vocab)).astype(np.float32)
    for i, big in enumerate((2.0 ** 11, 2.0 ** 18, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100, 1.7e38)):
        x[i] = np.where(r.random(vocab) < 0.1, big * (1 - 2.0 ** -7 * r.integers(0, 3, vocab)), x[i])
        x[i, vocab // 2] = big
    x[6] -= np.float32(2.0 ** 60)
    x[7] = np.where(r.random(vocab) < 0.7, LOWEST[bf16], x[7])
    x[8] = np.where(r.random(vocab) < 0.7, LOWEST[bf16], -np.inf)
    x[9] = LOWEST[bf16]
    x[10] = -np.inf
    x[10, vocab // 3] = LOWEST[bf16]
    x[11] = np.where(r.random(vocab) < 0.5, -np.inf, np.clip(x[11], -3, 3) * 1e38)
    x[8, 3], x[11, 3] = LOWEST[bf16], 1e38
    logits = synth.f32_to_bf16_bits(x) if bf16 else x
    v = values(logits)
    targets = [3] * 10 + [vocab // 3, 3]
    logp, ent, ids, tops = run(logits, vocab, scale, targets, 5)
    y = (v - v.max(1, keepdims=True)) * float(np.float32(scale))
    gone = y < -800
    p = np.where(gone, 0.0, np.exp(np.where(gone, 0.0, y)))
    s = p.sum(1)
    p /= s[:, None]
    y0 = np.where(gone, 0.0, y)
    # as above, and without the sums' own size: differences come first, each rounded to half a step
    a1, a2 = (p * np.abs(y0)).sum(1), (p * y0 * y0).sum(1)
    chain = (vocab / 128 + 64) * 2.0 ** -24
    tol = chain + 2.0 ** -22 * (2 + a1) + 2.0 ** -22 * np.log(s)

    def near(got, want, tol, what, far=False):
        far = far | (want < -3e38)  # past what 32 bits hold
        assert (got[far] < -2e38).all(), what
        off = np.abs(got[~far] - want[~far]) - (np.broadcast_to(tol, want.shape) + 2.0 ** -21 * np.abs(want))[~far]
        assert off.size == 0 or off.max() <= 0, f"{what} off by {off.max():.3e} over its bound"

    with np.errstate(over="ignore"):  # differences past the type's range
        past = np.isinf(v.astype(np.float32) - v.max(1, keepdims=True).astype(np.float32))
    near(logp, y[np.arange(12), targets] - np.log(s), tol, "logp", past[np.arange(12), targets])
    near(ent, np.log(s) - (p * y0).sum(1), tol + a1 * (2 * chain + 2.0 ** -21) + 2.0 ** -22 * a2, "entropy")
    order = np.argsort(-v, axis=1, kind="stable")[:, :5]
    assert np.array_equal(ids, order)
    near(tops, np.take_along_axis(y, order, 1) - np.log(s)[:, None], tol[:, None], "top",
         np.take_along_axis(past, order, 1))
    assert gu.device_error() == 0
