"""The paged cache operators in 64 bits, on the host (test infrastructure), and the caches the tests build.

Everything is numpy: bf16 as uint16 bits, E4M3 as uint8 codes, values in float64.
"""
import numpy as np

from bit_weight_only_mxfp4_gb300 import synth

from .parity import bf16_to_f64


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = -a if c & 128 else a
    return t


_E4M3 = _e4m3_table()


def e4m3_to_f64(codes):
    return _E4M3[codes]


class Cache:
    """A page pool with seeded contents and a table of shuffled pages.  Table entries past a sequence's pages are
    holes, and with `junk` every row that no sequence has holds NaN."""

    def __init__(self, seed, lens, kv_heads, d, page, fp8=False, k_std=1.0, spare=2, junk=True):
        r = synth.rng(150, seed, 0)
        self.lens = np.asarray(lens, np.int32)
        self.page, self.fp8, self.kv_heads, self.d = page, fp8, kv_heads, d
        need = [-(-int(n) // page) for n in lens]
        self.pages = sum(need) + spare
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(need), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page, d)
        kf = r.standard_normal(shape).astype(np.float32) * np.float32(k_std)
        vf = r.standard_normal(shape).astype(np.float32)
        dead = np.ones((self.pages, page), bool)
        for b, n in enumerate(lens):
            t = np.arange(int(n))
            dead[self.table[b, t // page], t % page] = False
        self.k_scales = self.v_scales = None
        if fp8:
            import oracle
            (self.k, self.k_scales), (self.v, self.v_scales) = (
                [np.array(a) for a in oracle.fp8_quantize(x.reshape(-1, d))[:2]] for x in (kf, vf))
            self.k, self.v = self.k.reshape(shape), self.v.reshape(shape)
            self.k_scales, self.v_scales = self.k_scales.reshape(shape[:3]), self.v_scales.reshape(shape[:3])
        else:
            self.k, self.v = (synth.f32_to_bf16_bits(x).reshape(shape) for x in (kf, vf))
        if junk:
            for c in (self.k, self.v):
                np.moveaxis(c, 2, 1)[dead] = 0x7F if fp8 else 0x7FC0
            for c in (self.k_scales, self.v_scales) if fp8 else ():
                np.moveaxis(c, 2, 1)[dead] = np.nan

    def rows(self, b):
        """(keys, values, has a row) of sequence b in 64 bits: [kv_heads][len][d], [len]."""
        n = int(self.lens[b])
        t = np.arange(n)
        page = self.table[b, t // self.page]
        ok = page >= 0
        at = (np.where(ok, page, 0), slice(None), t % self.page)
        got = []
        for c, s in ((self.k, self.k_scales), (self.v, self.v_scales)):
            if self.fp8:
                x = e4m3_to_f64(c[at]) * s[at][..., None].astype(np.float64)
            else:
                x = bf16_to_f64(c[at]).reshape(n, self.kv_heads, self.d)
            got.append(np.where(ok[:, None, None], x, 0.0).transpose(1, 0, 2))
        return got[0], got[1], ok


def attention(cache, q, starts, scale, softcap=0.0, window=0, slopes=None, sinks=None, prefix=None):
    """(out, lse, spread, slack) in 64 bits for q bits [tokens][heads][d].  spread = sum of weight * |v|: what a
    relative error of the weights moves the output by; slack: a bound on the error of one score, in natural units, when
    its products are exact and summed in 32 bits in any order, with truncation (2 d steps of 2^-24 of sum |q k|), the
    cap's own error (softcap * 2^-21) and the bias's."""
    tokens, heads, d = q.shape
    qf = bf16_to_f64(q).reshape(q.shape)
    group = heads // cache.kv_heads
    out, spread = np.zeros((tokens, heads, d)), np.zeros((tokens, heads, d))
    lse = np.full((tokens, heads), -np.inf)
    slack = np.zeros((tokens, heads))
    if sinks is not None:
        lse[:] = sinks
    for b in range(len(cache.lens)):
        n = int(cache.lens[b])
        first, last = (b, b + 1) if starts is None else (int(starts[b]), int(starts[b + 1]))
        if n == 0 or first == last:
            continue
        k, v, ok = cache.rows(b)
        j = np.arange(n)
        p = (n - (last - first) + np.arange(last - first))[:, None]
        see = j <= p
        if prefix is not None:
            see = see | (j < int(prefix[b]))
        see = see & ok & (p >= 0)
        if window:
            see = see & (j > p - window)
        for h in range(heads):
            kk, vv = k[h // group], v[h // group]
            rows = qf[first:last, h]
            z = scale * (rows @ kk.T)
            err = 2 * d * 2.0 ** -24 * abs(scale) * (np.abs(rows) @ np.abs(kk).T)
            if softcap:
                z = softcap * np.tanh(z / softcap)
                err = np.minimum(err, 2 * softcap) + softcap * 2.0 ** -21
            if slopes is not None:
                z = z + float(slopes[h]) * (j - p)
                err = err + np.abs(z) * 2.0 ** -23
            z = np.where(see, z, -np.inf)
            top = z.max(1)
            if sinks is not None:
                top = np.maximum(top, float(sinks[h]))
            top = np.where(np.isfinite(top), top, 0.0)
            w = np.exp(z - top[:, None])
            total = w.sum(1)
            if sinks is not None:
                total = total + np.exp(float(sinks[h]) - top)
            w = w / np.where(total > 0, total, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse[first:last, h] = np.log(total) + top
            out[first:last, h] = w @ vv
            spread[first:last, h] = w @ np.abs(vv)
            slack[first:last, h] = np.where(see, err, 0.0).max(1)
    return out, lse, spread, slack


def check_attention(got_out, got_lse, want, weight_eps, what):
    """got_out bits.  |out - r| <= half a step of bf16 (2^-8 |r|) + the weights' relative error * sum w |v|, where the
    weights are off by weight_eps (what they are rounded to before the product) and twice the score's slack (weight and
    divisor), and 2^-16 for the sums, exponentials and the joining of parts; |lse - r| <= slack + 2^-20 (1 + |r|)."""
    out, lse, spread, slack = want
    y = bf16_to_f64(got_out).reshape(out.shape)
    assert np.isfinite(y).all(), f"{what}: not finite"
    tol = 2.0 ** -8 * np.abs(out) + (weight_eps + 2 * slack[..., None] + 2.0 ** -16) * spread
    worst = np.max(np.abs(y - out) - tol, initial=-1.0)
    assert worst <= 0, f"{what}: out off by {worst:.3e} over its bound"
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: empty rows"
    off = np.abs(got_lse[~empty] - lse[~empty]) - slack[~empty] - 2.0 ** -20 * (1 + np.abs(lse[~empty]))
    assert np.max(off, initial=-1.0) <= 0, f"{what}: lse off by {np.max(off):.3e} over its bound"


def rotate(x, pos, inv_freq, interleaved):
    """x [..., rot] in 64 bits; pos broadcasts against the pairs [..., rot / 2]."""
    a = pos * inv_freq
    c, s = np.cos(a), np.sin(a)
    y = x.copy()
    n = x.shape[-1] // 2
    i, j = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, n), slice(n, None))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y
