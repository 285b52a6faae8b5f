"""The paged key-value cache operators, case by case: appending a step's keys and values with the position rotation on
the way, attention of one new token per sequence over the pages, and attention of a prompt's (or a chunk's) new tokens.

A sequence's tokens 0 .. lens[b] - 1 live in pages of `page` tokens: token t is row t % page of page
table[b][t // page], in k and v of [pages][kv_heads][page][head_dim].  The cache is bf16, or E4M3 codes with one fp32
scale per token and kv head (amax / 448).  A step's new tokens are the last ones of their sequence: one each, or
starts[b] .. starts[b + 1] - 1 of the flat token list.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------------------- cases
def _case(op, heads, kv_heads, head_dim, page, fp8, batch, new, past, shape, **more):
    c = dict(op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, fp8=fp8, batch=batch, new=new,
             past=past, shape=shape)
    if op == "append":
        c.update(rot=head_dim, interleaved=False, axes=1)
    else:
        c.update(softcap=0.0, window=0, alibi=False, sinks=False)
        if op == "prefill":
            c.update(prefix=False)
    c.update(more)
    return c


def listed():
    """`new`: most new tokens of a sequence (0: a decode step, one each); `past`: most tokens cached before them."""
    return [
        # a decode step of one user: 6 KB of work, so what counts is latency
        dict(_case("append", 16, 4, 128, 16, False, 1, 0, 4096, 1), name="append_one"),
        # a decode step of a busy server, cache in 8 bits
        dict(_case("append", 64, 8, 64, 16, True, 64, 0, 8191, 2), name="append_step_fp8"),
        # prompts with images: positions of three axes (time, height, width), pairs shared out among them
        dict(_case("append", 28, 4, 128, 64, False, 4, 2500, 300, 3, axes=3), name="append_images"),
        # a long prompt, a quarter of each head rotated by adjacent pairs, cache in 8 bits
        dict(_case("append", 40, 10, 128, 32, True, 1, 8191, 0, 4, rot=32, interleaved=True), name="append_prompt_fp8"),
        # one user, early in the answer
        dict(_case("decode", 16, 4, 128, 16, False, 1, 0, 332, 5), name="decode_one_short"),
        # one user, a long context, layers with a sink logit per head
        dict(_case("decode", 64, 8, 64, 16, False, 1, 0, 32767, 6, sinks=True), name="decode_one_long"),
        # a ragged batch
        dict(_case("decode", 16, 4, 128, 64, False, 32, 0, 8191, 7), name="decode_batch"),
        # a large ragged batch with empty places, cache in 8 bits
        dict(_case("decode", 64, 8, 64, 16, True, 64, 0, 16383, 8, sinks=True), name="decode_batch_fp8"),
        # scores capped by a tanh and biased by distance, within a window
        dict(_case("decode", 40, 10, 128, 32, False, 12, 0, 12000, 9, softcap=50.0, window=4096, alibi=True),
             name="decode_capped"),
        # short turns of four conversations
        dict(_case("prefill", 16, 4, 128, 16, False, 4, 120, 1500, 10), name="prefill_short"),
        # one long prompt, its first part seen from everywhere
        dict(_case("prefill", 16, 4, 128, 64, False, 1, 8192, 0, 11, prefix=True), name="prefill_long"),
        # chunks of long prompts over what is cached of them, cache in 8 bits
        dict(_case("prefill", 64, 8, 64, 32, True, 3, 2048, 6000, 12, sinks=True), name="prefill_chunks_fp8"),
    ]


_LAYOUTS = ((16, 4, 128), (64, 8, 64), (40, 10, 128), (28, 4, 128), (8, 8, 64), (12, 1, 64))


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    heads, kv_heads, head_dim = rng.choice(_LAYOUTS)
    page, fp8, shape = rng.choice((16, 32, 64, 128)), rng.random() < 0.5, rng.randrange(1 << 30)
    op = rng.choice(("append", "decode", "prefill"))
    if op == "append":
        more = dict(rot=rng.choice((head_dim, head_dim // 2, 32)), interleaved=rng.random() < 0.5,
                    axes=rng.choice((1, 1, 3)))
        if rng.random() < 0.5:
            return _case(op, heads, kv_heads, head_dim, page, fp8, _spread(rng, 1, 256), 0, _spread(rng, 1, 8191),
                         shape, **more)
        new = _spread(rng, 2, 8191)
        most = max(1, min(8, 8191 * 60 * 128 // (new * (heads + 2 * kv_heads) * head_dim)))
        return _case(op, heads, kv_heads, head_dim, page, fp8, rng.randint(1, most), new, rng.randint(0, 2000), shape,
                     **more)
    more = dict(softcap=rng.choice((0.0, 0.0, 30.0)), window=rng.choice((0, 0, 128, 1000)), alibi=rng.random() < 0.25,
                sinks=rng.random() < 0.4)
    if op == "decode":
        past = _spread(rng, 1, 32767)
        most = max(1, min(128, 64 * 16384 * 8 * 64 // ((past + 1) * kv_heads * head_dim)))
        return _case(op, heads, kv_heads, head_dim, page, fp8, _spread(rng, 1, most), 0, past, shape, **more)
    new = _spread(rng, 2, 4096)
    room = 16 * 8192 * 8192 // (heads * new)  # keys of all sequences that the largest listed case's work allows
    past = rng.randint(0, max(0, min(16000, room - new)))
    batch = rng.randint(1, max(1, min(8, room // (new + past))))
    return _case(op, heads, kv_heads, head_dim, page, fp8, batch, new, past, shape, prefix=rng.random() < 0.25, **more)


def _sizes(case):
    """(new tokens, cached tokens with the new ones, prefix) of each sequence: the first is the longest, the others
    spread below it, and a large decode batch has empty places."""
    r = random.Random(case["shape"])
    new, lens, prefix = [], [], []
    for b in range(case["batch"]):
        n = 1 if case["new"] == 0 else case["new"] if b == 0 else r.randint(1, case["new"])
        past = case["past"] if b == 0 else r.randint(0, case["past"])
        full = n + past
        if case["new"] == 0 and b and case["batch"] >= 16 and r.random() < 0.05:
            full = 0
        new.append(n)
        lens.append(full)
        prefix.append(r.randint(0, full) if case.get("prefix") else 0)
    return new, lens, prefix


def _pairs(case):
    """(keys read, query-key pairs) over all sequences, of one head."""
    keys = pairs = 0
    w = case["window"]
    for n, full, pre in zip(*_sizes(case)):
        if full == 0:
            continue
        p = torch.arange(full - n, full, dtype=torch.int64)
        hi = torch.clamp(p + 1, min=pre)
        lo = torch.clamp(p + 1 - w, min=0) if w else torch.zeros_like(p)
        pairs += int((hi - lo).sum())
        keys += int(hi.max() - lo.min())
    return keys, pairs


def work(case):
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    new, lens, _ = _sizes(case)
    tokens = sum(n for n, full in zip(new, lens) if full)
    row = g * 2 * (d + 4 if case["fp8"] else 2 * d)  # a token's keys and values in the cache
    if case["op"] == "append":
        return {"bytes": tokens * ((h + 2 * g) * d * 2 + h * d * 2 + row + 4 * case["axes"]),
                "flops": tokens * (h + g) * case["rot"] * 3}
    keys, pairs = _pairs(case)
    return {"bytes": keys * row + tokens * h * (d * 4 + 4), "flops": pairs * h * d * 4}


# ------------------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, g, d, page, batch = case["heads"], case["kv_heads"], case["head_dim"], case["page"], case["batch"]
    new, lens, prefix = _sizes(case)
    tokens = sum(new)
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    pages = sum(need) + 3  # a pool is never full
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = table.cuda()
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table).contiguous()

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def cache():
        x = normal(pages, g, page, d)
        if not case["fp8"]:
            return x.bfloat16(), None
        scale = x.abs().amax(-1) / E4M3_MAX
        return (x / scale[..., None]).to(torch.float8_e4m3fn), scale

    (k, k_scales), (v, v_scales) = cache(), cache()
    s = dict(case=case, k=k, v=v, k_scales=k_scales, v_scales=v_scales, table=table, tokens=tokens, starts=None,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["new"]:
        s["starts"] = torch.tensor([0] + [sum(new[:i + 1]) for i in range(batch)], dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        pairs = case["rot"] // 2
        s["qkv"] = normal(tokens, (h + 2 * g) * d).bfloat16()
        s["inv_freq"] = 500000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
        s["q_out"] = torch.empty((tokens, h, d), dtype=torch.bfloat16, device="cuda")
        s["positions"] = s["pair_axis"] = None
        if case["axes"] == 3:  # a quarter of the pairs turn with time, the rest by height and width
            s["positions"] = torch.randint(0, 20000, (3, tokens), generator=gen, device="cuda", dtype=torch.int32)
            i = torch.arange(pairs, device="cuda")
            s["pair_axis"] = torch.where(i < pairs // 4, 0, torch.where(i < pairs // 4 + 3 * pairs // 8, 1, 2)).to(
                torch.uint8)
    else:
        s["q"] = normal(tokens, h, d).bfloat16()
        s["scale"] = 1.0 / math.sqrt(d)
        s["slopes"] = s["sinks"] = s["prefix"] = None
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, h + 1, dtype=torch.float32, device="cuda") / h)
        if case["sinks"]:
            s["sinks"] = normal(h)
        if case.get("prefix"):
            s["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty((tokens, h, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((tokens, h), dtype=torch.float32, device="cuda")
    if own:
        from bit_weight_only_mxfp4_gb300 import loader, thinmx
        s["kv"] = loader.paged_kv(k, v, table, s["lens"], k_scales, v_scales)
        if case["op"] == "append":
            s["turns"] = loader.rope_turns(s["inv_freq"])
        else:
            s["ws_bytes"] = thinmx.tt_paged_attention_workspace_bytes(h, g, d)
            s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "append":
        return _append(s)
    return _attention(s)


def _own(s):
    from bit_weight_only_mxfp4_gb300 import thinmx
    c = s["case"]
    h, g, d = c["heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "append":
        x, row = s["qkv"].data_ptr(), (h + 2 * g) * d
        thinmx.tt_paged_rope_append(s["kv"], x, x + 2 * h * d, x + 2 * (h + g) * d, row, row, s["tokens"], s["starts"],
                                    h, s["turns"], c["rot"], c["interleaved"], s["positions"], c["axes"],
                                    s["pair_axis"], s["q_out"])
        return _cache(s, s["q_out"])
    if c["op"] == "decode":
        thinmx.tt_paged_decode_attention(s["kv"], s["q"], h * d, h, s["scale"], c["softcap"], c["window"], s["slopes"],
                                         s["sinks"], s["out"], s["lse"], s["ws"], s["ws_bytes"])
    else:
        thinmx.tt_paged_prefill_attention(s["kv"], s["q"], h * d, s["starts"], s["tokens"], h, s["scale"],
                                          c["softcap"], c["window"], s["slopes"], s["sinks"], s["prefix"], s["out"],
                                          s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _cache(s, q):
    got = {"q": q, "k": s["k"], "v": s["v"]}
    if s["case"]["fp8"]:
        got.update(k_scales=s["k_scales"], v_scales=s["v_scales"])
    return got


def _places(s):
    """(sequence, place in it) of every new token."""
    t = torch.arange(s["tokens"], device="cuda")
    if s["starts"] is None:
        return t, s["lens"].long() - 1
    starts, lens = s["starts"].long(), s["lens"].long()
    seq = torch.searchsorted(starts, t, right=True) - 1
    return seq, lens[seq] - (starts[seq + 1] - t)


def _append(s):
    c = s["case"]
    h, g, d, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    seq, place = _places(s)
    here = place >= 0  # a sequence of length zero has no place for a token
    x = s["qkv"].float().reshape(s["tokens"], h + 2 * g, d)
    pos = place[None] if s["positions"] is None else s["positions"].long()
    axis = torch.zeros(c["rot"] // 2, dtype=torch.long, device="cuda") if s["pair_axis"] is None else s["pair_axis"].long()
    angle = pos[axis].t().double() * s["inv_freq"]  # in 64 bits: far positions
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    turned, kept = x[:, :h + g, :c["rot"]], x[:, :h + g, c["rot"]:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    qk = torch.cat((turned, kept), -1)
    q = torch.where(here[:, None, None], qk[:, :h], 0.0).bfloat16()
    where = s["table"][seq, place.clamp(min=0) // page].long()[here], slice(None), (place % page)[here]
    for name, y in (("k", qk[:, h:]), ("v", x[:, h + g:])):
        y = y[here]
        if c["fp8"]:
            scale = y.abs().amax(-1) / E4M3_MAX
            code = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0).clamp(-E4M3_MAX, E4M3_MAX)
            s[name].view(torch.uint8)[where] = code.to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scales"][where] = scale
        else:
            s[name][where] = y.bfloat16()
    return _cache(s, q)


def _gather(s, name):
    """Keys or values in 32 bits, [sequence][kv head][token][head_dim], and zero where there is no token."""
    x = s[name].float()
    if s["case"]["fp8"]:
        x = x * s[name + "_scales"][..., None]
    b, width = s["table"].shape
    _, g, page, d = x.shape
    x = x[s["table"].clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(b, g, width * page, d)
    inside = torch.arange(width * page, device="cuda") < s["lens"][:, None]
    return torch.where(inside[:, None, :, None], x, 0.0)


def _attention(s):
    c = s["case"]
    h, g, d, batch = c["heads"], c["kv_heads"], c["head_dim"], c["batch"]
    keys, values = _gather(s, "k"), _gather(s, "v")
    seq, place = _places(s)
    if s["starts"] is None:
        most, row = 1, torch.zeros_like(seq)
    else:
        most, row = c["new"], torch.arange(s["tokens"], device="cuda") - s["starts"].long()[seq]
    q = torch.zeros((batch, most, g, h // g, d), device="cuda")
    p = torch.full((batch, most), -1, dtype=torch.long, device="cuda")
    q[seq, row] = s["q"].float().reshape(-1, g, h // g, d)
    p[seq, row] = place
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, g, h // g * most, d)
    score = (q @ keys.transpose(-1, -2)).reshape(batch, h, most, -1) * s["scale"]
    if c["softcap"]:
        score = torch.tanh(score / c["softcap"]) * c["softcap"]
    j = torch.arange(score.shape[-1], device="cuda")
    far = j - p[..., None]
    if c["alibi"]:
        score = score + s["slopes"][:, None, None] * far[:, None]
    seen = far <= 0
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][:, None, None])
    seen = seen & (j < s["lens"][:, None, None])
    if c["window"]:
        seen = seen & (far > -c["window"])
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    if c["sinks"]:
        top = torch.maximum(top, s["sinks"][:, None, None])
    top = torch.where(torch.isinf(top), 0.0, top)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    if c["sinks"]:
        total = total + torch.exp(s["sinks"][:, None, None] - top)
    out = (weight.reshape(batch, g, h // g * most, -1) @ values).reshape(batch, h, most, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.log(total[..., 0]) + top[..., 0]
    return {"out": out[seq, :, row].bfloat16(), "lse": lse[seq, :, row]}


# ---------------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    c = s["case"]
    h, g, d, page, rot = c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["rot"]
    new, lens, _ = _sizes(c)
    x = s["qkv"].double().view(s["tokens"], h + 2 * g, d)
    got = {n: s[n].double() for n in (("k", "v", "k_scales", "v_scales") if c["fp8"] else ("k", "v"))}
    q = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    first = torch.arange(rot // 2, device="cuda")
    first, step = (2 * first, 1) if c["interleaved"] else (first, rot // 2)
    t = 0
    for b, (n, full) in enumerate(zip(new, lens)):
        if full:
            place = torch.arange(full - n, full, device="cuda")
            if s["positions"] is None:
                pos = place.double()[:, None].expand(n, rot // 2)
            else:
                pos = s["positions"][:, t:t + n].double()[s["pair_axis"].long()].t()
            turn = torch.polar(torch.ones_like(pos), pos * s["inv_freq"])[:, None]
            y = x[t:t + n].clone()
            z = torch.complex(y[:, :h + g, first], y[:, :h + g, first + step]) * turn
            y[:, :h + g, first], y[:, :h + g, first + step] = z.real, z.imag
            q[t:t + n] = y[:, :h]
            at, row = s["table"][b].long()[place // page], place % page
            for name, part in (("k", y[:, h:h + g]), ("v", y[:, h + g:])):
                if c["fp8"]:
                    scale = part.abs().amax(-1) / E4M3_MAX
                    got[name + "_scales"][at, :, row] = scale
                    part = torch.where(scale[..., None] > 0, part / scale[..., None], 0.0)
                got[name][at, :, row] = part
        t += n
    return {"q": q, **got}


def _exact_attention(s):
    c = s["case"]
    h, g, d, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    group = h // g
    new, lens, prefix = _sizes(c)
    out = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], h), -math.inf, dtype=torch.float64, device="cuda")
    sinks = None if s["sinks"] is None else s["sinks"].double()
    t = 0
    for b, (n, full, pre) in enumerate(zip(new, lens, prefix)):
        if sinks is not None:
            lse[t:t + n] = sinks
        if full:
            j = torch.arange(full, device="cuda")
            p = torch.arange(full - n, full, device="cuda")[:, None]
            hide = (j > p) & (j >= pre)
            if c["window"]:
                hide |= j <= p - c["window"]
            at, row = s["table"][b].long()[j // page], j % page
            for i in range(g):
                k, v = s["k"][at, i, row].double(), s["v"][at, i, row].double()
                if c["fp8"]:
                    k, v = k * s["k_scales"][at, i, row].double()[:, None], v * s["v_scales"][at, i, row].double()[:, None]
                for e in range(i * group, (i + 1) * group):
                    z = s["q"][t:t + n, e].double() @ k.t() * s["scale"]
                    if c["softcap"]:
                        z = c["softcap"] * torch.tanh(z / c["softcap"])
                    if c["alibi"]:
                        z += s["slopes"][e].double() * (j - p)
                    z.masked_fill_(hide, -math.inf)
                    all_z = torch.logsumexp(z, 1)
                    if sinks is not None:
                        all_z = torch.logaddexp(all_z, sinks[e])
                    lse[t:t + n, e] = all_z
                    out[t:t + n, e] = torch.exp(z - all_z[:, None]) @ v
        t += n
    return {"out": out, "lse": lse}
