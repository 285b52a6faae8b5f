"""Drafted trees and branching sequences over the paged key-value cache, case by case: attention of a tree of drafted
tokens, log probabilities of given tokens with entropy and top alternatives, the bookkeeping of a drafted step (the
tree's masks, the walk that accepts drafts, the accepted rows moved together), and the pages of sequences that branch
and of pools that have become scattered.

The cache is that of the paged operators: token t of sequence b is row t % page of page table[b][t // page], in k and v of
[layers][pages][kv_heads][page][head_dim], bf16, or E4M3 codes with one fp32 scale per token and kv head.  A step's new
tokens are the last ones of their sequence: starts[b] .. starts[b + 1] - 1 of the flat token list.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
WORDS = 2  # words of a mask row: trees of up to 64 tokens


# ------------------------------------------------------------------------------------------------------------- cases
def _tree(heads, kv_heads, head_dim, page, fp8, batch, new, past, shape, **more):
    return dict(dict(op="tree", heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, fp8=fp8, batch=batch,
                     new=new, past=past, shape=shape, softcap=0.0, window=0, alibi=False, sinks=False), **more)


def _logprobs(rows, vocab, bf16, top, **more):
    return dict(dict(op="logprobs", rows=rows, vocab=vocab, bf16=bf16, top=top, pad=0, scale=1.0), **more)


def _pool(op, layers, kv_heads, head_dim, page, fp8, batch, new, past, shape, **more):
    return dict(dict(op=op, layers=layers, kv_heads=kv_heads, head_dim=head_dim, page=page, fp8=fp8, batch=batch, new=new,
                     past=past, shape=shape), **more)


def listed():
    """`new`: most new tokens of a sequence; `past`: most tokens cached before them."""
    return [
        # one user, early in the answer, a few drafts
        dict(_tree(16, 4, 128, 16, False, 1, 8, 332, 1), name="tree_one_short"),
        # one user, a long context, a large tree, layers with a sink logit per head
        dict(_tree(64, 8, 64, 16, False, 1, 64, 32767, 2, sinks=True), name="tree_one_long"),
        # a ragged batch of conversations
        dict(_tree(16, 4, 128, 64, False, 32, 16, 8191, 3), name="tree_batch"),
        # a large ragged batch with empty places, cache in 8 bits
        dict(_tree(64, 8, 64, 16, True, 48, 24, 12000, 4, sinks=True), name="tree_batch_fp8"),
        # one sampled token with its alternatives
        dict(_logprobs(1, 128256, True, 20), name="logprobs_one"),
        # the nodes of a batch's trees, the best token of each, at a temperature
        dict(_logprobs(512, 201088, True, 1, scale=1.25), name="logprobs_trees"),
        # a prompt's tokens scored, logits in 32 bits
        dict(_logprobs(2047, 100352, False, 5), name="logprobs_prompt"),
        # a drafted step of one user around the model: what counts is latency
        dict(_pool("step", 24, 4, 128, 16, False, 1, 8, 332, 8), name="step_one"),
        # a drafted step of a busy server, cache in 8 bits
        dict(_pool("step", 24, 8, 64, 16, True, 64, 32, 500, 9), name="step_batch_fp8"),
        # one user's beams: two of four go on twice
        dict(_pool("fork", 36, 4, 128, 16, False, 4, 0, 1000, 10), name="fork_beams"),
        # beams of a busy server, cache in 8 bits, large pages
        dict(_pool("fork", 24, 8, 64, 64, True, 128, 0, 1000, 11), name="fork_batch_fp8"),
        # a pool after most of its sequences have ended
        dict(_pool("compact", 24, 4, 128, 16, False, 48, 0, 1500, 12), name="compact_pool"),
    ]


_LAYOUTS = ((16, 4, 128), (64, 8, 64), (40, 10, 128), (28, 4, 128), (8, 8, 64), (12, 1, 64))


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "logprobs", "step", "fork", "compact"))
    if op == "logprobs":
        vocab = rng.choice((100352, 128256, 201088, _spread(rng, 1000, 260000)))
        rows = _spread(rng, 1, max(1, min(4096, 2047 * 100352 // vocab)))
        return _logprobs(rows, vocab, rng.random() < 0.7, rng.choice((0, 1, 5, 20)), pad=rng.choice((0, 0, 1, 56)),
                         scale=rng.choice((1.0, 0.7, 1.6)))
    heads, kv_heads, head_dim = rng.choice(_LAYOUTS)
    page, fp8, shape = rng.choice((16, 32, 64, 128)), rng.random() < 0.5, rng.randrange(1 << 30)
    if op == "tree":
        new, past = _spread(rng, 1, 64), _spread(rng, 1, 32767)
        most = 48 * 24 * 12000 * 64 * 64 // (new * (past + new) * heads * head_dim)
        most = min(most, 48 * 12000 * 8 * 64 // ((past + new) * kv_heads * head_dim))
        return _tree(heads, kv_heads, head_dim, page, fp8, _spread(rng, 1, max(1, min(64, most))), new, past, shape,
                     softcap=rng.choice((0.0, 0.0, 30.0)), window=rng.choice((0, 0, 128, 1000)),
                     alibi=rng.random() < 0.25, sinks=rng.random() < 0.4)
    layers, past = rng.choice((1, 24, 36)), _spread(rng, 1, 1500)
    most = 48 * 1500 * 24 * 4 * 128 // ((past + page) * layers * kv_heads * head_dim)
    batch = _spread(rng, 1 if op == "step" else 2, max(2, min(128, most)))
    return _pool(op, layers, kv_heads, head_dim, page, fp8, batch, _spread(rng, 1, 64) if op == "step" else 0, past, shape)


def _sizes(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the first is the longest, the others spread below
    it, and a large batch has empty places."""
    r = random.Random(case["shape"])
    new, lens = [], []
    for b in range(case["batch"]):
        n = case["new"] if b == 0 else r.randint(min(1, case["new"]), case["new"])
        past = case["past"] if b == 0 else r.randint(0, case["past"])
        if b and case["batch"] >= 16 and r.random() < 0.05:
            n = past = 0
        new.append(n)
        lens.append(n + past)
    return new, lens


def _parents(case):
    """The trees of a step, flat: a token's parent among its sequence's new tokens, -1 for the first one."""
    r = random.Random(case["shape"] + 1)
    return [[-1] + [r.randint((i - 1) // 4, i - 1) for i in range(1, n)] if n else [] for n in _sizes(case)[0]]


def _accepted(case):
    """The nodes that a step accepts, for each sequence: a way down from the first one.  It ends before the rows that it
    fills would be rows that it moves, so that a pass finds its rows as the one before did."""
    r = random.Random(case["shape"] + 2)
    ways = []
    for parents in _parents(case):
        way = [0] if parents else []
        while way and r.random() < 0.9:
            below = [i for i, p in enumerate(parents) if p == way[-1]]
            if not below:
                break
            way.append(r.choice(below))
        while any(i != j and i < len(way) for j, i in enumerate(way)):
            way.pop()
        ways.append(way)
    return ways


def _from(case):
    """Beams: every second sequence goes on, the others become copies of one of those or end."""
    r = random.Random(case["shape"] + 3)
    batch = case["batch"]
    return [b if b % 2 == 0 else -1 if r.random() < 0.1 else 2 * r.randrange((batch + 1) // 2) for b in range(batch)]


def _table(case):
    """A table of pages dealt out at random, and the number of pages: a pool has some left (and a scattered one, most)."""
    r = random.Random(case["shape"] + 4)
    need = [-(-n // case["page"]) for n in _sizes(case)[1]]
    width = max(1, max(need)) + 1
    pages = sum(need) * (3 if case["op"] == "compact" else 1) + 2 * case["batch"] + 3
    order = r.sample(range(pages), sum(need))
    table = []
    for n in need:
        table.append([order.pop() for _ in range(n)] + [-1] * (width - n))
    return table, pages


def _row_bytes(case):
    """A token's keys and values in one layer's cache."""
    return case["kv_heads"] * 2 * (case["head_dim"] + 4 if case["fp8"] else 2 * case["head_dim"])


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["bf16"] else 4) + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
    new, lens = _sizes(case)
    tokens, page, row = sum(new), case["page"], _row_bytes(case)
    if case["op"] == "tree":
        h, d, w = case["heads"], case["head_dim"], case["window"]
        keys = pairs = 0
        for parents, full in zip(_parents(case), lens):
            past, depth = full - len(parents), []
            for p in parents:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            far = min(depth, default=0)
            keys += len(parents) + (min(past, max(0, w - 1 - far)) if w else past) if parents else 0
            pairs += sum((min(past, max(0, w - 1 - e)) + min(e + 1, w) if w else past + e + 1) for e in depth)
        return {"bytes": keys * row + tokens * (h * (d * 4 + 4) + 4 * WORDS), "flops": pairs * h * d * 4}
    if case["op"] == "step":
        moved = sum(i != j for way in _accepted(case) for j, i in enumerate(way))
        return {"bytes": moved * row * case["layers"] * 2 + tokens * 4 * (4 + WORDS) + case["batch"] * 4 * (4 + case["new"]),
                "flops": 0}
    table, pages = _table(case)
    meta = 2 * 4 * case["batch"] * (len(table[0]) + 1)
    if case["op"] == "fork":
        rows = sum(lens[a] % page for b, a in enumerate(_from(case)) if a >= 0 and a != b)
        return {"bytes": rows * row * case["layers"] * 2 + meta, "flops": 0}
    used = sum(-(-n // page) for n in lens)
    moved = sum(p >= used for line in table for p in line)
    return {"bytes": moved * page * row * case["layers"] * 2 + meta, "flops": 0}


# ------------------------------------------------------------------------------------------------------------ inputs
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, gen)
    g, d, page, batch, layers = case["kv_heads"], case["head_dim"], case["page"], case["batch"], case.get("layers", 1)
    new, lens = _sizes(case)
    tokens = sum(new)
    table, pages = _table(case)
    # the pool's pages in another order for every seed; the scattered pool's stay: which ones move is the case's
    table = _ints(table)
    if case["op"] != "compact":
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.where(table >= 0, order[table.clamp(min=0).long()], table).contiguous()
    kind = torch.float8_e4m3fn if case["fp8"] else torch.bfloat16
    s = dict(case=case, table=table, tokens=tokens, pages=pages, k_scales=None, v_scales=None, lens=_ints(lens),
             starts=_ints([sum(new[:b]) for b in range(batch + 1)]))
    for name in ("k", "v"):
        s[name] = torch.empty((layers, pages, g, page, d), dtype=kind, device="cuda")
        if case["fp8"]:
            s[name + "_scales"] = torch.empty((layers, pages, g, page), device="cuda")
        for i in range(layers):
            x = torch.randn((pages, g, page, d), generator=gen, device="cuda")
            if case["fp8"]:
                s[name + "_scales"][i] = x.abs().amax(-1) / E4M3_MAX
                x = x / s[name + "_scales"][i][..., None]
            s[name][i] = x.to(kind)
    if case["op"] == "tree":
        _prepare_tree(s, gen)
    elif case["op"] == "step":
        _prepare_step(s, gen)
    else:
        s["from"] = _ints(_from(case))
        s["table_out"], s["lens_out"] = torch.empty_like(table), torch.empty_like(s["lens"])
        s["left"] = _ints([0])
    if own:
        _own_prepare(s)
    return s


def _prepare_tree(s, gen):
    c = s["case"]
    h, d = c["heads"], c["head_dim"]
    masks = []
    for parents in _parents(c):
        rows = []
        for i, p in enumerate(parents):
            rows.append((rows[p] if p >= 0 else 0) | 1 << i)
        masks += [[(m >> 32 * w & 0xffffffff) - (m >> 32 * w + 31 & 1) * (1 << 32) for w in range(WORDS)] for m in rows]
    s["masks"] = _ints(masks)
    s["q"] = torch.randn((s["tokens"], h, d), generator=gen, device="cuda").bfloat16()
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = s["sinks"] = None
    if c["alibi"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, h + 1, dtype=torch.float32, device="cuda") / h)
    if c["sinks"]:
        s["sinks"] = torch.randn(h, generator=gen, device="cuda")
    s["out"] = torch.empty((s["tokens"], h, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((s["tokens"], h), dtype=torch.float32, device="cuda")


def _prepare_step(s, gen):
    c = s["case"]
    tokens, batch = s["tokens"], c["batch"]
    s["parents"] = _ints([p for parents in _parents(c) for p in parents])
    drafts = torch.randperm(100000, generator=gen, device="cuda")[:tokens].to(torch.int32)
    chosen = torch.randint(100000, 128000, (tokens,), generator=gen, device="cuda", dtype=torch.int32)  # no draft's
    at, to, first = [], [], 0
    for parents, way in zip(_parents(c), _accepted(c)):
        at += [first + i for i in way[:-1]]
        to += [first + i for i in way[1:]]
        first += len(parents)
    chosen[_ints(at).long()] = drafts[_ints(to).long()]
    s["drafts"], s["chosen"] = drafts, chosen
    s["masks"], s["positions"] = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((tokens, WORDS), (tokens,)))
    s["path"] = torch.empty((batch, c["new"]), dtype=torch.int32, device="cuda")
    s["counts"], s["next"], s["lens_out"] = (torch.empty_like(s["lens"]) for _ in range(3))


def _prepare_logprobs(case, gen):
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    stride = vocab + case["pad"]
    logits = torch.empty((rows, stride), dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
    for i in range(0, rows, 256):
        x = torch.randn((min(256, rows - i), stride), generator=gen, device="cuda") * 2.5
        logits[i:i + 256] = x + 4.0 * (x > 9.0) * x.abs().sqrt()  # a few that stand out
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    if rows > 1:
        targets[torch.rand(rows, generator=gen, device="cuda") < 0.02] = -1  # rows that are padding
    s = dict(case=case, logits=logits, targets=targets)
    s["logp"], s["entropy"] = (torch.empty(rows, device="cuda") for _ in range(2))
    s["top_ids"] = torch.empty((rows, top), dtype=torch.int32, device="cuda")
    s["top_logp"] = torch.empty((rows, top), device="cuda")
    if own:
        from bit_weight_only_mxfp4_gb300 import thinmx
        s["ws_bytes"] = thinmx.tt_token_logprobs_workspace_bytes(rows, vocab, top)
        s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    return s


def _own_prepare(s):
    from bit_weight_only_mxfp4_gb300 import loader, thinmx
    c = s["case"]

    def layer(i, table, lens):
        scales = (s["k_scales"][i], s["v_scales"][i]) if c["fp8"] else (None, None)
        return loader.paged_kv(s["k"][i], s["v"][i], table, lens, *scales)

    kvs = [layer(i, s["table"], s["lens"]) for i in range(len(s["k"]))]
    s["kv"], s["layers"] = kvs[0], loader.paged_layers(kvs)
    if c["op"] == "tree":
        s["ws_bytes"] = thinmx.tt_paged_tree_workspace_bytes(c["heads"], c["kv_heads"], c["head_dim"])
    elif c["op"] in ("fork", "compact"):
        s["kv_out"] = layer(0, s["table_out"], s["lens_out"])
        s["ws_bytes"] = thinmx.tt_paged_pages_workspace_bytes(s["kv"])
    else:
        return
    s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    return {"tree": _attention, "logprobs": _log_probabilities, "step": _step, "fork": _fork, "compact": _compact}[op](s)


def _own(s):
    from bit_weight_only_mxfp4_gb300 import thinmx
    c = s["case"]
    if c["op"] == "tree":
        h, d = c["heads"], c["head_dim"]
        thinmx.tt_paged_tree_attention(s["kv"], s["q"], h * d, s["starts"], s["tokens"], h, s["scale"], c["softcap"],
                                       c["window"], s["slopes"], s["sinks"], s["masks"], WORDS, s["out"], s["lse"],
                                       s["ws"], s["ws_bytes"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "logprobs":
        kind = thinmx.TT_LOGITS_BF16 if c["bf16"] else thinmx.TT_LOGITS_F32
        thinmx.tt_token_logprobs(s["logits"], kind, c["rows"], c["vocab"], c["vocab"] + c["pad"], c["scale"],
                                 s["targets"], c["top"], s["logp"], s["entropy"], s["top_ids"], s["top_logp"], s["ws"],
                                 s["ws_bytes"])
        return {n: s[n] for n in ("logp", "entropy", "top_ids", "top_logp")}
    if c["op"] == "step":
        thinmx.tt_draft_tree(s["parents"], s["starts"], s["lens"], c["batch"], s["tokens"], WORDS, s["masks"],
                             s["positions"])
        thinmx.tt_draft_accept(s["parents"], s["drafts"], s["chosen"], s["starts"], c["batch"], s["tokens"], c["new"],
                               s["path"], s["counts"], s["next"])
        thinmx.tt_paged_keep(s["layers"], c["layers"], s["starts"], s["path"], c["new"], s["counts"], s["lens_out"])
        return _pool_outputs(s, *(s[n] for n in ("masks", "positions", "path", "counts", "next", "lens_out")))
    if c["op"] == "fork":  # then a page for the next token, where one is wanted
        thinmx.tt_paged_fork(s["layers"], c["layers"], s["from"], None, s["table_out"], s["lens_out"], s["left"], s["ws"],
                             s["ws_bytes"])
        thinmx.tt_paged_resize(s["kv_out"], s["lens_out"] + 1, None, s["table_out"], s["lens_out"], s["left"], s["ws"],
                               s["ws_bytes"])
    else:
        thinmx.tt_paged_compact(s["layers"], c["layers"], None, s["table_out"], s["left"], s["ws"], s["ws_bytes"])
        return _pool_outputs(s, s["table_out"], s["left"])
    return _pool_outputs(s, s["table_out"], s["lens_out"], s["left"])


def _pool_outputs(s, *more):
    names = ("k", "v", "k_scales", "v_scales") if s["case"]["fp8"] else ("k", "v")
    return dict({n: s[n] for n in names}, more=list(more))


def _caches(s):
    return [s[n] for n in (("k", "v", "k_scales", "v_scales") if s["case"]["fp8"] else ("k", "v"))]


def _bits(x):
    """8-bit values are moved by their codes."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _places(s):
    """(sequence, number among its new tokens, tokens cached before them) of every new token."""
    t = torch.arange(s["tokens"], device="cuda")
    starts, lens = s["starts"].long(), s["lens"].long()
    seq = torch.searchsorted(starts, t, right=True) - 1
    return seq, t - starts[seq], lens[seq] - (starts[seq + 1] - starts[seq])


def _gather(s, name):
    """Keys or values in 32 bits, [sequence][kv head][token][head_dim], and zero where there is no token."""
    x = s[name][0].float()
    if s["case"]["fp8"]:
        x = x * s[name + "_scales"][0][..., None]
    b, width = s["table"].shape
    _, g, page, d = x.shape
    x = x[s["table"].clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(b, g, width * page, d)
    inside = torch.arange(width * page, device="cuda") < s["lens"][:, None]
    return torch.where(inside[:, None, :, None], x, 0.0)


def _attention(s):
    c = s["case"]
    h, g, d, batch, most = c["heads"], c["kv_heads"], c["head_dim"], c["batch"], c["new"]
    keys, values = _gather(s, "k"), _gather(s, "v")
    seq, row, before = _places(s)
    bit = torch.arange(most, device="cuda")
    sees = (s["masks"].long()[:, bit // 32] >> bit % 32 & 1).bool()  # [token][new token of its sequence]
    depth = (sees.sum(1) - 1).clamp(min=0)
    width = keys.shape[2]

    def spread(x, fill):
        y = torch.full((batch, most) + x.shape[1:], fill, dtype=x.dtype, device="cuda")
        y[seq, row] = x
        return y

    q = spread(s["q"].float().reshape(-1, g, h // g, d), 0.0).permute(0, 2, 3, 1, 4).reshape(batch, g, h // g * most, d)
    score = (q @ keys.transpose(-1, -2)).reshape(batch, h, most, width) * s["scale"]
    if c["softcap"]:
        score = torch.tanh(score / c["softcap"]) * c["softcap"]
    # each key's place in its text: a new token's by its depth in the tree
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    j = torch.arange(width, device="cuda")
    drafted = j - first[:, None]
    new = (drafted >= 0) & (drafted < most)
    deep = torch.gather(spread(depth, 0), 1, drafted.clamp(0, most - 1))
    place = torch.where(new, first[:, None] + deep, j)
    far = place[:, None] - (first[:, None] + spread(depth, 0))[..., None]
    inside = torch.gather(spread(sees, False), 2, drafted.clamp(0, most - 1)[:, None].expand(batch, most, width))
    seen = (drafted < 0)[:, None] | (inside & new[:, None])
    seen = seen & (j < s["lens"][:, None])[:, None]
    if c["window"]:
        seen = seen & (far > -c["window"])
    if c["alibi"]:
        score = score + s["slopes"][:, None, None] * far[:, None]
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


def _log_probabilities(s):
    c = s["case"]
    logits = s["logits"][:, :c["vocab"]].float()
    x = logits * c["scale"]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total) + top
    entropy = (torch.log(total) - (e * (x - top)).sum(1, keepdim=True) / total)[:, 0]
    at = s["targets"].long()
    logp = torch.where(at >= 0, torch.gather(x, 1, at.clamp(min=0)[:, None])[:, 0] - lse[:, 0], 0.0)
    ids, left = [], logits.clone()
    i = torch.arange(c["vocab"], device="cuda")
    for _ in range(c["top"]):  # the largest, and of equal ones the first
        best = torch.where(left == left.amax(1, keepdim=True), i, c["vocab"]).amin(1)
        ids.append(best)
        left.scatter_(1, best[:, None], -math.inf)
    ids = torch.stack(ids, 1) if ids else torch.empty((c["rows"], 0), dtype=torch.long, device="cuda")
    return {"logp": logp, "entropy": entropy, "top_ids": ids.int(), "top_logp": torch.gather(x, 1, ids) - lse}


def _step(s):
    c = s["case"]
    batch, most, page = c["batch"], c["new"], c["page"]
    seq, row, before = _places(s)
    starts, parents = s["starts"].long(), s["parents"].long()
    # the tokens above each token, by following the parents
    sees = torch.zeros((s["tokens"], WORDS * 32), dtype=torch.bool, device="cuda")
    at = row
    for _ in range(most):
        sees |= (torch.arange(WORDS * 32, device="cuda") == at[:, None]) & (at >= 0)[:, None]
        at = torch.where(at >= 0, parents[starts[seq] + at.clamp(min=0)], at)
    bits = sees.reshape(-1, WORDS, 32).long() << torch.arange(32, device="cuda")
    masks = bits.sum(-1)
    masks = torch.where(masks >= 1 << 31, masks - (1 << 32), masks).int()
    positions = (before + sees.sum(1) - 1).int()
    # the way down: from a node to its first child that has the chosen token
    above = starts[seq] + parents.clamp(min=0)
    right = (parents >= 0) & (s["drafts"] == s["chosen"][above])
    follow = torch.full((s["tokens"] + 1,), most, dtype=torch.long, device="cuda")
    follow = follow.scatter_reduce(0, torch.where(right, above, s["tokens"]), row, "amin")
    alive = starts[1:] > starts[:-1]
    here = torch.where(alive, 0, most)
    path, nxt = [], torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    for _ in range(most):
        on = here < most
        path.append(torch.where(on, here, -1))
        flat = torch.where(on, starts[:-1] + here, 0)
        nxt = torch.where(on, s["chosen"][flat], nxt)
        here = torch.where(on, follow[flat], most)
    path = torch.stack(path, 1)
    counts = (path >= 0).sum(1)
    first = s["lens"].long() - (starts[1:] - starts[:-1])
    lens = first + counts
    # the accepted rows, moved together
    b, j = torch.nonzero((path >= 0) & (path != torch.arange(most, device="cuda")), as_tuple=True)
    src, dst = first[b] + path[b, j], first[b] + j
    table = s["table"].long()
    for x in _caches(s):
        x = _bits(x)
        x[:, table[b, dst // page], :, dst % page] = x[:, table[b, src // page], :, src % page]
    return _pool_outputs(s, masks, positions, path.int(), counts.int(), nxt, lens.int())


def _take(table, want, pages):
    """(table with the lowest pages that it does not name in the places `want`, in order; pages left, or minus those
    that were missing)."""
    used = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(table >= 0, table, pages).long().flatten()] = True
    free = torch.nonzero(~used[:pages])[:, 0].int()
    nth = (torch.cumsum(want.flatten(), 0) - 1).reshape(want.shape)
    got = torch.cat((free, torch.full((want.numel(),), -1, dtype=torch.int32, device="cuda")))[nth.clamp(min=0)]
    return torch.where(want, got, table), (len(free) - want.sum()).reshape(1).int()


def _fork(s):
    c = s["case"]
    page, batch = c["page"], c["batch"]
    src, b = s["from"].long(), torch.arange(c["batch"], device="cuda")
    alive, stays = src >= 0, src == torch.arange(batch, device="cuda")
    src = src.clamp(min=0)
    lens = torch.where(alive, s["lens"][src], 0)
    e = torch.arange(s["table"].shape[1], device="cuda")
    keep = alive[:, None] & (stays[:, None] | (e < (-(-lens // page))[:, None]))
    table = torch.where(keep, s["table"][src], -1)
    # a part page is copied, but for the first sequence that goes on from one which does not stay itself
    same = (s["from"][:, None] == s["from"]) & (b < b[:, None])
    takes = ~same.any(1) & ~stays[src]
    copies = alive & ~stays & ~takes & (lens % page > 0)
    tail = copies[:, None] & (e == (lens // page)[:, None])
    table, left = _take(torch.where(tail, -1, table), tail, s["pages"])
    i = torch.nonzero(copies)[:, 0]
    at = (lens[i] // page)[:, None]
    old, new = (torch.gather(t[r].long(), 1, at.long())[:, 0] for t, r in ((s["table"], src[i]), (table, i)))
    rows = torch.arange(page, device="cuda") < (lens[i] % page)[:, None]
    for x in _caches(s):
        x = _bits(x)
        part = rows.reshape(rows.shape[0], 1, page, *([1] if x.dim() == 5 else []))
        for y in x:
            y[new] = torch.where(part, y[old], y[new])
    # then a page for the next token
    used, need = -(-lens // page), -(-(lens + 1) // page)
    want = (table < 0) & (e >= used[:, None]) & (e < need[:, None])
    table, left = _take(torch.where(e < need[:, None], table, -1), want, s["pages"])
    return _pool_outputs(s, table, lens, left)


def _compact(s):
    pages, table = s["pages"], s["table"]
    used = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(table >= 0, table, pages).long().flatten()] = True
    used = used[:pages]
    count = used.sum()
    low = torch.arange(pages, device="cuda") < count
    src, dst = torch.nonzero(used & ~low)[:, 0], torch.nonzero(~used & low)[:, 0]
    for x in _caches(s):
        for y in _bits(x):
            y[dst] = y[src]
    to = torch.arange(pages, device="cuda")
    to[src] = dst
    return _pool_outputs(s, torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table), count.reshape(1).int())


# ---------------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "logprobs": _exact_logprobs, "step": _exact_step, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](s)


def _exact_tree(s):
    c = s["case"]
    h, g, d, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    out = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], h), -math.inf, dtype=torch.float64, device="cuda")
    sinks = None if s["sinks"] is None else s["sinks"].double()
    t = 0
    for b, (parents, full) in enumerate(zip(_parents(c), _sizes(c)[1])):
        n = len(parents)
        if n == 0:
            continue
        past = full - n
        above = torch.zeros((n, n), dtype=torch.bool)
        for i, p in enumerate(parents):
            if p >= 0:
                above[i] = above[p]
            above[i, i] = True
        above = above.cuda()
        deep = above.sum(1) - 1
        place = torch.cat((torch.arange(past, device="cuda"), past + deep))
        gap = (past + deep)[:, None] - place
        hide = torch.cat((torch.zeros((n, past), dtype=torch.bool, device="cuda"), ~above), 1)
        if c["window"]:
            hide |= gap >= c["window"]
        j = torch.arange(full, device="cuda")
        at, row = s["table"][b].long()[j // page], j % page
        for i in range(g):
            k, v = s["k"][0, at, i, row].double(), s["v"][0, at, i, row].double()
            if c["fp8"]:
                k *= s["k_scales"][0, at, i, row].double()[:, None]
                v *= s["v_scales"][0, at, i, row].double()[:, None]
            for e in range(i * (h // g), (i + 1) * (h // g)):
                z = s["q"][t:t + n, e].double() @ k.t() * s["scale"]
                if c["softcap"]:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                if c["alibi"]:
                    z -= s["slopes"][e].double() * gap
                z.masked_fill_(hide, -math.inf)
                total = torch.logsumexp(z, 1)
                if sinks is not None:
                    total = torch.logaddexp(total, sinks[e])
                lse[t:t + n, e] = total
                out[t:t + n, e] = torch.exp(z - total[:, None]) @ v
        t += n
    return {"out": out, "lse": lse}


def _exact_logprobs(s):
    c = s["case"]
    logp, entropy, ids, tops = [], [], [], []
    for i in range(0, c["rows"], 256):
        x = s["logits"][i:i + 256, :c["vocab"]].double()
        order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :c["top"]]
        lp = torch.log_softmax(x * c["scale"], 1)
        at = s["targets"][i:i + 256].long()
        logp.append(torch.where(at < 0, 0.0, lp[torch.arange(len(x), device="cuda"), at.clamp(min=0)]))
        entropy.append(-(lp.exp() * lp).sum(1))
        ids.append(order.int())
        tops.append(lp.gather(1, order))
    return {n: torch.cat(x) for n, x in (("logp", logp), ("entropy", entropy), ("top_ids", ids), ("top_logp", tops))}


def _exact_step(s):
    c = s["case"]
    page = c["page"]
    masks, positions, path, counts, nxt, lens, t = [], [], [], [], [], [], 0
    src, dst = [], []
    table, chosen = s["table"].tolist(), s["chosen"].tolist()
    for b, (parents, way, full) in enumerate(zip(_parents(c), _accepted(c), _sizes(c)[1])):
        past, up = full - len(parents), []
        for i, p in enumerate(parents):
            up.append({i} | (up[p] if p >= 0 else set()))
            word = [sum(1 << e % 32 for e in up[i] if e // 32 == w) for w in range(WORDS)]
            masks.append([w - (1 << 32) if w >= 1 << 31 else w for w in word])
            positions.append(past + len(up[i]) - 1)
        path.append(way + [-1] * (c["new"] - len(way)))
        counts.append(len(way))
        nxt.append(chosen[t + way[-1]] if way else -1)
        lens.append(past + len(way))
        src += [(table[b][(past + i) // page], (past + i) % page) for i in way]
        dst += [(table[b][(past + j) // page], (past + j) % page) for j in range(len(way))]
        t += len(parents)
    old = [y.clone() for y in map(_bits, _caches(s))]
    (sp, sr), (dp, dr) = (map(torch.tensor, zip(*x)) for x in (src, dst))
    for x, y in zip(map(_bits, _caches(s)), old):
        x[:, dp, :, dr] = y[:, sp, :, sr]
    return _pool_outputs(s, *map(_ints, (masks, positions, path, counts, nxt, lens)))


def _exact_fork(s):
    c = s["case"]
    page, batch = c["page"], c["batch"]
    come, old, lens0 = _from(c), s["table"].tolist(), _sizes(c)[1]
    width = len(old[0])
    table, lens, copies, owner = [], [], [], {b: b for b in range(batch) if come[b] == b}
    for b, a in enumerate(come):
        n = lens0[a] if a >= 0 else 0
        line = list(old[a]) if a == b else [p if e < -(-n // page) else -1 for e, p in enumerate(old[a])] if a >= 0 else [-1] * width
        if a >= 0 and n % page and owner.setdefault(a, b) != b:
            line[n // page] = -1
            copies.append((b, n // page, old[a][n // page], n % page))
        table.append(line)
        lens.append(n)

    def lowest():
        named = {p for line in table for p in line}
        return [p for p in range(s["pages"]) if p not in named]

    for (b, e, page_from, rows), to in zip(copies, lowest()):
        table[b][e] = to
        for x in map(_bits, _caches(s)):
            x[:, to, :, :rows] = x[:, page_from, :, :rows]
    table = [[p if e < -(-(n + 1) // page) else -1 for e, p in enumerate(line)] for line, n in zip(table, lens)]
    wants = [b for b in range(batch) if lens[b] % page == 0 and table[b][lens[b] // page] < 0]
    free = lowest()
    for b, to in zip(wants, free):
        table[b][lens[b] // page] = to
    return _pool_outputs(s, _ints(table), _ints(lens), _ints([len(free) - len(wants)]))


def _exact_compact(s):
    table = s["table"].tolist()
    named = sorted({p for line in table for p in line if p >= 0})
    rest = [p for p in range(len(named)) if p not in set(named)]
    to = dict(zip([p for p in named if p >= len(named)], rest))
    for p, q in to.items():
        for x in map(_bits, _caches(s)):
            x[:, q] = x[:, p]
    return _pool_outputs(s, _ints([[to.get(p, p) for p in line] for line in table]), _ints([len(named)]))
