"""The operators of drafted decoding together, as a server uses them: pages taken, drafts appended and attended as a
tree, the model's choices accepted, their rows kept; sequences forked, ended and moved together on the way.  Against
decoding token by token."""
import math

import numpy as np
import pytest

from bit_weight_only_mxfp4_gb300 import loader, synth, thinmx

from . import branch_ref as br
from . import gpu_util as gu
from . import paged_ref as ref
from .parity import bf16_to_f64

pytestmark = pytest.mark.gpu

VOCAB, HEADS, KVH, D, PAGE, LAYERS = 97, 16, 4, 64, 16, 2
ROW = (HEADS + 2 * KVH) * D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


class Model:
    """A token's queries, keys and values are the token's alone (a row of a table for each layer), so that they have the
    same bits however many tokens are computed together.  The next token is one that the last one decides, by far."""

    def __init__(self, seed):
        import torch
        r = synth.rng(171, seed, 0)
        self.qkv = gu.dev(synth.f32_to_bf16_bits(r.standard_normal((LAYERS, VOCAB, ROW)).astype(np.float32)))
        self.head = torch.from_numpy(r.standard_normal((HEADS * D, VOCAB)).astype(np.float32)).cuda()
        self.after = torch.from_numpy(r.permutation(VOCAB)).cuda()
        freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
        self.turns = loader.rope_turns(freq)

    def logits(self, tokens, out):
        import torch
        x = out.view(torch.bfloat16).float().reshape(len(tokens), -1) @ self.head * 0.1
        x[torch.arange(len(tokens), device="cuda"), self.after[tokens.long()]] += 100.0
        return x.bfloat16().contiguous()


class Server:
    """Caches of all layers over one table, pages taken as they are needed."""

    def __init__(self, model, batch, pages, width, fp8):
        import torch
        self.m, self.batch, self.fp8 = model, batch, fp8
        kind = torch.uint8 if fp8 else torch.int16
        self.k, self.v = (torch.zeros((LAYERS, pages, KVH, PAGE, D), dtype=kind, device="cuda") for _ in range(2))
        self.s = [torch.zeros((LAYERS, pages, KVH, PAGE), device="cuda") for _ in range(2)] if fp8 else None
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.kvs = [loader.paged_kv(self.k[i], self.v[i], self.table, self.lens,
                                    *((self.s[0][i], self.s[1][i]) if fp8 else ())) for i in range(LAYERS)]
        self.layers = loader.paged_layers(self.kvs)
        # one workspace for the decode and tree attention
        nb = max(thinmx.tt_paged_tree_workspace_bytes(HEADS, KVH, D),
                 thinmx.tt_paged_attention_workspace_bytes(HEADS, KVH, D))
        self.ws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
        nb = thinmx.tt_paged_pages_workspace_bytes(self.kvs[0])
        self.pws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
        self.left = torch.zeros(1, dtype=torch.int32, device="cuda")

    def grow(self, by):
        """Pages for `by` more tokens of each sequence, whose lengths then count them."""
        want = self.lens + by
        thinmx.tt_paged_resize(self.kvs[0], want, None, self.table, self.lens, self.left, *self.pws)
        self.lens.copy_(want)

    def attend(self, tokens, starts, positions=None, masks=None):
        import torch
        n = len(tokens)
        outs = []
        for i in range(LAYERS):
            x = self.m.qkv[i][tokens.long()].contiguous()
            p = x.data_ptr()
            q = torch.empty((n, HEADS, D), dtype=torch.int16, device="cuda")
            out = torch.empty_like(q)
            thinmx.tt_paged_rope_append(self.kvs[i], p, p + 2 * HEADS * D, p + 2 * (HEADS + KVH) * D, ROW, ROW, n, starts,
                                        HEADS, self.m.turns, D, False, positions, 1, None, q)
            if masks is None:
                thinmx.tt_paged_decode_attention(self.kvs[i], q, HEADS * D, HEADS, 1 / math.sqrt(D), 0.0, 0, None, None,
                                                 out, None, *self.ws)
            else:
                thinmx.tt_paged_tree_attention(self.kvs[i], q, HEADS * D, starts, n, HEADS, 1 / math.sqrt(D), 0.0, 0,
                                               None, None, masks, masks.shape[1], out, None, *self.ws)
            outs.append(out)
        return outs

    def choose(self, tokens, out):
        """The model's choices, with their log probabilities checked."""
        import torch
        x = self.m.logits(tokens, out)
        n = len(tokens)
        ids, logp = torch.empty((n, 1), dtype=torch.int32, device="cuda"), torch.empty((n, 1), device="cuda")
        nb = thinmx.tt_token_logprobs_workspace_bytes(n, VOCAB, 1)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        thinmx.tt_token_logprobs(x, thinmx.TT_LOGITS_BF16, n, VOCAB, VOCAB, 1.0, None, 1, None, None, ids, logp, ws, nb)
        want = torch.log_softmax(x.double(), 1).max(1)[0]
        assert float((logp[:, 0].double() - want).abs().max()) < 1e-5
        return ids[:, 0].contiguous()

    def rows(self, b):
        """The cached rows of sequence b, all layers: [..., length, D] bits, and scales."""
        n, table = int(self.lens[b]), gu.host(self.table)[b]
        t = np.arange(n)
        at = table[t // PAGE], t % PAGE
        assert (at[0] >= 0).all()
        return [gu.host(x)[:, at[0], :, at[1]] for x in [self.k, self.v] + (self.s or [])]


def plain(model, prompts, steps, fp8):
    """Token by token: (tokens after each prompt, the server with its rows, outputs of every token)."""
    import torch
    s = Server(model, len(prompts), 60, 12, fp8)
    now = torch.tensor([p[0] for p in prompts], dtype=torch.int32, device="cuda")
    said, outs = [], []
    for i in range(steps):
        s.grow(1)
        out = s.attend(now, None)
        outs.append([gu.host(x, np.uint16) for x in out])
        said.append(now.tolist())
        nxt = s.choose(now, out[-1])
        now = torch.tensor([p[i + 1] if i + 1 < len(p) else int(nxt[b]) for b, p in enumerate(prompts)],
                           dtype=torch.int32, device="cuda")
    return np.array(said).T.tolist(), s, outs


@pytest.mark.parametrize("fp8", [False, True])
def test_drafted_decoding_gives_what_decoding_gives(fp8):
    import torch
    model = Model(1)
    steps = 70
    prompts = [[5], [8], [41]]
    said, one, outs = plain(model, prompts, steps, fp8)
    r = synth.rng(171, 2, 0)
    s = Server(model, 3, 60, 12, fp8)
    done = [[p[0]] for p in prompts]  # the last one is chosen, and not yet cached
    order = list(range(3))            # whose text a place has
    taken = 0
    while max(len(t) for t in done) + 9 < steps:
        # trees of 1 to 8 nodes: mostly the text's own continuation, and other tokens beside it
        new = [int(r.integers(1, 9)) for _ in range(3)]
        parents, drafts = [], []
        for b, n in enumerate(new):
            up, depth, own = br.parents_of(r, n), [], []
            for i, p in enumerate(up):
                depth.append(depth[p] + 1 if p >= 0 else 0)
                right = said[order[b]][len(done[b]) - 1 + depth[i]]
                taken_before = any(up[e] == p and own[e] == right for e in range(i))
                own.append(right if i == 0 or (r.random() < 0.8 and not taken_before) else (right + 1) % VOCAB)
            parents += up
            drafts += own
        starts = gu.dev(np.cumsum([0] + new).astype(np.int32))
        n = sum(new)
        parents, drafts = gu.dev(np.array(parents, np.int32)), gu.dev(np.array(drafts, np.int32))
        s.grow(gu.dev(np.array(new, np.int32)))
        masks, positions, path = (torch.empty(shape, dtype=torch.int32, device="cuda") for shape in ((n, 1), (n,), (3, 8)))
        counts, nxt = (torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2))
        thinmx.tt_draft_tree(parents, starts, s.lens, 3, n, 1, masks, positions)
        out = s.attend(drafts, starts, positions, masks)
        chosen = s.choose(drafts, out[-1])
        thinmx.tt_draft_accept(parents, drafts, chosen, starts, 3, n, 8, path, counts, nxt)
        thinmx.tt_paged_keep(s.layers, LAYERS, starts, path, 8, counts, s.lens)
        count, ways, first = counts.tolist(), path.tolist(), starts.tolist()
        for b in range(3):
            way = [drafts[first[b] + i].item() for i in ways[b][:count[b]]]
            at = len(done[b]) - 1
            assert way == said[order[b]][at:at + count[b]] and nxt[b].item() == said[order[b]][at + count[b]]
            # what the accepted nodes saw is what decoding saw
            for j in range(count[b]):
                for layer in range(LAYERS):
                    got = bf16_to_f64(gu.host(out[layer], np.uint16)[first[b] + ways[b][j]])
                    want = bf16_to_f64(outs[at + j][layer][order[b]])
                    # a weighted mean of values of unit size, rounded to bf16 twice, weights to bf16 or f16 in between
                    assert np.abs(got - want).max() <= 6 * 2.0 ** -8 * max(1.0, np.abs(want).max())
            done[b] += way[1:] + [nxt[b].item()]
            assert int(s.lens[b]) == len(done[b]) - 1
        taken += 1
        if taken == 4:  # the third sequence ends, and its place goes on with the first one's text
            come = gu.dev(np.array([0, 1, 0], np.int32))
            thinmx.tt_paged_fork(s.layers, LAYERS, come, None, s.table, s.lens, s.left, *s.pws)
            order[2], done[2] = order[0], list(done[0])
        if taken % 5 == 0:
            thinmx.tt_paged_compact(s.layers, LAYERS, None, s.table, s.left, *s.pws)
            table = gu.host(s.table)
            assert s.left.item() == len(set(table[table >= 0].tolist())) == table.max() + 1
    assert gu.device_error() == 0
    for b in range(3):
        n = int(s.lens[b])
        for got, want in zip(s.rows(b), one.rows(order[b])):
            assert np.array_equal(got, want[:n])  # [token][layer][kv head]..: the same bits


def test_three_attentions_share_a_workspace():
    """Decode, prompt and tree attention in turn on one workspace, each as on its own."""
    import torch
    from .test_gpu_paged import _attend, _handle
    from .test_gpu_tree import attend, queries
    heads, kvh, d = 16, 4, 128
    nb = max(thinmx.tt_paged_tree_workspace_bytes(heads, kvh, d), thinmx.tt_paged_attention_workspace_bytes(heads, kvh, d))
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb
    cache = ref.Cache(31, [3000, 700], kvh, d, 16)
    kv = _handle(cache)
    starts = np.array([0, 9, 14], np.int32)
    masks = [m for n in (9, 5) for m in br.masks_of(br.parents_of(synth.rng(171, 3, n), n))]
    q = queries(31, 14, heads, d)

    def calls(w):
        return [_attend(kv, q[:2], None, 0.1, ws=w), attend(kv, q, starts, masks, 1, 0.1, ws=w),
                _attend(kv, q, starts, 0.1, ws=w), attend(kv, q, starts, masks, 1, 0.1, ws=w),
                _attend(kv, q[:2], None, 0.1, ws=w)]

    for got, want in zip(calls(ws), calls(None)):
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert gu.device_error() == 0
