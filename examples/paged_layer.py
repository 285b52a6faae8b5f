"""One decoder layer served over the paged key-value cache, on the library's kernels alone.

Prompts of several lengths are projected, their keys and values appended to the pages with the position rotation, and
attended; then the sequences decode together, one token each per step, the whole layer in one CUDA graph whose lengths
grow in place.  The projections are bf16 (tt_bf16_matvec, up to eight rows a call), the gate/up MXFP4 SwiGLU, the cache
bf16 or FP8.

    python examples/paged_layer.py [--fp8] [--steps 16]

checks that decoding token by token gives what one prompt over all tokens gives.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_only_mxfp4_gb300 import loader, thinmx  # noqa: E402


class Layer:
    """Random weights of a small layer; rows of activations in, rows out (no norms: the point is the cache)."""

    def __init__(self, hidden=512, heads=16, kv_heads=4, head_dim=64, inter=1024, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.inter = hidden, heads, kv_heads, head_dim, inter
        self.row = (heads + 2 * kv_heads) * head_dim

        def weight(n, k):
            return torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)

        self.qkv, self.o = weight(self.row, hidden).bfloat16(), weight(hidden, heads * head_dim).bfloat16()
        self.gate_up = loader.mxfp4_gate_up_from_f32(weight(inter, hidden), weight(inter, hidden))
        self.down = weight(hidden, inter).bfloat16()
        inv_freq = 500000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64, device="cuda") / (head_dim // 2))
        self.turns = loader.rope_turns(inv_freq)

    def matvec(self, w, x, y):
        for i in range(0, len(x), 8):
            m = min(8, len(x) - i)
            thinmx.tt_bf16_matvec(w, w.shape[0], w.shape[1], x[i:i + m], m, y[i:i + m])

    def __call__(self, cache, x, starts, work):
        """x [tokens][hidden] -> [tokens][hidden]; starts as in tt_paged_rope_append (None: one token per sequence)."""
        n, h, g, d = len(x), self.heads, self.kv_heads, self.head_dim
        qkv, q, att = work["qkv"][:n], work["q"][:n], work["att"][:n]
        self.matvec(self.qkv, x, qkv)
        p = qkv.data_ptr()
        thinmx.tt_paged_rope_append(cache.kv, p, p + 2 * h * d, p + 2 * (h + g) * d, self.row, self.row, n, starts, h,
                                    self.turns, d, False, None, 1, None, q)
        scale = 1.0 / math.sqrt(d)
        if starts is None:
            thinmx.tt_paged_decode_attention(cache.kv, q, h * d, h, scale, 0.0, 0, None, None, att, None, cache.ws,
                                             cache.ws_bytes)
        else:
            thinmx.tt_paged_prefill_attention(cache.kv, q, h * d, starts, n, h, scale, 0.0, 0, None, None, None, att,
                                              None, cache.ws, cache.ws_bytes)
        mid, hid, out = work["mid"][:n], work["hid"][:n], work["out"][:n]
        self.matvec(self.o, att.view(n, h * d), mid)
        for i in range(0, n, 8):
            m = min(8, n - i)
            thinmx.tt_mxfp4_swiglu_matvec(self.gate_up, self.inter, self.hidden, mid[i:i + m], m, hid[i:i + m])
        self.matvec(self.down, hid, out)
        return out

    def work(self, tokens):
        def rows(width):
            return torch.empty((tokens, width), dtype=torch.bfloat16, device="cuda")
        hd = self.heads * self.head_dim
        return dict(qkv=rows(self.row), q=rows(hd), att=rows(hd), mid=rows(self.hidden), hid=rows(self.inter),
                    out=rows(self.hidden))


class Cache:
    """The layer's pages, dealt out to the sequences in turn."""

    def __init__(self, layer, most, page=16, fp8=False):
        batch, need = len(most), [-(-n // page) for n in most]
        shape = (sum(need), layer.kv_heads, page, layer.head_dim)
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        k, v = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
        ks, vs = ((torch.zeros(shape[:3], device="cuda") for _ in range(2)) if fp8 else (None, None))
        table = torch.full((batch, max(need)), -1, dtype=torch.int32)
        free = iter(torch.randperm(shape[0]).tolist())
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([next(free) for _ in range(n)], dtype=torch.int32)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.kv = loader.paged_kv(k, v, table.cuda(), self.lens, ks, vs)
        self.ws_bytes = thinmx.tt_paged_attention_workspace_bytes(layer.heads, layer.kv_heads, layer.head_dim)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")


def prompt(layer, cache, xs):
    """One prompt per sequence, from an empty cache; the rows of each sequence's tokens."""
    lens = [len(x) for x in xs]
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    out = layer(cache, torch.cat(xs), starts, layer.work(sum(lens)))
    return list(out.split(lens))


def serve(fp8=False, steps=16, lens=(37, 5, 130)):
    """(rows by decoding, rows by one prompt) of the last `steps` tokens of every sequence: [steps][batch][hidden]."""
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn(n + steps, layer.hidden, generator=g, device="cuda").bfloat16() for n in lens]
    most = [n + steps for n in lens]
    cache = Cache(layer, most, fp8=fp8)
    prompt(layer, cache, [x[:n] for x, n in zip(xs, lens)])
    x, work = torch.zeros((len(lens), layer.hidden), dtype=torch.bfloat16, device="cuda"), layer.work(len(lens))

    def step():
        cache.lens += 1
        layer(cache, x, None, work)

    step()  # a call may be captured once it has been made
    cache.lens -= 1  # (the row that it wrote is the next one to be written)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    rows = []
    for i in range(steps):
        x.copy_(torch.stack([s[n + i] for s, n in zip(xs, lens)]))
        graph.replay()
        rows.append(work["out"].clone())
    whole = prompt(layer, Cache(layer, most, fp8=fp8), xs)
    torch.cuda.synchronize()
    assert thinmx.tt_device_error_read() == 0
    return torch.stack(rows), torch.stack([r[-steps:] for r in whole], 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--fp8", action="store_true", help="E4M3 cache with a scale per token and kv head")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    one, whole = serve(a.fp8, a.steps)
    far = ((one.float() - whole.float()).norm() / whole.float().norm()).item()
    print(f"{a.steps} steps of 3 sequences: decoded rows against one prompt's, relative difference {far:.2e}")


if __name__ == "__main__":
    main()
