"""Weight loader: canonical fp32 / MXFP4 tensors on the device -> the packed
layouts the matvec kernels stream.  Every step runs in the library's CUDA
kernels through the C ABI; torch only allocates the buffers."""
from __future__ import annotations

import torch

from . import thinmx


def quantize_mxfp4(w: torch.Tensor, status: torch.Tensor | None = None):
    """fp32 [n, k] (k % 32 == 0) -> (codes uint8 [n, k/2], scales uint8 [n, k/32])."""
    assert w.is_cuda and w.dtype == torch.float32 and w.is_contiguous()
    n, k = w.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((n, k // 32), dtype=torch.uint8, device=w.device)
    thinmx.tt_quantize_mxfp4(w, n, k, codes, scales, status)
    return codes, scales


def pack_swiglu(gate, up, n: int, k: int) -> torch.Tensor:
    """gate/up = (codes, scales, postscale fp32 [n] or None) -> packed buffer."""
    nbytes = thinmx.tt_mxfp4_swiglu_packed_bytes(n, k)
    if nbytes == 0:
        raise ValueError(f"unsupported gate/up shape n={n} k={k}")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=gate[0].device)
    thinmx.tt_mxfp4_pack_swiglu(gate[0], gate[1], gate[2], up[0], up[1], up[2], n, k, packed,
                                nbytes)
    return packed


def mxfp4_gate_up_from_f32(wg: torch.Tensor, wu: torch.Tensor, pg=None, pu=None) -> torch.Tensor:
    """Quantise both fp32 matrices and pack them; the canonical codes are freed."""
    n, k = wg.shape
    gc, gs = quantize_mxfp4(wg)
    uc, us = quantize_mxfp4(wu)
    packed = pack_swiglu((gc, gs, pg), (uc, us, pu), n, k)
    del gc, gs, uc, us
    return packed


def expert_table(buffers) -> torch.Tensor:
    """The device array of expert buffer addresses the MoE entry points take
    (one int64 per expert, in expert order).  The buffers must stay alive as
    long as the table is used."""
    dev = buffers[0].device
    return torch.tensor([b.data_ptr() for b in buffers], dtype=torch.int64, device=dev)


def moe_expert_from_f32(w_gate_up: torch.Tensor, w_down: torch.Tensor):
    """One expert's fp32 gate/up [2*inter, hidden] (gate rows first) and down
    [hidden, inter] matrices -> its own packed gate/up and down buffers."""
    two_i, hidden = w_gate_up.shape
    inter = two_i // 2
    gc, gs = quantize_mxfp4(w_gate_up)
    gu = pack_swiglu((gc[:inter], gs[:inter], None), (gc[inter:], gs[inter:], None), inter,
                     hidden)
    dc, ds = quantize_mxfp4(w_down)
    nbytes = thinmx.tt_mxfp4_rows_packed_bytes(hidden, inter)
    dn = torch.empty(nbytes, dtype=torch.uint8, device=w_down.device)
    thinmx.tt_mxfp4_pack_rows(dc, ds, hidden, inter, dn, nbytes)
    return gu, dn


def paged_kv(k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
             k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
    """The cache description the paged entry points take: k, v
    [pages, kv_heads, page_size, head_dim] in bf16 (or its bits in int16 /
    uint16), or in float8_e4m3fn (or its codes in uint8 / int8) with fp32 scales
    [pages, kv_heads, page_size]; page_table int32
    [batch, pages_per_seq]; lens int32 [batch].  It keeps its tensors alive;
    it is made once, and later steps write into page_table and lens."""
    fp8 = k_scales is not None
    for t in (k, v, page_table, lens, k_scales, v_scales):
        assert t is None or (t.is_cuda and t.is_contiguous())
    assert k.shape == v.shape and k.dtype == v.dtype
    assert k.dtype in ((torch.float8_e4m3fn, torch.uint8, torch.int8) if fp8 else
                       (torch.bfloat16, torch.int16, torch.uint16))
    assert (v_scales is not None) == fp8
    pages, kv_heads, page_size, head_dim = k.shape
    assert page_table.dtype == lens.dtype == torch.int32
    batch, width = page_table.shape
    assert lens.shape == (batch,)
    if fp8:
        assert k_scales.shape == v_scales.shape == (pages, kv_heads, page_size)
        assert k_scales.dtype == v_scales.dtype == torch.float32
    kv = thinmx.tt_paged_kv(
        k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if fp8 else None,
        v_scales.data_ptr() if fp8 else None, page_table.data_ptr(), lens.data_ptr(), pages,
        thinmx.TT_KV_FP8 if fp8 else thinmx.TT_KV_BF16, page_size, kv_heads, head_dim, batch,
        width)
    kv.tensors = (k, v, page_table, lens, k_scales, v_scales)
    return kv


def paged_layers(kvs):
    """The caches of several layers (paged_kv, over one page_table and one lens) as
    the array that tt_paged_keep, tt_paged_fork and tt_paged_compact take.  It keeps
    their tensors alive."""
    layers = (thinmx.tt_paged_kv * len(kvs))(*kvs)
    layers.tensors = [getattr(kv, "tensors", None) for kv in kvs]
    return layers


def rope_turns(inv_freq: torch.Tensor) -> torch.Tensor:
    """Rotation frequencies, fp64 [n] in radians per position -> the table
    tt_paged_rope_append takes."""
    assert inv_freq.is_cuda and inv_freq.dtype == torch.float64 and inv_freq.is_contiguous()
    turns = torch.empty(inv_freq.numel(), dtype=torch.int64, device=inv_freq.device)
    thinmx.tt_rope_turns(inv_freq, inv_freq.numel(), turns)
    return turns
