"""Host-side orchestration of the NVFP4 routed-expert path on the C ABI.

Torch provides device memory and the stream; each step is one call into
``libnvfp4.so``.  ``MoEExperts.forward`` is the MoE layer's expert part:
gather + per-group dynamic quantize -> grouped gate_up GEMM -> SwiGLU +
per-group requantize -> grouped down GEMM (the routed-expert projections of
the "Qwen3.8-Flash-Next-NVFP4" page, quantized W4A4).
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Optional

import torch

from . import (EPI_NONE, EPI_SWIGLU, GS_AMAX_GIVEN, GS_FROM_AMAX, GS_GIVEN, NORM_E4M3, NORM_NVFP4, OUT_BF16, OUT_F32,
               SF_MMA_TILED, SF_ROWMAJOR, nvfp4_add_rmsnorm_quantize, nvfp4_kv_append, nvfp4_kv_dequantize,
               nvfp4_paged_attention, nvfp4_paged_attention_workspace_size,
               mxfp4_grouped_gemm as _mxfp4_grouped_gemm, mxfp4_quantize as _mxfp4_quantize, mxfp4_to_nvfp4, nvfp4_dequantize, nvfp4_grouped_gemm, nvfp4_grouped_gemm_swiglu_nvfp4,
               nvfp4_global_scale_from_amax, nvfp4_grouped_gemm_w4a16, nvfp4_moe_combine,
               nvfp4_w4a16_workspace_size,
               nvfp4_moe_route,
               nvfp4_moe_quantize, nvfp4_moe_route_workspace_size, nvfp4_padded_rows_bound, nvfp4_quantize,
               nvfp4_swiglu_quantize,
               nvfp4_workspace_size)


@dataclass
class Packed:
    """An NVFP4 tensor in device memory.

    q: uint8 [rows_alloc, K/2]; sf: uint8 scales (``layout``); gs: fp32 [G]
    global scales.  With ``offsets`` (int32 [G+1] on the device) rows sit in
    128-aligned per-group slots.  ``gs_given``: gs is a tensor of the caller's (a
    calibrated scale); quantizing into this Packed again gives it scales of its own.
    """
    q: torch.Tensor
    sf: torch.Tensor
    gs: torch.Tensor
    rows: int
    K: int
    layout: int
    offsets: Optional[torch.Tensor] = None
    num_groups: int = 1
    gs_given: bool = False


def _own_scales(p: Packed, G: int):
    """Make p.gs a tensor that a call may write G scales to."""
    if p.gs_given:
        p.gs, p.gs_given = torch.empty(max(1, G), dtype=torch.float32, device=p.q.device), False
    elif p.gs.numel() < G:
        raise ValueError(f"out: {G} global scales are wanted, not {p.gs.numel()}")


def workspace(num_groups: int, device="cuda") -> torch.Tensor:
    n = nvfp4_workspace_size(max(1, num_groups))
    return torch.empty(n, dtype=torch.uint8, device=device)


def alloc_rows(rows: int, num_groups: int, grouped: bool, layout: int) -> int:
    if grouped:
        return nvfp4_padded_rows_bound(rows, num_groups)
    return (rows + 127) // 128 * 128 if layout == SF_MMA_TILED else rows


def sf_bytes(rows_alloc: int, K: int) -> int:
    return rows_alloc * (K // 16)


def empty_packed(rows: int, K: int, num_groups: int = 1, offsets=None, layout=SF_MMA_TILED,
                 device="cuda") -> Packed:
    ra = alloc_rows(rows, num_groups, offsets is not None, layout)
    q = torch.empty((max(ra, 1), K // 2), dtype=torch.uint8, device=device)
    sf = torch.empty(max(sf_bytes(ra, K), 1), dtype=torch.uint8, device=device)
    gs = torch.empty(max(1, num_groups), dtype=torch.float32, device=device)
    return Packed(q, sf, gs, rows, K, layout, offsets, num_groups if offsets is not None else 1)


def quantize(x: torch.Tensor, row_index=None, offsets=None, num_groups: int = 1, layout=SF_MMA_TILED,
             global_scale=None, out: Optional[Packed] = None, ws=None, dev_status=None, rows=None) -> Packed:
    """NVFP4-quantize bf16 rows (dynamic global scale unless ``global_scale`` is given)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    K = x.shape[1]
    R = rows if rows is not None else (row_index.shape[0] if row_index is not None else x.shape[0])
    G = num_groups if offsets is not None else 1
    p = out if out is not None else empty_packed(R, K, G, offsets, layout, x.device)
    _own_scales(p, G)
    p.offsets, p.num_groups, p.rows = offsets, G, R
    mode = GS_FROM_AMAX
    if global_scale is not None:
        p.gs.copy_(global_scale)
        mode = GS_GIVEN
    ws = ws if ws is not None else workspace(G, x.device)
    nvfp4_quantize(x, R, K, x.stride(0), row_index, offsets, G, mode, p.gs, p.q, p.sf, layout, ws, dev_status)
    return p


def moe_quantize(x: torch.Tensor, slot: torch.Tensor, offsets: torch.Tensor, num_groups: int, layout=SF_MMA_TILED,
                 out: Optional[Packed] = None, ws=None, dev_status=None, rows=None) -> Packed:
    """Routed-expert activations quantized in token order: the same packed rows
    as ``quantize(x, row_index, offsets, ...)`` with row_index the inverse of
    ``slot`` [T, k] (routed row of each token choice), each token read once."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and slot.dim() == 2
    T, k = slot.shape
    K = x.shape[1]
    R = rows if rows is not None else T * k
    p = out if out is not None else empty_packed(R, K, num_groups, offsets, layout, x.device)
    _own_scales(p, num_groups)
    p.offsets, p.num_groups, p.rows = offsets, num_groups, R
    ws = ws if ws is not None else workspace(num_groups, x.device)
    nvfp4_moe_quantize(x, T, K, x.stride(0), slot, k, offsets, num_groups, GS_FROM_AMAX, p.gs, p.q, p.sf, layout,
                       ws, dev_status)
    return p


def dequantize(p: Packed, out_dtype=OUT_F32) -> torch.Tensor:
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    y = torch.empty((p.rows, p.K), dtype=dt, device=p.q.device)
    nvfp4_dequantize(p.q, p.sf, p.layout, p.gs, p.offsets, p.num_groups, p.rows, p.K, y, out_dtype)
    return y


def remap_mxfp4(q_mx: torch.Tensor, e8: torch.Tensor, n_tensors: int, rows: int, K: int, layout=SF_MMA_TILED,
                ws=None, dev_status=None, inplace: bool = False) -> Packed:
    """Lossless MXFP4 -> NVFP4 remap of n_tensors [rows, K] tensors."""
    q_nv = q_mx if inplace else torch.empty_like(q_mx)
    sf = torch.empty(n_tensors * rows * (K // 16), dtype=torch.uint8, device=q_mx.device)
    gs = torch.empty(n_tensors, dtype=torch.float32, device=q_mx.device)
    ws = ws if ws is not None else workspace(n_tensors, q_mx.device)
    mxfp4_to_nvfp4(q_mx, e8, n_tensors, rows, K, q_nv, sf, layout, gs, ws, dev_status)
    return Packed(q_nv, sf, gs, n_tensors * rows, K, layout, None, n_tensors)


def mxfp4_quantize(x: torch.Tensor, layout=SF_ROWMAJOR, dev_status=None):
    """MXFP4 encode of bf16 rows [rows, K]: (codes uint8 [rows, K/2], UE8M0
    scales, one per 32 elements, in `layout`)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, K = x.shape
    q = torch.empty((rows, K // 2), dtype=torch.uint8, device=x.device)
    if layout == SF_MMA_TILED:
        e8 = torch.empty(((rows + 127) // 128 * 128) * (K // 32), dtype=torch.uint8, device=x.device)
    else:
        e8 = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    _mxfp4_quantize(x, rows, K, x.stride(0), q, e8, layout, dev_status)
    return q, e8


def mx_grouped_gemm(a_q: torch.Tensor, a_sf: torch.Tensor, w_q: torch.Tensor, w_sf: torch.Tensor, N: int, K: int,
                    rows: int, offsets: Optional[torch.Tensor] = None, num_experts: int = 1, out_dtype=OUT_BF16,
                    y=None, dev_status=None) -> torch.Tensor:
    """MXFP4 x MXFP4 grouped GEMM: Y [rows, N] = per expert A_e W_e^T
    (activations in 128-aligned expert slots, tensor-core scale layout)."""
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if y is None:
        y = torch.empty((rows, N), dtype=dt, device=a_q.device)
    E = num_experts if offsets is not None else 1
    _mxfp4_grouped_gemm(a_q, a_sf, w_q, w_sf, offsets, E, rows, N, K, y, out_dtype, None, dev_status)
    return y


def grouped_gemm(a: Packed, w: Packed, N: int, out_dtype=OUT_BF16, y=None, dev_status=None) -> torch.Tensor:
    """Y [a.rows, N] = per expert (a_gs[e] * w_gs[e]) * A_e W_e^T."""
    assert a.layout == SF_MMA_TILED and w.layout == SF_MMA_TILED
    E = a.num_groups if a.offsets is not None else 1
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if y is None:
        y = torch.empty((a.rows, N), dtype=dt, device=a.q.device)
    nvfp4_grouped_gemm(a.q, a.sf, a.gs, w.q, w.sf, w.gs, a.offsets, E, a.rows, N, a.K, y, out_dtype, EPI_NONE,
                       None, None, dev_status)
    return y


def gate_up_interleave_index(E: int, I: int, device="cuda") -> torch.Tensor:
    """Source row of each packed row of a fused gate_up weight [E*2I, K] in the
    order the SwiGLU epilogue reads: per expert, 32-row groups holding 16 gate
    rows and then the 16 matching up rows (gate rows are 0..I-1 of the expert,
    up rows I..2I-1 in the source).  int32 [E*2I]."""
    assert I % 64 == 0
    n = torch.arange(E * 2 * I, dtype=torch.int64)
    e, m = n // (2 * I), n % (2 * I)
    j, r = m // 32, m % 32
    src = e * 2 * I + torch.where(r < 16, 16 * j + r, I + 16 * j + (r - 16))
    return src.to(torch.int32).to(device)


def pack_weights(w: torch.Tensor, E: int, rows_per: int, row_index=None, ws=None) -> Packed:
    """Static NVFP4 quantization of per-expert weights [E*rows_per, K] (one global
    scale per expert, MMA-tiled scales), optionally reordering rows within each
    expert (``row_index``, e.g. ``gate_up_interleave_index``)."""
    offs = torch.arange(0, (E + 1) * rows_per, rows_per, dtype=torch.int32, device=w.device)
    p = quantize(w, row_index, offs, E, SF_MMA_TILED, ws=ws)
    p.offsets, p.num_groups, p.rows = None, 1, E * rows_per
    return p


def grouped_gemm_swiglu(a: Packed, w_gate_up: Packed, N: int, h=None, amax=None, dev_status=None):
    """h [a.rows, N/2] = bf16(silu(g) * u) straight from the gate_up GEMM's
    accumulators, plus the per-expert amax of h (fp32 [E]).  ``w_gate_up`` is
    packed in the interleaved row order of ``gate_up_interleave_index``."""
    assert a.layout == SF_MMA_TILED and w_gate_up.layout == SF_MMA_TILED
    E = a.num_groups if a.offsets is not None else 1
    if h is None:
        h = torch.empty((a.rows, N // 2), dtype=torch.bfloat16, device=a.q.device)
    if amax is None:
        amax = torch.empty(E, dtype=torch.float32, device=a.q.device)
    nvfp4_grouped_gemm(a.q, a.sf, a.gs, w_gate_up.q, w_gate_up.sf, w_gate_up.gs, a.offsets, E, a.rows, N, a.K, h,
                       OUT_BF16, EPI_SWIGLU, amax, None, dev_status)
    return h, amax


def grouped_gemm_swiglu_nvfp4(a: Packed, w_gate_up: Packed, N: int, h_gs: torch.Tensor, out: Optional[Packed] = None,
                              dev_status=None) -> Packed:
    """gate_up GEMM + SwiGLU whose epilogue quantizes h with the given per-expert
    global ``h_gs`` (the down projection's calibrated input scale): the packed
    down-GEMM input, with no bf16 h in memory."""
    assert a.layout == SF_MMA_TILED and w_gate_up.layout == SF_MMA_TILED
    E = a.num_groups if a.offsets is not None else 1
    I = N // 2
    p = out if out is not None else empty_packed(a.rows, I, E, a.offsets, SF_MMA_TILED, a.q.device)
    p.offsets, p.num_groups, p.rows = a.offsets, E, a.rows
    p.gs, p.gs_given = h_gs, True
    nvfp4_grouped_gemm_swiglu_nvfp4(a.q, a.sf, a.gs, w_gate_up.q, w_gate_up.sf, w_gate_up.gs, a.offsets, E, a.rows,
                                    N, a.K, h_gs, p.q, p.sf, None, dev_status)
    return p


def w4a16_workspace(rows: int, num_groups: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(nvfp4_w4a16_workspace_size(rows, num_groups, K), dtype=torch.uint8, device=device)


def grouped_gemm_w4a16(x: torch.Tensor, w: Packed, N: int, row_index=None, offsets=None, num_groups: int = 1,
                       rows=None, out_dtype=OUT_BF16, swiglu=False, y=None, ws=None, dev_status=None) -> torch.Tensor:
    """Weight-only NVFP4 (row-major scales) x bf16 activations, per expert:
    Y [rows, N] (or h [rows, N/2] with ``swiglu``; gate rows first)."""
    assert x.dtype == torch.bfloat16 and w.layout == SF_ROWMAJOR
    M = rows if rows is not None else (row_index.shape[0] if row_index is not None else x.shape[0])
    G = num_groups if offsets is not None else 1
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    cols = N // 2 if swiglu else N
    if y is None:
        y = torch.empty((M, cols), dtype=dt, device=x.device)
    if ws is None:
        ws = w4a16_workspace(M, G, w.K, x.device)
    nvfp4_grouped_gemm_w4a16(x, x.stride(0), x.shape[0], row_index, w.q, w.sf, w.gs, offsets, G, M, N, w.K, y,
                             out_dtype, EPI_SWIGLU if swiglu else EPI_NONE, ws, dev_status)
    return y


def swiglu_quantize(y: torch.Tensor, offsets, num_groups: int, layout=SF_MMA_TILED, out: Optional[Packed] = None,
                    h=None, ws=None, dev_status=None):
    rows, I2 = y.shape
    I = I2 // 2
    G = num_groups if offsets is not None else 1
    p = out if out is not None else empty_packed(rows, I, G, offsets, layout, y.device)
    _own_scales(p, G)
    p.offsets, p.num_groups, p.rows = offsets, G, rows
    h = h if h is not None else torch.empty((rows, I), dtype=torch.bfloat16, device=y.device)
    ws = ws if ws is not None else workspace(G, y.device)
    ydt = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    nvfp4_swiglu_quantize(y, ydt, rows, I, offsets, G, p.gs, p.q, p.sf, layout, h, ws, dev_status)
    return p, h


class MoEExperts:
    """Routed experts of one MoE layer in NVFP4 W4A4.

    w_gate_up: packed [E*2I, H], one global scale per expert: rows 0..I-1 of
    each expert = gate, I..2I-1 = up; with ``fused_swiglu`` the rows are in the
    order of ``gate_up_interleave_index`` instead.  w_down: packed [E*H, I].
    forward(x bf16 [T, H], row_index int32 [R], offsets int32 [E+1]) -> Y bf16 [R, H]
    in routed order (the weighted combine is outside this layer).  With
    ``h_scale`` set (a given down-input global per expert, see
    ``calibrate_h_scale``) the gate_up epilogue writes NVFP4 h directly.
    """

    def __init__(self, w_gate_up: Packed, w_down: Packed, E: int, H: int, I: int, max_rows: int,
                 out_dtype=OUT_BF16, mid_dtype=OUT_BF16, device="cuda", fused_swiglu: bool = False):
        self.fused_swiglu = fused_swiglu
        self.h_scale: Optional[torch.Tensor] = None   # given down-input global per expert (fp32 [E])
        self.amax = torch.zeros(E, dtype=torch.float32, device=device)
        self.w_gate_up, self.w_down = w_gate_up, w_down
        self.E, self.H, self.I = E, H, I
        self.out_dtype, self.mid_dtype = out_dtype, mid_dtype
        self.ws = workspace(E, device)
        self.a1 = empty_packed(max_rows, H, E, torch.empty(0), SF_MMA_TILED, device)
        self.a2 = empty_packed(max_rows, I, E, torch.empty(0), SF_MMA_TILED, device)
        mdt = torch.bfloat16 if mid_dtype == OUT_BF16 else torch.float32
        odt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
        self.y1 = torch.empty((max_rows, 2 * I), dtype=mdt, device=device)
        self.h = torch.empty((max_rows, I), dtype=torch.bfloat16, device=device)
        self.y2 = torch.empty((max_rows, H), dtype=odt, device=device)
        self.max_rows = max_rows

    def _quantize_input(self, x, row_index, offsets, slot, dev_status):
        R = row_index.shape[0]
        if slot is not None:
            return moe_quantize(x, slot, offsets, self.E, SF_MMA_TILED, out=self.a1, ws=self.ws,
                                dev_status=dev_status, rows=R)
        return quantize(x, row_index, offsets, self.E, SF_MMA_TILED, out=self.a1, ws=self.ws,
                        dev_status=dev_status, rows=R)

    def forward(self, x: torch.Tensor, row_index: torch.Tensor, offsets: torch.Tensor, dev_status=None,
                slot: Optional[torch.Tensor] = None):
        """``slot`` [T, k] (routed row of each token choice), when given, selects
        the token-order quantize that reads each token row once."""
        R = row_index.shape[0]
        assert R <= self.max_rows
        E, H, I = self.E, self.H, self.I
        a1 = self._quantize_input(x, row_index, offsets, slot, dev_status)
        if self.h_scale is not None:
            # calibrated down-input global: the gate_up epilogue writes NVFP4 h itself
            a2 = grouped_gemm_swiglu_nvfp4(a1, self.w_gate_up, 2 * I, self.h_scale, out=self.a2,
                                           dev_status=dev_status)
        elif self.fused_swiglu:
            # SwiGLU in the gate_up epilogue; its amax feeds the requantize directly
            h, amax = grouped_gemm_swiglu(a1, self.w_gate_up, 2 * I, h=self.h[:R], amax=self.amax,
                                          dev_status=dev_status)
            a2 = self.a2
            a2.offsets, a2.num_groups, a2.rows = offsets, E, R
            nvfp4_quantize(h, R, I, I, None, offsets, E, GS_AMAX_GIVEN, amax, a2.q, a2.sf, SF_MMA_TILED, self.ws,
                           dev_status)
            a2.gs = amax
        else:
            y1 = self.y1[:R]
            grouped_gemm(a1, self.w_gate_up, 2 * I, self.mid_dtype, y=y1, dev_status=dev_status)
            a2, _ = swiglu_quantize(y1, offsets, E, SF_MMA_TILED, out=self.a2, h=self.h[:R], ws=self.ws,
                                    dev_status=dev_status)
        y2 = self.y2[:R]
        grouped_gemm(a2, self.w_down, H, self.out_dtype, y=y2, dev_status=dev_status)
        return y2


def calibrate_h_scale(experts: "MoEExperts", x, row_index, offsets, slot=None, margin: float = 1.0,
                      dev_status=None) -> torch.Tensor:
    """A down-input global per expert from one calibration batch, as a
    calibration pass would set the checkpoint's input_scale, installed on
    ``experts``: the dynamic path's first two stages give the per-expert max |h|
    (SwiGLU epilogue), and the library turns it into s_g = margin * max|h| / 2688
    (1 for an expert without tokens) with the same arithmetic as the dynamic
    global scale.  With margin 1 the result is exactly the s_g a dynamic forward
    derives for the same batch."""
    assert experts.fused_swiglu
    experts.h_scale = None
    R = row_index.shape[0]
    a1 = experts._quantize_input(x, row_index, offsets, slot, dev_status)
    _, amax = grouped_gemm_swiglu(a1, experts.w_gate_up, 2 * experts.I, h=experts.h[:R], amax=experts.amax,
                                  dev_status=dev_status)
    gs = torch.empty(experts.E, dtype=torch.float32, device=amax.device)
    nvfp4_global_scale_from_amax(amax, experts.E, margin, gs, dev_status)
    experts.h_scale = gs
    return gs


def route(topk_ids: torch.Tensor, num_experts: int, dev_status=None):
    """Expert-grouped order of routed rows: (offsets [E+1], row_index [T*k], slot [T, k])."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    off = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    ri = torch.empty(T * k, dtype=torch.int32, device=dev)
    slot = torch.empty((T, k), dtype=torch.int32, device=dev)
    ws = torch.empty(nvfp4_moe_route_workspace_size(T, num_experts), dtype=torch.uint8, device=dev)
    nvfp4_moe_route(topk_ids, T, k, num_experts, off, ri, slot, ws, dev_status)
    return off, ri, slot


def combine(y: torch.Tensor, slot: torch.Tensor, weights: torch.Tensor, out_dtype=OUT_BF16, out=None,
            dev_status=None):
    """out[t] = sum_j weights[t, j] * y[slot[t, j]] (fp32 accumulation); slots
    outside y's rows are skipped and reported in dev_status."""
    T, k = slot.shape
    H = y.shape[1]
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=y.device)
    ydt = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    nvfp4_moe_combine(y, ydt, y.shape[0], slot, weights, T, k, H, out, out_dtype, dev_status)
    return out


class MoELayer:
    """A whole routed-expert MoE block on one GPU: routing order, the NVFP4
    W4A4 experts, and the weighted combine back to [T, H].

    forward(x bf16 [T, H], topk_ids int32 [T, k], topk_weights fp32 [T, k]) -> bf16 [T, H].
    The router itself (BF16 gate, top-k) stays outside, as on the pages.
    """

    def __init__(self, experts: MoEExperts, max_tokens: int, topk: int, device="cuda"):
        self.experts = experts
        E = experts.E
        self.off = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.ri = torch.empty(max_tokens * topk, dtype=torch.int32, device=device)
        self.slot = torch.empty((max_tokens, topk), dtype=torch.int32, device=device)
        self.rws = torch.empty(nvfp4_moe_route_workspace_size(max_tokens, E), dtype=torch.uint8, device=device)
        self.out = torch.empty((max_tokens, experts.H), dtype=torch.bfloat16, device=device)

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, dev_status=None):
        T, k = topk_ids.shape
        E = self.experts.E
        slot = self.slot[:T]
        ri = self.ri[:T * k]
        nvfp4_moe_route(topk_ids, T, k, E, self.off, ri, slot, self.rws, dev_status)
        y = self.experts.forward(x, ri, self.off, dev_status, slot=slot)
        out = self.out[:T]
        nvfp4_moe_combine(y, OUT_F32 if y.dtype == torch.float32 else OUT_BF16, y.shape[0], slot, topk_weights, T, k,
                          self.experts.H, out, OUT_BF16, dev_status)
        return out

    def capture(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, dev_status=None):
        """Record forward() on these input tensors as a CUDA graph.

        Returns (graph, out): graph.replay() reruns the whole block (routing
        order, experts, combine: about ten kernel launches and memsets) on the
        current contents of x, topk_ids and topk_weights, which keep their
        shapes and addresses, and leaves the result in out.  forward() issues
        no host synchronisation and allocates nothing, so it captures as is;
        one eager call first sets the kernels' launch attributes.

        ``out`` is a view of this layer's own output buffer, not a copy: a
        later eager forward(), or the replay of another graph captured on this
        layer, overwrites it.  Copy it out (or read it) before either runs."""
        self.forward(x, topk_ids, topk_weights, dev_status)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self.forward(x, topk_ids, topk_weights, dev_status)
        return graph, out


# ---------------------------------------------------------------- the norm in front of a projection
def _rows(t: torch.Tensor, K: int, what: str):
    """A bf16 [rows, K] operand with unit stride along K: its row stride."""
    shape, stride = t.shape, t.stride()
    if t.dtype != torch.bfloat16 or len(shape) != 2 or shape[1] != K or (stride[1] != 1 and K > 1):
        raise ValueError(f"{what}: a bf16 [rows, {K}] tensor with contiguous rows is wanted")
    return stride[0] if shape[0] > 1 else K


def _norm_args(x, weight, residual, residual_out):
    if x.dim() != 2:
        raise ValueError("x: a bf16 [rows, K] tensor is wanted")
    rows, K = x.shape
    ld_x = _rows(x, K, "x")
    if weight.dtype != torch.bfloat16 or weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError(f"weight: a contiguous bf16 [{K}] tensor is wanted")
    ld_res = 0
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual: the shape of x is wanted")
        ld_res = _rows(residual, K, "residual")
    ld_ro = 0
    if residual_out is None and residual is not None:
        residual_out, ld_ro = torch.empty_like(x, memory_format=torch.contiguous_format), K
    elif residual_out is not None:
        if residual_out.shape != x.shape:
            raise ValueError("residual_out: the shape of x is wanted")
        ld_ro = _rows(residual_out, K, "residual_out")
    _same_device(x, weight, residual, residual_out)
    return rows, K, ld_x, ld_res, residual_out, ld_ro


def _same_device(first, *others):
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def _status(t):
    """A status word for the device to write, or None."""
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1):
        raise ValueError("dev_status: an int32 tensor of one element is wanted")


_HERE = contextlib.nullcontext()


def _cuda(t: torch.Tensor) -> bool:
    return t.get_device() >= 0


def _on(t: torch.Tensor):
    """A context in which t's device is the current one (torch's own costs some
    microseconds even when it already is)."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"CUDA tensors are wanted, not {t.device}")
    return _HERE if torch._C._cuda_getDevice() == d else torch.cuda.device(d)


def add_rmsnorm_nvfp4(x: torch.Tensor, weight: torch.Tensor, global_scale: torch.Tensor, residual=None,
                      eps: float = 1e-6, layout=SF_MMA_TILED, out: Optional[Packed] = None, residual_out=None,
                      y=None, dev_status=None):
    """r = x + residual, y = rmsnorm(r) * weight, and y as NVFP4 with the given
    global scale (a calibrated ``input_scale``, fp32 [1]), in one pass.

    Returns (packed y, r, y): the packed y holds ``global_scale`` itself (no copy);
    r is ``residual_out`` (allocated when a residual is given; may be ``residual``
    itself) or x; y is the bf16 buffer passed as ``y``, or None."""
    rows, K, ld_x, ld_res, residual_out, ld_ro = _norm_args(x, weight, residual, residual_out)
    if global_scale.dtype != torch.float32 or global_scale.numel() != 1:
        raise ValueError("global_scale: an fp32 tensor of one element is wanted")
    if y is not None and (y.dtype != torch.bfloat16 or y.shape != x.shape or not y.is_contiguous()):
        raise ValueError("y: a contiguous bf16 tensor of x's shape is wanted")
    p = out if out is not None else empty_packed(rows, K, 1, None, layout, x.device)
    ra = alloc_rows(rows, 1, False, layout)
    if p.K != K or p.layout != layout or p.q.dim() != 2 or p.q.shape[0] < ra or p.q.shape[1] != K // 2 or \
            p.q.dtype != torch.uint8 or not p.q.is_contiguous():
        raise ValueError("out: packed uint8 codes of this K and layout with enough rows are wanted")
    if p.sf.dtype != torch.uint8 or not p.sf.is_contiguous() or p.sf.numel() < sf_bytes(ra, K):
        raise ValueError("out: uint8 scales, enough of them, are wanted")
    _status(dev_status)
    _same_device(x, global_scale, y, p.q, p.sf, dev_status)
    p.gs, p.gs_given, p.offsets, p.num_groups, p.rows = global_scale, True, None, 1, rows
    with _on(x):
        nvfp4_add_rmsnorm_quantize(x, ld_x, residual, ld_res, rows, K, weight, eps, residual_out, ld_ro, y,
                                   NORM_NVFP4, global_scale, p.q, p.sf, layout, dev_status)
    return p, (residual_out if residual_out is not None else x), y


def add_rmsnorm_e4m3(x: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6, q=None, scale=None,
                     residual_out=None, y=None, dev_status=None):
    """As add_rmsnorm_nvfp4 with an 8-bit output: (q uint8 [rows, K] E4M3 bytes,
    scale fp32 [rows], r, y); q * scale[:, None] stands for y."""
    rows, K, ld_x, ld_res, residual_out, ld_ro = _norm_args(x, weight, residual, residual_out)
    if q is None:
        q = torch.empty_like(x, dtype=torch.uint8, memory_format=torch.contiguous_format)
    elif q.element_size() != 1 or q.shape != x.shape or not q.is_contiguous():
        raise ValueError("q: a contiguous one-byte tensor of x's shape is wanted")
    if scale is None:
        scale = weight.new_empty(rows, dtype=torch.float32)
    elif scale.dtype != torch.float32 or scale.numel() != rows or not scale.is_contiguous():
        raise ValueError("scale: fp32 [rows] is wanted")
    if y is not None and (y.dtype != torch.bfloat16 or y.shape != x.shape or not y.is_contiguous()):
        raise ValueError("y: a contiguous bf16 tensor of x's shape is wanted")
    _status(dev_status)
    _same_device(x, q, scale, y, dev_status)
    with _on(x):
        nvfp4_add_rmsnorm_quantize(x, ld_x, residual, ld_res, rows, K, weight, eps, residual_out, ld_ro, y,
                                   NORM_E4M3, scale, q, None, SF_ROWMAJOR, dev_status)
    return q, scale, (residual_out if residual_out is not None else x), y


# ---------------------------------------------------------------- the paged NVFP4 KV cache
def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [positions, rot_dim] for ``PagedKVCache.append``: per position the
    rot_dim/2 cosines, then the sines, of position * base^(-2i/rot_dim); the
    angles in 64 bits, so that far positions keep their digits."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * (base ** (-i / rot_dim))[None, :]
    return torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()


def _heads(t: torch.Tensor, tokens, D: int, what: str):
    """A bf16 [tokens, heads, D] operand whose heads of a token are contiguous: its token stride."""
    shape, stride = t.shape, t.stride()
    if t.dtype != torch.bfloat16 or len(shape) != 3 or shape[2] != D or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{what}: a bf16 [tokens, heads, {D}] tensor is wanted")
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != D):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return stride[0] if shape[0] > 1 else shape[1] * D


class PagedKVCache:
    """One attention layer's paged NVFP4 KV cache.

    k_q, v_q: uint8 [num_pages, heads, page_size, D/2] codes; k_sf, v_sf: uint8
    [num_pages, heads, page_size, D/16] scales; k_gs, v_gs: fp32 [1] static
    global scales.  ``PagedKVCache.empty`` allocates them.  A slot is
    page * page_size + row; the caller keeps the page tables."""

    def __init__(self, k_q, k_sf, k_gs, v_q, v_sf, v_gs):
        if k_q.dim() != 4:
            raise ValueError("k_q: uint8 [num_pages, heads, page_size, D/2] is wanted")
        self.num_pages, self.heads, self.page_size, half = k_q.shape
        self.head_dim = D = 2 * half
        for name, t, n in (("k_q", k_q, half), ("v_q", v_q, half), ("k_sf", k_sf, D // 16), ("v_sf", v_sf, D // 16)):
            if t.dtype != torch.uint8 or tuple(t.shape) != (*k_q.shape[:3], n) or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous uint8 {[*k_q.shape[:3], n]} tensor is wanted")
        for name, t in (("k_gs", k_gs), ("v_gs", v_gs)):
            if t.dtype != torch.float32 or t.numel() != 1:
                raise ValueError(f"{name}: an fp32 tensor of one element is wanted")
        _same_device(k_q, k_sf, k_gs, v_q, v_sf, v_gs)
        self.k_q, self.k_sf, self.k_gs, self.v_q, self.v_sf, self.v_gs = k_q, k_sf, k_gs, v_q, v_sf, v_gs
        self._need = {}                 # workspace bytes by (batch, max_query, q_heads), at most 256 of them
        self._captured = []             # workspaces that captured graphs point to

    @classmethod
    def empty(cls, num_pages: int, page_size: int, heads: int, head_dim: int, k_gs: torch.Tensor, v_gs: torch.Tensor,
              device="cuda") -> "PagedKVCache":
        def u8(n):
            return torch.empty((num_pages, heads, page_size, n), dtype=torch.uint8, device=device)
        return cls(u8(head_dim // 2), u8(head_dim // 16), k_gs, u8(head_dim // 2), u8(head_dim // 16), v_gs)

    def append(self, k, v, slots, q=None, q_out=None, positions=None, rope=None, interleaved: bool = False,
               dev_status=None):
        """Quantize k, v (bf16 [tokens, heads, D], the keys rotated to
        ``positions`` by ``rope``) into ``slots`` (int64, negative = skip), and
        return the rotated queries (``q_out``, allocated when not given; may be
        q itself), or None without q."""
        D, tokens = self.head_dim, k.shape[0]
        ld_k, ld_v = _heads(k, None, D, "k"), _heads(v, tokens, D, "v")
        if k.shape[1] != self.heads or v.shape[1] != self.heads:
            raise ValueError(f"k, v: {self.heads} heads are wanted")
        if slots.dtype != torch.int64 or slots.shape != (tokens,) or not slots.is_contiguous():
            raise ValueError("slots: a contiguous int64 [tokens] tensor is wanted")
        rot = rows = 0
        if rope is not None:
            if rope.dtype != torch.float32 or rope.dim() != 2 or not rope.is_contiguous():
                raise ValueError("rope: a contiguous fp32 [positions, rot_dim] tensor is wanted")
            rows, rot = rope.shape
            if positions is None or positions.dtype != torch.int64 or positions.shape != (tokens,) or \
                    not positions.is_contiguous():
                raise ValueError("positions: a contiguous int64 [tokens] tensor is wanted")
        ld_q = ld_qo = hq = 0
        if q is not None:
            ld_q, hq = _heads(q, tokens, D, "q"), q.shape[1]
            if q_out is None:
                q_out, ld_qo = torch.empty_like(q, memory_format=torch.contiguous_format), hq * D
            else:
                ld_qo = _heads(q_out, tokens, D, "q_out")
                if q_out.shape != q.shape:
                    raise ValueError("q_out: the shape of q is wanted")
        _status(dev_status)
        _same_device(self.k_q, k, v, slots, q, q_out, positions, rope, dev_status)
        with _on(self.k_q):
            nvfp4_kv_append(k, ld_k, v, ld_v, tokens, self.heads, D, slots, q, ld_q, hq, q_out, ld_qo, positions, rope,
                            rows, rot, int(interleaved), self.k_gs, self.v_gs, self.k_q, self.k_sf, self.v_q,
                            self.v_sf, self.num_pages, self.page_size, dev_status)
        return q_out if q is not None else None

    def workspace(self, batch: int, max_query: int, q_heads: int) -> torch.Tensor:
        """A workspace for ``attend`` calls of up to these sizes on one stream."""
        return torch.empty(max(self._size(batch, max_query, q_heads), 1), dtype=torch.uint8, device=self.k_q.device)

    def _size(self, batch: int, max_query: int, q_heads: int) -> int:
        # by the SM count of the cache's device
        with _on(self.k_q) if _cuda(self.k_q) else _HERE:
            return nvfp4_paged_attention_workspace_size(batch, max_query, q_heads, self.heads, self.head_dim)

    def attend(self, q, seq_lens, page_table, query_offsets=None, max_query: Optional[int] = None, softmax_scale=None,
               causal: bool = True, out=None, out_dtype=OUT_BF16, lse=None, ws=None, dev_status=None):
        """Attention of q (bf16 [tokens, q_heads, D]) over the cache.

        seq_lens int32 [batch]: cached tokens, the queries' own included;
        page_table int32 [batch, pages]; query_offsets int32 [batch + 1] with at
        most ``max_query`` queries each, which has to be given with them (None:
        one query per sequence); lse: fp32 [tokens, q_heads] to fill.  Returns
        out [tokens, q_heads, D].  Offsets that break this are reported in
        ``dev_status`` and nothing is computed.

        ``ws`` (from ``workspace``; allocated when not given) serves one call at a
        time.  One that is given to a captured call is kept as long as this cache:
        a graph holds no reference to it, and a later capture's start gives
        unused memory back to the device."""
        D = self.head_dim
        ld_q = _heads(q, None, D, "q")
        tokens, hq, _ = q.shape
        if seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
            raise ValueError("seq_lens: a contiguous int32 [batch] tensor is wanted")
        batch = seq_lens.shape[0]
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != batch or \
                not page_table.is_contiguous():
            raise ValueError("page_table: a contiguous int32 [batch, pages] tensor is wanted")
        if query_offsets is not None and (query_offsets.dtype != torch.int32 or query_offsets.shape != (batch + 1,) or
                                          not query_offsets.is_contiguous()):
            raise ValueError("query_offsets: a contiguous int32 [batch + 1] tensor is wanted")
        if query_offsets is None:
            if max_query not in (None, 1):
                raise ValueError("max_query: one query per sequence without query_offsets")
            max_query = 1
        elif max_query is None:
            raise ValueError("max_query: the most queries of a sequence is wanted with query_offsets")
        dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
        if out is None:
            out = torch.empty_like(q, dtype=dt, memory_format=torch.contiguous_format)
        elif out.dtype != dt or out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out: a contiguous {dt} tensor of q's shape is wanted")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != (tokens, hq) or not lse.is_contiguous()):
            raise ValueError("lse: a contiguous fp32 [tokens, q_heads] tensor is wanted")
        need = self._need.get((batch, max_query, hq))
        if need is None:
            if len(self._need) >= 256:
                self._need.clear()
            need = self._need[batch, max_query, hq] = self._size(batch, max_query, hq)
        given = ws is not None
        if not given:
            ws = self.k_q.new_empty(max(need, 1))
        elif ws.numel() * ws.element_size() < need or not ws.is_contiguous():
            raise ValueError("ws: too small, or with gaps (PagedKVCache.workspace gives one)")
        _status(dev_status)
        _same_device(self.k_q, q, seq_lens, page_table, query_offsets, out, lse, ws, dev_status)
        scale = D ** -0.5 if softmax_scale is None else softmax_scale
        with _on(self.k_q):
            if given and torch.cuda.is_current_stream_capturing() and not any(w is ws for w in self._captured):
                self._captured.append(ws)
            nvfp4_paged_attention(q, ld_q, tokens, query_offsets, max_query, seq_lens, batch, page_table,
                                  page_table.shape[1], hq, self.heads, D, self.k_q, self.k_sf, self.k_gs, self.v_q,
                                  self.v_sf, self.v_gs, self.num_pages, self.page_size, scale, int(causal), out,
                                  out_dtype, lse, ws, dev_status)
        return out

    def dequantize(self):
        """The whole pool back in bf16: (k, v), each [num_pages, heads, page_size, D]."""
        shape = (*self.k_q.shape[:3], self.head_dim)
        k = self.k_q.new_empty(shape, dtype=torch.bfloat16)
        v = torch.empty_like(k)
        with _on(self.k_q):
            nvfp4_kv_dequantize(self.k_q, self.k_sf, self.k_gs, self.v_q, self.v_sf, self.v_gs,
                                self.num_pages * self.page_size, self.heads, self.head_dim, k, v)
        return k, v
