"""Convenience sequences of the C-ABI calls, with torch allocating the buffers.

This module only orders calls into the library (amax -> scales -> pack ->
conv; norm -> codes -> linear) and allocates their outputs; it performs no
arithmetic of its own.

stream: a torch stream or a raw handle (default: torch's current stream). Work
on it is as under ``torch.cuda.stream(stream)``: outputs and scratch come from
the allocator's pool of that stream, so that no block is handed out again while
the stream still works on it. What the inputs wait for, and who else uses the
outputs, is the caller's to order, as with torch's own operations.
"""

from __future__ import annotations

import contextlib

import torch

from . import binding as B

DTYPES = {"bf16": B.IGC_BF16, "fp8": B.IGC_FP8_E4M3FN}
LAYOUTS = {"NCDHW": B.IGC_NCDHW, "NDHWC": B.IGC_NDHWC}


def _code(dtype):
    return DTYPES[dtype] if isinstance(dtype, str) else int(dtype)


def _allocating(stream, device):
    """The context in which buffers for work on `stream` are allocated."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def packed_weight(w_kctrs: torch.Tensor, dtype="bf16", x_layout="NDHWC", scale_pair=None, stream=None):
    """Pack a bf16 KCTRS filter (fp8: scale_pair must hold its {s, inv})."""
    dt = _code(dtype)
    cols = B.conv_packed_w_cols(w_kctrs.shape, dt)
    with _allocating(stream, w_kctrs.device):
        out = torch.empty((w_kctrs.shape[0], cols), dtype=torch.uint8 if dt == B.IGC_FP8_E4M3FN else torch.bfloat16,
                          device=w_kctrs.device)
    B.conv_pack_w(w_kctrs, out, w_kctrs.shape, dt, LAYOUTS[x_layout], scale_pair, stream)
    return out


def packed_input(x_ncdhw: torch.Tensor, dtype="bf16", scale_pair=None, stream=None):
    """NCDHW bf16 -> NDHWC (bf16 or fp8 codes), returned as a (N, D, H, W, C) tensor."""
    dt = _code(dtype)
    n, c, d, h, w = x_ncdhw.shape
    with _allocating(stream, x_ncdhw.device):
        out = torch.empty((n, d, h, w, c), dtype=torch.uint8 if dt == B.IGC_FP8_E4M3FN else torch.bfloat16,
                          device=x_ncdhw.device)
    B.conv_pack_x(x_ncdhw, out, x_ncdhw.shape, dt, scale_pair, stream)
    return out


def fp8_scales(x_bf16: torch.Tensor, w_bf16: torch.Tensor, stream=None):
    """Device float[4] = {s_x, inv_x, s_w, inv_w} from the two tensors' amax."""
    with _allocating(stream, x_bf16.device):
        amax = torch.empty(2, dtype=torch.float32, device=x_bf16.device)
        scales = torch.empty(4, dtype=torch.float32, device=x_bf16.device)
    B.conv_amax(x_bf16, x_bf16.numel(), amax[0:1], stream)
    B.conv_fp8_scales(amax[0:1], scales[0:2], stream)
    B.conv_amax(w_bf16, w_bf16.numel(), amax[1:2], stream)
    B.conv_fp8_scales(amax[1:2], scales[2:4], stream)
    return scales


def output(xshape, wshape, stride, pad, dil, device):
    do, ho, wo = B.conv_out_dims(xshape, wshape, stride, pad, dil)
    return torch.empty((xshape[0], wshape[0], do, ho, wo), dtype=torch.bfloat16, device=device)


def conv3d(x_ncdhw: torch.Tensor, w_kctrs: torch.Tensor, stride=(1, 1, 1), pad=(0, 0, 0), dil=(1, 1, 1),
           dtype="bf16", stream=None):
    """y = conv3d(x, w) from bf16 NCDHW x and bf16 KCTRS w, all on the GPU.

    Point-output shapes and bf16 1x1x1 filters read x as is; other shapes pack
    x to NDHWC first. fp8 quantises both operands with per-tensor amax/448
    scales."""
    dt = _code(dtype)
    xshape, wshape = tuple(x_ncdhw.shape), tuple(w_kctrs.shape)
    direct = dt == B.IGC_BF16 and direct_ncdhw(xshape, wshape, stride, pad, dil)
    scales = fp8_scales(x_ncdhw, w_kctrs, stream) if dt == B.IGC_FP8_E4M3FN else None
    sx = scales[0:2] if scales is not None else None
    sw = scales[2:4] if scales is not None else None
    with _allocating(stream, x_ncdhw.device):
        y = output(xshape, wshape, stride, pad, dil, x_ncdhw.device)
    if direct:
        wp = packed_weight(w_kctrs, dt, "NCDHW", sw, stream)
        B.conv_fwd(x_ncdhw, wp, y, xshape, wshape, stride, pad, dil, dt, B.IGC_NCDHW, scales, stream)
        return y
    xp = packed_input(x_ncdhw, dt, sx, stream)
    wp = packed_weight(w_kctrs, dt, "NDHWC", sw, stream)
    B.conv_fwd(xp, wp, y, xshape, wshape, stride, pad, dil, dt, B.IGC_NDHWC, scales, stream)
    return y


def direct_ncdhw(xshape, wshape, stride, pad, dil) -> bool:
    """True when the library reads bf16 NCDHW x as it is for this shape (point output, or the 1x1x1 pointwise
    path) instead of needing the NDHWC pack."""
    try:
        plan = B.conv_plan(xshape, wshape, stride, pad, dil, B.IGC_BF16, B.IGC_NCDHW)
    except B.IgcError:
        return False
    return plan.startswith("path=point")


# ---------------------------------------------------------------- tokens

CODES = {"int8": B.IGC_INT8, "fp8": B.IGC_FP8_E4M3FN}
_CODE_TYPES = {B.IGC_INT8: torch.int8, B.IGC_FP8_E4M3FN: torch.float8_e4m3fn}
_VALUE_TYPES = {torch.bfloat16: B.IGC_BF16, torch.float32: B.IGC_F32}


def _value_type(t: torch.Tensor) -> int:
    if t.dtype not in _VALUE_TYPES:
        raise TypeError(f"expected bfloat16 or float32 rows, got {t.dtype}")
    return _VALUE_TYPES[t.dtype]


def _row_stride(t, rows, cols, name):
    """Elements from row to row of a matrix whose rows are contiguous (a slice of a wider one may be passed)."""
    if t is None:
        return 0
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be {rows} x {cols}, got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if rows > 1 else max(t.stride(0), cols)


def _vector(t, n, dtype, name):
    if t is not None and (tuple(t.shape) != (n,) or t.dtype != dtype or (n > 1 and t.stride(0) != 1)):
        raise ValueError(f"{name} must be {n} contiguous values of {dtype}")
    return t


class Codes:
    """A matrix in 8 bits: `codes` (rows x linear_packed_cols(cols), zeros past cols), one fp32 `scales` value for
    each row; element (i, k) stands for codes[i, k] * scales[i]."""

    def __init__(self, rows: int, cols: int, kind, device):
        self.kind = CODES[kind] if isinstance(kind, str) else int(kind)
        self.rows, self.cols = rows, cols
        self.codes = torch.empty((rows, B.linear_packed_cols(cols)), dtype=_CODE_TYPES[self.kind], device=device)
        self.scales = torch.empty((rows,), dtype=torch.float32, device=device)

    @property
    def ld(self) -> int:
        return self.codes.shape[1]


def quantised(x: torch.Tensor, kind="int8", glu=False, stream=None) -> Codes:
    """Codes of the rows of x (bf16 or fp32): a linear weight by output channel, an activation by token; glu: of
    silu(first half) * second half of each row."""
    rows, wide = x.shape
    if glu and wide % 2:
        raise ValueError(f"a gated row holds two halves, got {wide} elements")
    cols = wide // 2 if glu else wide
    with _allocating(stream, x.device):
        q = Codes(rows, cols, kind, x.device)
    B.linear_quant(x, _row_stride(x, rows, wide, "x"), q.codes, q.ld, q.scales, rows, cols, _value_type(x), q.kind,
                   B.IGC_ACT_SILU_GLU if glu else B.IGC_ACT_NONE, stream)
    return q


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual=None, eps=1e-6, kind=None, stream=None):
    """(y, h): the norm of h = x + residual (h is x without one), y as x's type, or as Codes with kind "int8" / "fp8"."""
    rows, cols = x.shape
    dt = _value_type(x)
    for t, name in ((residual, "residual"), (weight, "weight")):
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{name} must be {x.dtype} like x, got {t.dtype}")
    with _allocating(stream, x.device):
        h = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if residual is not None else None
        y = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if kind is None else Codes(rows, cols, kind, x.device)
    out, ld, scales, y_type = (y, cols, None, dt) if kind is None else (y.codes, y.ld, y.scales, y.kind)
    B.norm_fwd(x, _row_stride(x, rows, cols, "x"), residual, _row_stride(residual, rows, cols, "residual"),
               _vector(weight, cols, x.dtype, "weight"), h, cols, out, ld, scales, rows, cols, eps, dt, y_type, stream)
    return y, (x if h is None else h)


def rms_norm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, dres=None, eps=1e-6, stream=None):
    """(dx, dw) of rms_norm's y with respect to h (so to x and to the residual alike) and the weight; dres: the
    gradient that reaches h along the residual stream, added to dx. dw is fp32."""
    rows, cols = h.shape
    dt = _value_type(h)
    for t, name in ((dy, "dy"), (dres, "dres"), (weight, "weight")):
        if t is not None and t.dtype != h.dtype:
            raise TypeError(f"{name} must be {h.dtype} like h, got {t.dtype}")
    with _allocating(stream, h.device):
        dx = torch.empty((rows, cols), dtype=h.dtype, device=h.device)
        dw = torch.empty((cols,), dtype=torch.float32, device=h.device)
        ws = torch.empty((B.norm_bwd_workspace_bytes(rows, cols),), dtype=torch.uint8, device=h.device)
    B.norm_bwd(dy, _row_stride(dy, rows, cols, "dy"), h, _row_stride(h, rows, cols, "h"),
               _vector(weight, cols, h.dtype, "weight"), dres, _row_stride(dres, rows, cols, "dres"), dx, cols, dw, rows,
               cols, eps, dt, ws, None, stream)
    return dx, dw


def linear(a: Codes, w: Codes, bias=None, out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """y[i, j] = sum_k a[i, k] * w[j, k] + bias[j] over the values both codes stand for (out: a matrix to write)."""
    if a.kind != w.kind:
        raise TypeError("both operands must have the same kind of codes")
    if a.cols != w.cols:
        raise ValueError(f"reduction lengths differ: {a.cols} and {w.cols}")
    m, n, k = a.rows, w.rows, a.cols
    with _allocating(stream, a.codes.device):
        y = torch.empty((m, n), dtype=out_dtype, device=a.codes.device) if out is None else out
        nws = B.linear_fwd_workspace_bytes(m, n, k, a.kind, _value_type(y))
        ws = torch.empty((nws,), dtype=torch.uint8, device=a.codes.device) if nws else None
    B.linear_fwd(a.codes, a.ld, a.scales, w.codes, w.ld, w.scales, _vector(bias, n, torch.float32, "bias"), y,
                 _row_stride(y, m, n, "out"), m, n, k, a.kind, _value_type(y), ws, None, stream)
    return y
