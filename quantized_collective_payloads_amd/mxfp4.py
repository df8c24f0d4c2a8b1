"""The MXFP4 payload (4.25 bits per weight), its product on the matrix cores, and
a linear layer whose three products run on it (mxfp4_* of include/qcp.h).

A payload of `lines` rows of n values is a pair (codes, scales): uint8
[lines, P/2] and uint8 [lines, P/32] with P = n rounded up to whole 128s.
"""
from __future__ import annotations

import torch

from . import (DTYPES, _check, _dev, _dtype_code, _ELEMS, _need, _ptr, _stream, _U8, library)


def mxfp4_padded(n: int) -> int:
    """Values that a payload row of n values holds: n rounded up to whole 128s."""
    p = int(library().qcp_mxfp4_padded(n))
    if p < 0:
        raise ValueError(f"row length {n} is negative or too large")
    return p


def _matrix(x, what: str):
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{what}: expected a torch.Tensor, got {type(x).__name__}")
    if x.dtype not in DTYPES:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {' or '.join(map(str, _ELEMS))}")
    if x.dim() != 2:
        raise ValueError(f"{what}: {x.dim()} dimensions, expected 2")
    return x


def _payload(codes, scales, what: str):
    """(lines, padded row length) of a payload after checking its two tensors."""
    for t, name, unit in ((codes, "codes", 64), (scales, "scales", 4)):
        _need(t, f"{what}{name}", _U8, 0)
        if t.dim() != 2:
            raise ValueError(f"{what}{name}: {t.dim()} dimensions, expected 2")
        if t.shape[1] % unit:
            raise ValueError(f"{what}{name}: rows of {t.shape[1]} bytes, expected a multiple of {unit}")
    if scales.shape != (codes.shape[0], codes.shape[1] // 16):
        raise ValueError(f"{what}scales: shape {tuple(scales.shape)} for codes of {tuple(codes.shape)}, "
                         f"expected {(codes.shape[0], codes.shape[1] // 16)}")
    return codes.shape[0], 2 * codes.shape[1]


def mxfp4_quantize(x: torch.Tensor, transpose: bool = False, codes=None, scales=None):
    """The payload (codes, scales) of a 2-D fp16/bf16/fp32 GPU tensor, or with
    `transpose` of x.t().  Rows may lie any distance apart, and a transposed view
    is read where it is; other strides are copied first.  Caller-supplied `codes`
    and `scales` must be contiguous uint8 of the payload's shape."""
    _matrix(x, "x")
    if x.numel() and x.stride(1) != 1 and x.shape[1] != 1:
        if x.stride(0) == 1 or x.shape[0] == 1:
            x, transpose = x.t(), not transpose
        else:
            x = x.contiguous()
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    if rows > 1 and ld < cols:                       # rows that overlap (an expanded tensor)
        x = x.contiguous()
        ld = cols
    lines, n = (cols, rows) if transpose else (rows, cols)
    P = mxfp4_padded(n)
    for t, what, shape in ((codes, "codes", (lines, P // 2)), (scales, "scales", (lines, P // 32))):
        if t is not None:
            _need(t, what, _U8, 0)
            if tuple(t.shape) != shape:
                raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
    dev = _dev(x, codes, scales)
    if codes is None:
        codes = torch.empty((lines, P // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((lines, P // 32), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check("mxfp4_quantize", library().mxfp4_quantize(
            _ptr(x), DTYPES[x.dtype], rows, cols, ld, int(bool(transpose)), _ptr(codes), _ptr(scales),
            _stream(dev)))
    return codes, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int, dtype=torch.bfloat16, out=None):
    """The [lines, cols] values that a payload stands for, rounded once to `dtype`."""
    lines, P = _payload(codes, scales, "")
    if mxfp4_padded(cols) != P:
        raise ValueError(f"codes: rows of {P} values for {cols} columns, expected {mxfp4_padded(cols)}")
    if out is not None:
        _matrix(out, "out")
        _need(out, "out", _ELEMS, 0)
        if tuple(out.shape) != (lines, cols):
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {(lines, cols)}")
    dev = _dev(codes, scales, out)
    if out is None:
        _dtype_code(dtype)
        out = torch.empty((lines, cols), dtype=dtype, device=dev)
    with torch.cuda.device(dev):
        _check("mxfp4_dequantize", library().mxfp4_dequantize(
            _ptr(codes), _ptr(scales), lines, cols, _ptr(out), DTYPES[out.dtype], cols, _stream(dev)))
    return out


def mxfp4_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
                 b_scales: torch.Tensor, dtype=torch.bfloat16, out=None):
    """A B^T for the payloads of A [M, K] and B [N, K]: [M, N] in `dtype`,
    accumulated in fp32 and rounded once."""
    M, K = _payload(a_codes, a_scales, "a_")
    N, Kb = _payload(b_codes, b_scales, "b_")
    if K != Kb:
        raise ValueError(f"b_codes: rows of {Kb} values, a_codes of {K}")
    if out is not None:
        _matrix(out, "out")
        _need(out, "out", _ELEMS, 0)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {(M, N)}")
    dev = _dev(a_codes, a_scales, b_codes, b_scales, out)
    if out is None:
        _dtype_code(dtype)
        out = torch.empty((M, N), dtype=dtype, device=dev)
    with torch.cuda.device(dev):
        _check("mxfp4_matmul", library().mxfp4_matmul(
            _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), M, N, K, _ptr(out),
            DTYPES[out.dtype], N, _stream(dev)))
    return out


class _Linear(torch.autograd.Function):
    """y = Q(x) Q(w)^T, with Q along the dimension that is summed over; the
    backward products round dy, w and x along theirs, so gradients are those of
    the products with the rounding passed straight through.  Of x, only the 4-bit
    payload that dW needs is kept."""

    @staticmethod
    def forward(ctx, x, w):
        y = mxfp4_matmul(*mxfp4_quantize(x), *mxfp4_quantize(w), dtype=x.dtype)
        kept = mxfp4_quantize(x, transpose=True) if ctx.needs_input_grad[1] else (None, None)
        ctx.save_for_backward(w if ctx.needs_input_grad[0] else None, *kept)
        ctx.kinds = x.dtype, w.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        w, xc, xs = ctx.saved_tensors
        dx = dw = None
        if w is not None:
            dx = mxfp4_matmul(*mxfp4_quantize(dy), *mxfp4_quantize(w, transpose=True), dtype=ctx.kinds[0])
        if xc is not None:
            dw = mxfp4_matmul(*mxfp4_quantize(dy, transpose=True), xc, xs, dtype=ctx.kinds[1])
        return dx, dw


def mxfp4_linear(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """x [..., in] times weight [out, in] transposed, in x's type, with both
    operands of the forward and of the two backward products rounded to MXFP4 in
    blocks along the dimension they sum over.  Differentiable in both."""
    _matrix(weight, "weight")
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a torch.Tensor with at least one dimension")
    if x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x: last dimension {x.shape[-1]}, weight's {weight.shape[1]}")
    _matrix(x.reshape(-1, x.shape[-1]) if x.dim() != 2 else x, "x")
    _dev(x, weight)
    y = _Linear.apply(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), weight)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], weight.shape[0])
