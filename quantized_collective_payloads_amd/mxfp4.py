"""The MXFP4 payload (4.25 bits per weight), its product on the matrix cores, and
a linear layer whose three products run on it (mxfp4_* of include/qcp.h).

A payload of `lines` rows of n values is a pair (codes, scales): uint8
[lines, P/2] and uint8 [lines, P/32] with P = n rounded up to whole 128s.

The kernels for small sizes take a few microseconds, so each function first asks
what every valid call answers with yes, in as few questions as it can, and goes
through the checks that name the fault only where the answer is no.
"""
from __future__ import annotations

import torch
from torch.autograd.forward_ad import unpack_dual

from . import (DTYPES, _dev, _dtype_code, _ELEMS, _enqueue, _need, _U8, library)

_u8 = torch.uint8
_UNSLICED = 62 * 128              # 31 stages of 256: slices of K begin at 32


def mxfp4_padded(n: int) -> int:
    """Values that a payload row of n values holds: n rounded up to whole 128s."""
    p = int(library().qcp_mxfp4_padded(n))
    if p < 0:
        raise ValueError(f"row length {n} is negative or too large")
    return p


def _pad(n: int) -> int:
    return (n + 127) // 128 * 128


def _matrix(x, what: str):
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{what}: expected a torch.Tensor, got {type(x).__name__}")
    if x.dtype not in DTYPES:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {' or '.join(map(str, _ELEMS))}")
    if x.dim() != 2:
        raise ValueError(f"{what}: {x.dim()} dimensions, expected 2")
    return x


def _payload(codes, scales, what: str):
    """(lines, padded row length, GPU) of a payload after checking its two tensors;
    the GPU is -1 for CPU tensors."""
    try:
        (lines, cb), shape, index = codes.shape, scales.shape, codes.get_device()
        if (codes.dtype is _u8 and scales.dtype is _u8 and cb % 64 == 0 and shape == (lines, cb // 16)
                and index == scales.get_device() and codes.is_contiguous() and scales.is_contiguous()):
            return lines, 2 * cb, index
    except (AttributeError, ValueError):
        pass
    for t, name, unit in ((codes, "codes", 64), (scales, "scales", 4)):
        _need(t, f"{what}{name}", _U8, 0)
        if t.dim() != 2:
            raise ValueError(f"{what}{name}: {t.dim()} dimensions, expected 2")
        if t.shape[1] % unit:
            raise ValueError(f"{what}{name}: rows of {t.shape[1]} bytes, expected a multiple of {unit}")
    if scales.shape != (codes.shape[0], codes.shape[1] // 16):
        raise ValueError(f"{what}scales: shape {tuple(scales.shape)} for codes of {tuple(codes.shape)}, "
                         f"expected {(codes.shape[0], codes.shape[1] // 16)}")
    _dev(codes, scales)
    raise ValueError(f"{what}codes: not a payload")


def _result(out, rows: int, cols: int, dtype, like):
    """The output tensor: the caller's after its checks, or a new one."""
    if out is None:
        if dtype not in DTYPES:
            _dtype_code(dtype)
        return like.new_empty((rows, cols), dtype=dtype)
    _matrix(out, "out")
    _need(out, "out", _ELEMS, 0)
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"out: shape {tuple(out.shape)}, expected {(rows, cols)}")
    return out


def _same_gpu(index: int, *ts):
    """All on GPU `index`; else the fault's name."""
    if index < 0 or any(t.get_device() != index for t in ts):
        _dev(*ts)
        raise ValueError("qcp: tensors on different devices")


def mxfp4_quantize(x: torch.Tensor, transpose: bool = False, codes=None, scales=None):
    """The payload (codes, scales) of a 2-D fp16/bf16/fp32 GPU tensor, or with
    `transpose` of x.t().  Rows may lie any distance apart, and a transposed view
    is read where it is; other strides are copied first.  Caller-supplied `codes`
    and `scales` must be contiguous uint8 of the payload's shape."""
    if type(x) is not torch.Tensor or x.dim() != 2 or x.dtype not in DTYPES:
        _matrix(x, "x")
    rows, cols = x.shape
    ld = cols
    if not x.is_contiguous():
        if x.numel() and x.stride(1) != 1 and cols != 1:
            if x.stride(0) == 1 or rows == 1:
                x, transpose = x.t(), not transpose
                rows, cols = cols, rows
            else:
                x = x.contiguous()
        ld = x.stride(0) if rows > 1 else cols
        if ld < cols:                                # rows that overlap (an expanded tensor)
            x, ld = x.contiguous(), cols
    lines, n = (cols, rows) if transpose else (rows, cols)
    P = _pad(n)
    index = x.get_device()
    for t, what, shape in ((codes, "codes", (lines, P // 2)), (scales, "scales", (lines, P // 32))):
        if t is not None:
            _need(t, what, _U8, 0)
            if tuple(t.shape) != shape:
                raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
            _same_gpu(index, x, t)
    if index < 0:
        _dev(x)
    if codes is None:
        codes = x.new_empty((lines, P // 2), dtype=_u8)
    if scales is None:
        scales = codes.new_empty((lines, P // 32))
    _enqueue("mxfp4_quantize", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, ld, 1 if transpose else 0,
             codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mxfp4_quantize_both(x: torch.Tensor):
    """The payloads of a 2-D fp16/bf16/fp32 GPU tensor and of its transpose, as
    mxfp4_quantize(x) and mxfp4_quantize(x, transpose=True) give them, in one pass."""
    if type(x) is not torch.Tensor or x.dim() != 2 or x.dtype not in DTYPES:
        _matrix(x, "x")
    rows, cols = x.shape
    ld, swap = cols, False
    if not x.is_contiguous():
        if x.numel() and x.stride(1) != 1 and x.stride(0) == 1 and x.stride(1) >= rows:
            x, swap = x.t(), True
            rows, cols = cols, rows
            ld = x.stride(0)
        elif x.stride(1) == 1 and x.stride(0) >= cols:
            ld = x.stride(0)
        else:
            x = x.contiguous()
    index = x.get_device()
    if index < 0:
        _dev(x)
    pc, pr = _pad(cols), _pad(rows)
    codes = x.new_empty((rows, pc // 2), dtype=_u8)
    a = codes, codes.new_empty((rows, pc // 32))
    b = codes.new_empty((cols, pr // 2)), codes.new_empty((cols, pr // 32))
    _enqueue("mxfp4_quantize_both", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, ld, a[0].data_ptr(),
             a[1].data_ptr(), b[0].data_ptr(), b[1].data_ptr())
    return (b, a) if swap else (a, b)


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int, dtype=torch.bfloat16, out=None):
    """The [lines, cols] values that a payload stands for, rounded once to `dtype`."""
    lines, P, index = _payload(codes, scales, "")
    if cols < 0 or _pad(cols) != P:
        raise ValueError(f"codes: rows of {P} values for {cols} columns, expected {mxfp4_padded(cols)}")
    if index < 0 or out is not None:
        _same_gpu(index, codes, *(() if out is None else (_result(out, lines, cols, dtype, codes),)))
    y = _result(out, lines, cols, dtype, codes)
    _enqueue("mxfp4_dequantize", index, codes.data_ptr(), scales.data_ptr(), lines, cols, y.data_ptr(),
             DTYPES[y.dtype], cols)
    return y


def mxfp4_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
                 b_scales: torch.Tensor, dtype=torch.bfloat16, out=None):
    """A B^T for the payloads of A [M, K] and B [N, K]: [M, N] in `dtype`,
    accumulated in fp32 and rounded once."""
    M, K, index = _payload(a_codes, a_scales, "a_")
    N, Kb, other = _payload(b_codes, b_scales, "b_")
    if K != Kb:
        raise ValueError(f"b_codes: rows of {Kb} values, a_codes of {K}")
    if index < 0 or index != other or out is not None:
        _same_gpu(index, a_codes, b_codes, *(() if out is None else (_result(out, M, N, dtype, a_codes),)))
    c = _result(out, M, N, dtype, a_codes)
    _multiply(index, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), M, N, K, c)
    return c


def _multiply(index, a, sa, b, sb, M, N, K, c):
    """The product into c; with scratch memory where the library has a use for it,
    which it never has for rows of up to _UNSLICED values."""
    work = library().qcp_mxfp4_matmul_work(M, N, K) if K > _UNSLICED else 0
    if work:
        scratch = c.new_empty(work, dtype=_u8)
        _enqueue("mxfp4_matmul_sliced", index, a, sa, b, sb, M, N, K, c.data_ptr(), DTYPES[c.dtype], N,
                 scratch.data_ptr(), work)
    else:
        _enqueue("mxfp4_matmul", index, a, sa, b, sb, M, N, K, c.data_ptr(), DTYPES[c.dtype], N)


class _Work:
    """Payloads of one call in one allocation; only their addresses are needed."""

    def __init__(self, like, *shapes):
        at, self.places = 0, []
        for lines, n in shapes:
            P = _pad(n)
            self.places.append((at, at + lines * P // 2))
            at += lines * P // 2 + (lines * P // 32 + 15) // 16 * 16
        self.buffer = like.new_empty(at, dtype=_u8)

    def __getitem__(self, k):
        return _at(self.buffer, self.places[k])


def _at(buffer, place):
    base = buffer.data_ptr()
    return base + place[0], base + place[1]


def _quantize_to(index, x, rows, cols, straight, transposed):
    """The payload of x, of its transpose, or both, to the addresses given."""
    if transposed is None:
        _enqueue("mxfp4_quantize", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, cols, 0, *straight)
    elif straight is None:
        _enqueue("mxfp4_quantize", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, cols, 1, *transposed)
    else:
        _enqueue("mxfp4_quantize_both", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, cols, *straight,
                 *transposed)


def _product(index, a, b, M, N, K, dtype, like):
    c = like.new_empty((M, N), dtype=dtype)
    _multiply(index, *a, *b, M, N, K, c)
    return c


def _linear(x, w, need_x: bool, need_w: bool):
    """(y, the payloads that the gradients asked for need): y = Q(x) Q(w)^T.  Reads x
    and w once for both payloads of each."""
    index, (T, I), O = x.get_device(), x.shape, w.shape[0]
    work, kept = _Work(x, (T, I), (O, I)), None
    if need_x or need_w:
        kept = _Work(x, *([(I, O)] if need_x else []), *([(I, T)] if need_w else []))
    _quantize_to(index, x, T, I, work[0], kept[-1] if need_w else None)
    _quantize_to(index, w, O, I, work[1], kept[0] if need_x else None)
    return _product(index, work[0], work[1], T, O, I, x.dtype, x), kept


class _Linear(torch.autograd.Function):
    """y = Q(x) Q(w)^T, with Q along the dimension that is summed over; the
    backward products round dy, w and x along theirs, so gradients are those of
    the products with the rounding passed straight through.  The forward keeps
    only the 4-bit payloads that the backward needs."""

    @staticmethod
    def forward(ctx, x, w):
        y, kept = _linear(x, w, *ctx.needs_input_grad)
        if kept is not None:
            ctx.save_for_backward(kept.buffer)
            ctx.kinds, ctx.sizes, ctx.places = (x.dtype, w.dtype), (*x.shape, w.shape[0]), kept.places
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        kept, = ctx.saved_tensors
        T, I, O = ctx.sizes
        need_x, need_w = ctx.needs_input_grad
        index, dx, dw = dy.get_device(), None, None
        dy = dy.contiguous()
        work = _Work(dy, *([(T, O)] if need_x else []), *([(O, T)] if need_w else []))
        _quantize_to(index, dy, T, O, work[0] if need_x else None, work[-1] if need_w else None)
        if need_x:
            dx = _product(index, work[0], _at(kept, ctx.places[0]), T, I, O, ctx.kinds[0], dy)
        if need_w:
            dw = _product(index, work[-1], _at(kept, ctx.places[-1]), O, I, T, ctx.kinds[1], dy)
        return dx, dw


def mxfp4_linear(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """x [..., in] times weight [out, in] transposed, in x's type, with both
    operands of the forward and of the two backward products rounded to MXFP4 in
    blocks along the dimension they sum over.  Differentiable in both, backwards; a
    forward-mode tangent raises NotImplementedError."""
    _matrix(weight, "weight")
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a torch.Tensor with at least one dimension")
    if x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x: last dimension {x.shape[-1]}, weight's {weight.shape[1]}")
    # flatten, where reshape(-1, 0) would not know how many rows
    x2 = x if x.dim() == 2 else x.flatten(0, -2) if x.dim() > 2 else x.unsqueeze(0)
    _matrix(x2, "x")
    _same_gpu(x.get_device(), x, weight)
    x2, w = x2.contiguous(), weight.contiguous()
    # without gradients only the product's own payloads: 77 tokens, 520 -> 1032: 26.1 -> 19.7 us.
    # A tangent of forward-mode differentiation, which the layer has no rule for, is for
    # autograd to refuse in either mode
    track = torch.is_grad_enabled() or unpack_dual(x2).tangent is not None or unpack_dual(w).tangent is not None
    y = _Linear.apply(x2, w) if track else _linear(x2, w, False, False)[0]
    return y if x.dim() == 2 else y.view(*x.shape[:-1], weight.shape[0])
