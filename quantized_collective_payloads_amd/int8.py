"""The INT8 payload with one scale per row (a token, an output channel), its products
on the matrix cores, and a linear layer that keeps its input in 8 bits for the
backward pass (int8_* of include/qcp.h).

A payload of `rows` rows of n values is a pair (codes, scales): uint8 [rows, P] in
two's complement, with P = n rounded up to whole 128s, and float32 [rows].  Both begin at
16 bytes: rows of a larger payload at multiples of 4 are payloads themselves.

As in mxfp4.py, each function first asks what every valid call answers with yes and
goes through the checks that name the fault only where the answer is no.
"""
from __future__ import annotations

import torch
from torch.autograd.forward_ad import unpack_dual

from . import DTYPES, _dev, _enqueue, _F32, _need, _U8, library
from .mxfp4 import _matrix, _pad, _result, _same_gpu

_u8, _f32 = torch.uint8, torch.float32
_HALF = (torch.float16, torch.bfloat16)
_UNSLICED = 63 * 128              # slices of K begin at 64 stages of 128
_FARTHEST = 1 << 23               # elements between the rows that the mixed product takes


def _payload(codes, scales, what: str):
    """(rows, padded row length, GPU) of a payload after checking its two tensors;
    the GPU is -1 for CPU tensors."""
    try:
        (rows, P), shape, index = codes.shape, scales.shape, codes.get_device()
        if (codes.dtype is _u8 and scales.dtype is _f32 and P % 128 == 0 and shape == (rows,)
                and index == scales.get_device() and codes.is_contiguous() and scales.is_contiguous()):
            return rows, P, index
    except (AttributeError, ValueError):
        pass
    _need(codes, f"{what}codes", _U8, 0)
    _need(scales, f"{what}scales", _F32, 0)
    if codes.dim() != 2:
        raise ValueError(f"{what}codes: {codes.dim()} dimensions, expected 2")
    if codes.shape[1] % 128:
        raise ValueError(f"{what}codes: rows of {codes.shape[1]} bytes, expected a multiple of 128")
    if tuple(scales.shape) != (codes.shape[0],):
        raise ValueError(f"{what}scales: shape {tuple(scales.shape)} for codes of {tuple(codes.shape)}, "
                         f"expected {(codes.shape[0],)}")
    _dev(codes, scales)
    raise ValueError(f"{what}codes: not a payload")


def _columns(P: int, cols: int, what: str = ""):
    if cols < 0 or _pad(cols) != P:
        raise ValueError(f"{what}codes: rows of {P} values for {cols} columns")


def _rows_of(x):
    """x with its elements side by side along rows that do not overlap, and how far
    apart they are."""
    rows, cols = x.shape
    if x.is_contiguous():
        return x, cols
    if x.stride(1) == 1 and (x.stride(0) >= cols or rows == 1):
        return x, x.stride(0) if rows > 1 else cols
    return x.contiguous(), cols


def int8_quantize(x: torch.Tensor, codes=None, scales=None):
    """The payload (codes, scales) of a 2-D fp16/bf16/fp32 GPU tensor.  Rows may lie any
    distance apart; other strides are copied first.  Caller-supplied `codes` (uint8) and
    `scales` (float32) must be contiguous and of the payload's shape."""
    if type(x) is not torch.Tensor or x.dim() != 2 or x.dtype not in DTYPES:
        _matrix(x, "x")
    rows, cols = x.shape
    x, ld = _rows_of(x)
    P, index = _pad(cols), x.get_device()
    if codes is not None or scales is not None:
        for t, what, kinds, shape in ((codes, "codes", _U8, (rows, P)), (scales, "scales", _F32, (rows,))):
            if t is not None:
                _need(t, what, kinds, 0)
                if tuple(t.shape) != shape:
                    raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
                _same_gpu(index, x, t)
    if index < 0:
        _dev(x)
    if codes is None:
        codes = x.new_empty((rows, P), dtype=_u8)
    if scales is None:
        scales = x.new_empty(rows, dtype=_f32)
    _enqueue("int8_quantize", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, ld, codes.data_ptr(),
             scales.data_ptr())
    return codes, scales


def int8_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int, dtype=torch.bfloat16, out=None):
    """The [rows, cols] values that a payload stands for, rounded once to `dtype`."""
    rows, P, index = _payload(codes, scales, "")
    _columns(P, cols)
    y = _result(out, rows, cols, dtype, codes)
    if index < 0 or out is not None:
        _same_gpu(index, codes, y)
    _enqueue("int8_dequantize", index, codes.data_ptr(), scales.data_ptr(), rows, cols, y.data_ptr(),
             DTYPES[y.dtype], cols)
    return y


def int8_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                dtype=torch.bfloat16, out=None):
    """A B^T for the payloads of A [M, K] and B [N, K]: [M, N] in `dtype`.  The sums over K
    (up to 130944) are exact."""
    M, K, index = _payload(a_codes, a_scales, "a_")
    N, Kb, other = _payload(b_codes, b_scales, "b_")
    if K != Kb:
        raise ValueError(f"b_codes: rows of {Kb} values, a_codes of {K}")
    c = _result(out, M, N, dtype, a_codes)
    if index < 0 or index != other or out is not None:
        _same_gpu(index, a_codes, b_codes, c)
    _multiply(index, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), M, N, K, c)
    return c


def _scratch(name: str, like, *sizes):
    """(scratch memory or None, its address, its bytes) for a product."""
    work = getattr(library(), name)(*sizes)
    if work <= 0:
        return None, None, 0
    t = like.new_empty(work, dtype=_u8)
    return t, t.data_ptr(), work


def _multiply(index, a, sa, b, sb, M, N, K, c):
    """The product into c; scratch memory is asked for only where the library may have a use
    for it, which it never has for rows of up to _UNSLICED codes."""
    t, at, size = _scratch("qcp_int8_matmul_work", c, M, N, K) if K > _UNSLICED else (None, None, 0)
    _enqueue("int8_matmul", index, a, sa, b, sb, M, N, K, c.data_ptr(), DTYPES[c.dtype], N, at, size)


def int8_matmul_mixed(a: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, cols: int,
                      transpose: bool = False, dtype=None, out=None):
    """A X for a 2-D fp16 or bf16 tensor A [M, K] (with `transpose`, `a` is [K, M] and A its
    transpose) and the payload of X [K, cols], read in a's type: [M, cols] in `dtype`,
    which is a's (the default) or float32, accumulated in fp32.  Rows of `a` up to 2^23 elements
    apart, and those of a transposed view, are read where they are; other strides, and rows
    that are farther apart or longer, are copied.  cols <= 2^24."""
    if type(a) is not torch.Tensor or a.dim() != 2 or a.dtype not in _HALF:
        _matrix(a, "a")
        if a.dtype not in _HALF:
            raise ValueError(f"a: dtype {a.dtype}, expected {' or '.join(map(str, _HALF))}")
    K, P, index = _payload(codes, scales, "")
    _columns(P, cols)
    M = a.shape[1 if transpose else 0]
    if a.shape[0 if transpose else 1] != K:
        raise ValueError(f"a: shape {tuple(a.shape)}{' (transposed)' if transpose else ''} for a payload of {K} rows")
    dtype = (a.dtype if dtype is None else dtype) if out is None else out.dtype
    if dtype not in (a.dtype, _f32):
        raise ValueError(f"dtype {dtype}, expected {a.dtype} or {_f32}")
    c = _result(out, M, cols, dtype, codes)
    if index < 0 or a.get_device() != index or out is not None:
        _same_gpu(index, codes, a, c)
    _mixed(index, a, codes.data_ptr(), scales.data_ptr(), M, cols, K, transpose, c)
    return c


def _mixed(index, a, codes, scales, M, N, K, transpose, c):
    if not a.is_contiguous() and a.stride(0) == 1 and a.shape[0] <= a.stride(1) <= _FARTHEST:
        a, transpose = a.t(), not transpose
    a, lda = _rows_of(a)
    if lda > _FARTHEST:
        # packed, along the dimension that is short enough (both are longer in no tensor)
        if a.shape[1] > _FARTHEST:
            a, transpose = a.t(), not transpose
        a, lda = a.contiguous(), a.shape[1]
    first, transpose = a.data_ptr(), 1 if transpose else 0
    t, at, size = _scratch("qcp_int8_mixed_work", c, M, N, K, transpose,
                           1 if first % 16 == 0 and lda % 8 == 0 and lda <= 1 << 22 else 0)
    _enqueue("int8_matmul_mixed", index, first, DTYPES[a.dtype], lda, transpose, codes, scales, M, N, K, c.data_ptr(),
             DTYPES[c.dtype], N, at, size)


def _quantized(index, x):
    """The payload of a contiguous matrix in one buffer: its codes, then its scales."""
    rows, cols = x.shape
    buffer = x.new_empty(rows * (_pad(cols) + 4), dtype=_u8)
    _enqueue("int8_quantize", index, x.data_ptr(), DTYPES[x.dtype], rows, cols, cols, *_at(buffer, rows, cols))
    return buffer


def _at(buffer, rows, cols):
    base = buffer.data_ptr()
    return base, base + rows * _pad(cols)


def _product(index, x, qx, w, O):
    """The product of x's payload, held in qx, and that at the addresses w."""
    T, I = x.shape
    y = x.new_empty((T, O))
    _multiply(index, *_at(qx, T, I), *w, T, O, _pad(I), y)
    return y


def _frozen_product(index, x, codes, scales):
    """The product of x's payload and a given one; for few rows in one launch."""
    (T, I), O = x.shape, codes.shape[0]
    if T <= 8 and library().qcp_int8_linear_rows_fit(T, O, I):
        y = x.new_empty((T, O))
        _enqueue("int8_linear_rows", index, x.data_ptr(), DTYPES[x.dtype], T, I, I, codes.data_ptr(), scales.data_ptr(),
                 O, y.data_ptr(), O)
        return y
    return _product(index, x, _quantized(index, x), (codes.data_ptr(), scales.data_ptr()), O)


def _backward(index, dy, payload, rows, cols, transpose, dtype):
    """dy times a payload, or its transpose times it, in `dtype`."""
    M = dy.shape[1 if transpose else 0]
    c = dy.new_empty((M, cols), dtype=dtype if dtype in (dy.dtype, _f32) else _f32)
    _mixed(index, dy, *payload, M, cols, rows, transpose, c)
    return c if c.dtype is dtype else c.to(dtype)


# Autograd accumulates a leaf's gradients on the stream on which a graph first reached the leaf,
# for as long as a graph that reaches it lives.  Where that is the default stream, a backward pass
# in a capture that gives the leaf a gradient makes the default stream wait for the capture, which
# no capture allows and the process may not survive.  Torch does not tell a leaf's stream.  So the
# layer notes its own stream at the leaves next to it and at those behind up to _BEHIND operators
# with one input (0.7 us of a forward call of 25), and its backward pass refuses such a capture for
# every noted leaf before it.  A leaf that only other operators have reached is not noted.
_FIRST_STREAM = "int8_linear: stream of the first graph"
_BEHIND = 8
_Leaf = torch._C._functions.AccumulateGrad


def _near_leaves(node):
    """What autograd keeps of each leaf near a node while a graph that reaches the leaf lives."""
    found = []
    for n, _ in node.next_functions:
        for _ in range(1 + _BEHIND):
            if n is None:
                break
            if type(n) is _Leaf:
                found.append(n)
                break
            up = [m for m, _ in n.next_functions if m is not None]
            n = up[0] if len(up) == 1 else None
    return found


def _leaves(node):
    """The same of all leaves before a node."""
    found, seen, todo = [], set(), [node]
    while todo:
        for n, _ in todo.pop().next_functions:
            if n is not None and n not in seen:
                seen.add(n)
                (found if type(n) is _Leaf else todo).append(n)
    return found


def _receives(leaf):
    """Whether the backward pass that runs gives a leaf a gradient."""
    try:
        return torch._C._will_engine_execute_node(leaf)
    except RuntimeError:                           # what autograd.grad says of the leaves that it was asked for
        return True


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index) if index >= 0 else -1


def _captured(index):
    return index >= 0 and torch.cuda.is_current_stream_capturing()


def _refuse_leaves_of_the_default_stream(node, index):
    if _captured(index) and any(n.metadata.get(_FIRST_STREAM) == 0 and _receives(n) for n in _leaves(node)):
        raise RuntimeError("int8_linear: a backward pass is captured while a graph of the same leaves, recorded on the "
                           "default stream, lives: free its outputs first, or record it on another stream")


class _Linear(torch.autograd.Function):
    """y = Q(x) Q(w)^T.  The payload of x, which the forward product needs, is also all that
    is kept of x: 8 bits a value; that of w is kept for dx.  The backward products read
    them in dy's type: dx = dy Q(w), dw = dy^T Q(x), the gradients of the product with the
    rounding to INT8 passed straight through, up to a rounding of each value to 16 bits."""

    @staticmethod
    def forward(ctx, x, w):
        index, (T, I), O = x.get_device(), x.shape, w.shape[0]
        need_x, need_w = ctx.needs_input_grad
        qx, qw = _quantized(index, x), _quantized(index, w)
        y = _product(index, x, qx, _at(qw, O, I), O)
        ctx.save_for_backward(qx if need_w else None, qw if need_x else None)
        ctx.sizes, ctx.kinds = (T, I, O), (x.dtype, w.dtype)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        qx, qw = ctx.saved_tensors
        T, I, O = ctx.sizes
        index, dx, dw = dy.get_device(), None, None
        _refuse_leaves_of_the_default_stream(ctx, index)
        if qw is not None:
            dx = _backward(index, dy, _at(qw, O, I), O, I, False, ctx.kinds[0])
        if qx is not None:
            dw = _backward(index, dy, _at(qx, T, I), T, I, True, ctx.kinds[1])
        return dx, dw


class _FrozenLinear(torch.autograd.Function):
    """The same on a weight that is a payload: a gradient for x alone, and nothing of x is kept."""

    @staticmethod
    def forward(ctx, x, codes, scales):
        y = _frozen_product(x.get_device(), x, codes, scales)
        ctx.save_for_backward(codes, scales)
        ctx.sizes = (x.shape[1], codes.shape[0])
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        codes, scales = ctx.saved_tensors
        I, O = ctx.sizes
        _refuse_leaves_of_the_default_stream(ctx, dy.get_device())
        dx = _backward(dy.get_device(), dy, (codes.data_ptr(), scales.data_ptr()), O, I, False, dy.dtype)
        return dx, None, None


def int8_linear(x: torch.Tensor, weight) -> torch.Tensor:
    """x [..., in] (fp16 or bf16) times weight [out, in] transposed, in x's type, with x
    rounded to INT8 by tokens and the weight by output channels.

    weight   a 2-D fp16/bf16/fp32 tensor, quantized at every call; or a payload (codes,
             scales) of int8_quantize, made once (serving, frozen weights), or (codes,
             scales, in): a payload's rows are whole 128s, and only where it is told does
             the layer know an x of another length within the same 128

    in <= 130944.  Differentiable in x and in a weight tensor, backwards, with the rounding to
    INT8 passed straight through.  The backward products read the payloads in the gradient's
    type, code * scale rounded to it, where the forward product takes it as it is; under fp16,
    weights above 65504 are infinite there.

    What waits for the backward pass: of x its payload, in (whole 128s) + 4 bytes a token, if
    the weight needs a gradient; of a weight tensor its payload, as much an output channel, if
    x does.  A layer in 16 bits holds 2 in bytes a token and refers to its weight: with fewer
    tokens than output channels this one holds more.

    A forward-mode tangent raises NotImplementedError.  A captured backward pass raises
    RuntimeError if it gives a gradient to a leaf of which autograd still holds a graph that
    the layer recorded on the default stream, and if the layer saw the leaf directly or behind
    up to 8 operators with one input.  Torch may end the process there, as under its own
    operators, and for leaves that the layer has not seen."""
    frozen = isinstance(weight, (tuple, list))
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a torch.Tensor with at least one dimension")
    if frozen:
        if len(weight) not in (2, 3) or (len(weight) == 3 and not isinstance(weight[2], int)):
            raise ValueError("weight: expected a tensor or a payload (codes, scales) or (codes, scales, in)")
        parts = tuple(weight[:2])
        O, P, _ = _payload(*parts, "weight ")
        if len(weight) == 3:
            _columns(P, weight[2], "weight ")
            if x.shape[-1] != weight[2]:
                raise ValueError(f"x: last dimension {x.shape[-1]}, weight's {weight[2]}")
        if P != _pad(x.shape[-1]):
            raise ValueError(f"x: last dimension {x.shape[-1]}, weight rows of {P} values")
    else:
        _matrix(weight, "weight")
        O = weight.shape[0]
        if x.shape[-1] != weight.shape[1]:
            raise ValueError(f"x: last dimension {x.shape[-1]}, weight's {weight.shape[1]}")
        parts = (weight,)
    # flatten, where reshape(-1, 0) would not know how many rows
    x2 = x if x.dim() == 2 else x.flatten(0, -2) if x.dim() > 2 else x.unsqueeze(0)
    if x2.dtype not in _HALF:
        raise ValueError(f"x: dtype {x2.dtype}, expected {' or '.join(map(str, _HALF))}")
    _same_gpu(x.get_device(), x, *parts)
    x2 = x2.contiguous()
    if not frozen:
        parts = (weight.contiguous(),)
    # a tangent of forward-mode differentiation, which the layer has no rule for, is for
    # autograd to refuse in either mode
    if torch.is_grad_enabled() or any(unpack_dual(t).tangent is not None for t in (x2, *parts)):
        y = (_FrozenLinear if frozen else _Linear).apply(x2, *parts)
        if y.requires_grad:
            stream = _raw_stream(y.get_device())
            for n in _near_leaves(y.grad_fn):
                n.metadata.setdefault(_FIRST_STREAM, stream)
    else:
        index = x2.get_device()
        if frozen:
            y = _frozen_product(index, x2, *parts)
        else:
            qw = _quantized(index, parts[0])
            y = _product(index, x2, _quantized(index, x2), _at(qw, O, x2.shape[1]), O)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], O)
