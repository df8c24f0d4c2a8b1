"""AdamW over the tensors of an optimizer shard (adamw_step of include/qcp.h).

The shard's owner runs it between the gradient reduce-scatter and the weight
all-gather: gradients come as the fp32 sums of dequant_reduce_requant or in 16
bits, the weights are fp32, and a 16-bit copy of them can be written on the way.
The moments of all tensors live in two flat buffers, in fp32 or as blockwise
E4M3 codes (m and sqrt(v), one power-of-two fp32 scale per G), which
dequantize_blockwise and the collectives take as they are.
"""
from __future__ import annotations

import ctypes

import torch

from . import (DTYPES, FORMATS, _check, _check_n_G, _dev, _ELEMS, _F32, _need, _ptr, _stream, _U8,
               library, n_blocks)

_STATES = {"f32": DTYPES[torch.float32], "e4m3": FORMATS["e4m3"]}
_COPIES = (torch.float16, torch.bfloat16)


def _list(ts, what: str):
    if isinstance(ts, torch.Tensor) or not isinstance(ts, (list, tuple)):
        raise ValueError(f"{what}: expected a list of tensors")
    return list(ts)


class AdamW:
    """The tensors that adamw_step updates, and their moments.

    params   list of contiguous fp32 GPU tensors; their storage is updated in place
    copies   None, or one fp16 or bf16 tensor per parameter (all of one type),
             which receives the rounded parameter at every step
    state    "e4m3" (8-bit moments) or "f32"
    G        block size of the 8-bit moments (in both states a tensor's moments
             begin at a multiple of it)
    m, v, m_scales, v_scales   the moments of an earlier run; zeros by default.
             Flat, tensor i at offsets[i]; n_state elements and, for "e4m3",
             uint8 codes with n_state/G scales.

    The tensors must keep their storage: a step on a parameter that was given
    another one since raises ValueError.
    """

    def __init__(self, params, copies=None, state: str = "e4m3", G: int = 128, m=None, v=None,
                 m_scales=None, v_scales=None):
        self.params = _list(params, "params")
        if not self.params:
            raise ValueError("params: empty list")
        if state not in _STATES:
            raise ValueError(f"state {state!r} is not one of {', '.join(map(repr, _STATES))}")
        _check_n_G(0, G)
        for i, p in enumerate(self.params):
            _need(p, f"params[{i}]", _F32, 0)
        self.copies = None if copies is None else _list(copies, "copies")
        if self.copies is not None:
            if len(self.copies) != len(self.params):
                raise ValueError(f"copies: {len(self.copies)} tensors for {len(self.params)} parameters")
            kinds = _COPIES if not self.copies else (self.copies[0].dtype,)
            for i, (c, p) in enumerate(zip(self.copies, self.params)):
                _need(c, f"copies[{i}]", _COPIES, p.numel())
                _need(c, f"copies[{i}]", kinds, p.numel())
        self.state, self.G = state, G
        self.sizes = [p.numel() for p in self.params]
        self.offsets, at = [], 0
        for n in self.sizes:
            self.offsets.append(at)
            at += n_blocks(n, G) * G
        self.n_state = at
        eight = state == "e4m3"
        kind, ns = (_U8 if eight else _F32), (at // G if eight else 0)
        for t, what, dt, n in ((m, "m", kind, at), (v, "v", kind, at),
                               (m_scales, "m_scales", _F32, ns), (v_scales, "v_scales", _F32, ns)):
            if t is not None:
                _need(t, what, dt, n)
        self.device = _dev(*self.params, *(self.copies or ()), m, v, m_scales, v_scales)

        def own(t, n, dt):
            return torch.zeros(n, dtype=dt[0], device=self.device) if t is None else t
        self.m, self.v = own(m, at, kind), own(v, at, kind)
        self.m_scales = own(m_scales, ns, _F32) if eight else None
        self.v_scales = own(v_scales, ns, _F32) if eight else None

        n = len(self.params)
        self._at = self._pointers()
        self._params = (ctypes.c_void_p * n)(*self._at)
        self._copies = None if self.copies is None else (ctypes.c_void_p * n)(*(c.data_ptr() for c in self.copies))
        self._copy_type = DTYPES[self.copies[0].dtype] if self.copies else 0
        self._sizes = (ctypes.c_int64 * n)(*self.sizes)
        self._offsets = (ctypes.c_int64 * n)(*self.offsets)
        self._table = ctypes.c_void_p * n
        self._written = self.params + (self.copies or [])

    def _pointers(self):
        return [p.data_ptr() for p in self.params]


def adamw_step(optimizer: AdamW, grads, step: int, lr: float, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale=None, seed: int = 0) -> None:
    """One AdamW step, in place.

    grads        one contiguous GPU tensor per parameter, of its size, all fp16,
                 bf16 or fp32
    step         1 for the first step
    grad_scale   None, or a one-element fp32 GPU tensor that multiplies every
                 gradient; it is read on the device when the step runs
    seed         of the 8-bit moments' stochastic rounding: the same seed, step
                 and inputs give the same bytes
    """
    o = optimizer
    grads = _list(grads, "grads")
    if len(grads) != len(o.sizes):
        raise ValueError(f"grads: {len(grads)} tensors for {len(o.sizes)} parameters")
    dev, kind = o.device, getattr(grads[0], "dtype", None)
    if kind not in DTYPES:
        _need(grads[0], "grads[0]", _ELEMS, 0)
    index = dev.index
    at = []
    for i, (g, n) in enumerate(zip(grads, o.sizes)):
        if (type(g) is not torch.Tensor or g.dtype is not kind or g.numel() != n
                or not g.is_contiguous() or g.get_device() != index):
            _need(g, f"grads[{i}]", (kind,), n)
            if g.numel() != n:
                raise ValueError(f"grads[{i}]: holds {g.numel()} elements, the parameter {n}")
            _dev(o.m, g)
        at.append(g.data_ptr())
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", _F32, 1)
        _dev(o.m, grad_scale)
    if o._pointers() != o._at:
        raise ValueError("params: a parameter was given another storage since the AdamW was made")
    with torch.cuda.device(dev):
        _check("adamw_step", library().adamw_step(
            o._params, o._table(*at), o._copies, o._sizes, o._offsets, len(at), DTYPES[kind],
            o._copy_type, _STATES[o.state], _ptr(o.m), _ptr(o.m_scales), _ptr(o.v),
            _ptr(o.v_scales), o.n_state, o.G, step, lr, beta1, beta2, eps, weight_decay,
            _ptr(grad_scale), seed & 0xFFFFFFFFFFFFFFFF, _stream(dev)))
    torch.autograd.graph.increment_version(o._written)
