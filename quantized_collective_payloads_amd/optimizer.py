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
from array import array

import torch

from . import (DTYPES, FORMATS, _check, _check_n_G, _dev, _ELEMS, _enqueue, _F32, _need, _U8, library, n_blocks)

_STATES = {"f32": DTYPES[torch.float32], "e4m3": FORMATS["e4m3"]}
_COPIES = (torch.float16, torch.bfloat16)
_MAX_TENSORS = 1024                               # QCP_ADAMW_MAX_TENSORS


def _list(ts, what: str):
    if isinstance(ts, torch.Tensor) or not isinstance(ts, (list, tuple)):
        raise ValueError(f"{what}: expected a list of tensors")
    return list(ts)


class AdamW:
    """The tensors that adamw_step updates, and their moments.

    params   list of contiguous fp32 GPU tensors; their storage is updated in place
    copies   None, or one fp16 or bf16 tensor per parameter (all of one type),
             which receives the rounded parameter at every step
    state    "e4m3" (8-bit moments, rounded at random: the default) or "f32"
    G        block size of the 8-bit moments (in both states a tensor's moments
             begin at a multiple of it)
    m, v, m_scales, v_scales   the moments of an earlier run; zeros by default.
             Flat, tensor i at offsets[i]; n_state elements and, for "e4m3",
             uint8 codes with n_state/G scales.

    The tensors must keep their storage: a step after a parameter, a copy or a
    moment was given another one, or one of another size, raises ValueError.  The
    attributes are read-only.
    """

    params = property(lambda self: self._params)
    copies = property(lambda self: self._copies)
    state = property(lambda self: self._state)
    G = property(lambda self: self._G)
    m = property(lambda self: self._m)
    v = property(lambda self: self._v)
    m_scales = property(lambda self: self._m_scales)
    v_scales = property(lambda self: self._v_scales)
    sizes = property(lambda self: self._sizes)
    offsets = property(lambda self: self._offsets)
    n_state = property(lambda self: self._n_state)

    def __init__(self, params, copies=None, state: str = "e4m3", G: int = 128, m=None, v=None,
                 m_scales=None, v_scales=None):
        params = _list(params, "params")
        if not params:
            raise ValueError("params: empty list")
        if state not in _STATES:
            raise ValueError(f"state {state!r} is not one of {', '.join(map(repr, _STATES))}")
        _check_n_G(0, G)
        for i, p in enumerate(params):
            _need(p, f"params[{i}]", _F32, 0)
        if copies is not None:
            copies = _list(copies, "copies")
            if len(copies) != len(params):
                raise ValueError(f"copies: {len(copies)} tensors for {len(params)} parameters")
            for i, (c, p) in enumerate(zip(copies, params)):
                _need(c, f"copies[{i}]", _COPIES, p.numel())
                _need(c, f"copies[{i}]", (copies[0].dtype,), p.numel())
        sizes, offsets, at = [p.numel() for p in params], [], 0
        for n in sizes:
            offsets.append(at)
            at += n_blocks(n, G) * G
        eight = state == "e4m3"
        kind, ns = (_U8 if eight else _F32), (at // G if eight else 0)
        for t, what, dt, n in ((m, "m", kind, at), (v, "v", kind, at),
                               (m_scales, "m_scales", _F32, ns), (v_scales, "v_scales", _F32, ns)):
            if t is not None:
                _need(t, what, dt, n)
        device = _dev(*params, *(copies or ()), m, v, m_scales, v_scales)

        def own(t, n, dt):
            return torch.zeros(n, dtype=dt[0], device=device) if t is None else t
        self._state, self._G, self._n_state = state, G, at
        self._params, self._copies = tuple(params), None if copies is None else tuple(copies)
        self._sizes, self._offsets = tuple(sizes), tuple(offsets)
        self._m, self._v = own(m, at, kind), own(v, at, kind)
        self._m_scales = own(m_scales, ns, _F32) if eight else None
        self._v_scales = own(v_scales, ns, _F32) if eight else None

        # what every step passes on, made once: the tensors above stay alive with it.  Every
        # step asks whether they still lie there and whether their storages (the distinct
        # ones) still have their sizes: one that shrank may lie where it did
        n = len(params)
        moments = tuple(t for t in (self._m, self._v, self._m_scales, self._v_scales) if t is not None)
        self._tensors = (*params, *(copies or ()), *moments)
        self._index, self._at = device.index, [t.data_ptr() for t in self._tensors]
        self._storages = tuple({s._cdata: s for s in map(torch.Tensor.untyped_storage, self._tensors)}.values())
        self._bytes = [s.nbytes() for s in self._storages]
        table = ctypes.c_void_p * n
        self._arrays = (table(*self._at[:n]), None if copies is None else table(*(c.data_ptr() for c in copies)),
                        (ctypes.c_int64 * n)(*sizes), (ctypes.c_int64 * n)(*offsets))
        self._bases = tuple(None if a is None else ctypes.addressof(a) for a in self._arrays)
        self._copy_type = DTYPES[copies[0].dtype] if copies else 0
        self._moments = (self._m.data_ptr(), self._m_scales.data_ptr() if eight else None,
                         self._v.data_ptr(), self._v_scales.data_ptr() if eight else None)

    def _moved(self):
        """The names of the tensors that no longer have the storage they were given with."""
        names = [f"params[{i}]" for i in range(len(self._params))]
        names += [f"copies[{i}]" for i in range(len(self._copies or ()))]
        names += ["m", "v", "m_scales", "v_scales"][:len(self._tensors) - len(names)]
        size = {s._cdata: n for s, n in zip(self._storages, self._bytes)}
        return [name for name, t, at in zip(names, self._tensors, self._at)
                if t.data_ptr() != at or t.untyped_storage().nbytes() != size.get(t.untyped_storage()._cdata)]


_numel, _data_ptr, _get_device = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.get_device
_is_contiguous, _nbytes = torch.Tensor.is_contiguous, torch.UntypedStorage.nbytes


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

    Captured into a graph, a step replays with the step number, seed and
    hyperparameters of its capture.
    """
    o = optimizer
    if type(grads) is not list:
        grads = _list(grads, "grads")
    if len(grads) != len(o._sizes):
        raise ValueError(f"grads: {len(grads)} tensors for {len(o._sizes)} parameters")
    index, kind = o._index, getattr(grads[0], "dtype", None)
    # four questions that all valid gradients answer with yes; the loop names the fault
    try:
        good = (kind in DTYPES and tuple(map(_numel, grads)) == o._sizes and all(map(_is_contiguous, grads))
                and {g.dtype for g in grads} == {kind} and set(map(_get_device, grads)) == {index})
    except (AttributeError, TypeError):
        good = False
    if not good:
        for i, (g, n) in enumerate(zip(grads, o._sizes)):
            _need(g, f"grads[{i}]", (kind,) if kind in DTYPES else _ELEMS, n)
            if g.numel() != n:
                raise ValueError(f"grads[{i}]: holds {g.numel()} elements, the parameter {n}")
            _dev(o._m, g)
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", _F32, 1)
        _dev(o._m, grad_scale)
    if list(map(_data_ptr, o._tensors)) != o._at or list(map(_nbytes, o._storages)) != o._bytes:
        raise ValueError(f"{', '.join(o._moved())}: given another storage since the AdamW was made")
    params, copies, sizes, offsets = o._bases
    m, ms, v, vs = o._moments
    at = array("Q", list(map(_data_ptr, grads)))              # a third of the time of a ctypes array
    table = at.buffer_info()[0]
    n, scale = len(grads), None if grad_scale is None else grad_scale.data_ptr()
    rest = (DTYPES[kind], o._copy_type, _STATES[o._state], m, ms, v, vs, o._n_state, o._G, step, lr, beta1, beta2,
            eps, weight_decay, scale)
    if n > _MAX_TENSORS:                                      # several calls: all of them or none
        _check("adamw_step", library().qcp_adamw_check(params, table, copies, sizes, offsets, n, *rest))
    for first in range(0, n, _MAX_TENSORS):
        k = 8 * first
        _enqueue("adamw_step", index, params + k, table + k, copies and copies + k, sizes + k, offsets + k,
                 min(_MAX_TENSORS, n - first), *rest, seed & 0xFFFFFFFFFFFFFFFF)
    torch.autograd.graph.increment_version(o._tensors)
