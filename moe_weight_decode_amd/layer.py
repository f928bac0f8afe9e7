"""The layer operators around the routed projections: RMS norm, router, gated
feed-forward half and their backward passes (``include/csf.h``).

Argument marshalling only, as the rest of the binding.  Every function checks
its tensors (device, type, shape, contiguity), allocates its outputs and its
workspace, enqueues on ``stream`` (default: the current one) and returns
without synchronising.  A ``stream`` other than the current one first waits for
the current stream's queued work, since the inputs may come from it and the
outputs' memory is allocated there; work on another stream that uses the
results must wait for ``stream``.  Inputs may be dropped as soon as the call
returns; one that is written again must wait for ``stream`` too.

``bound(function, *args, **kwargs)`` checks and marshals a call once: the
returned object enqueues the same call on the same buffers each time it is
called and returns the same outputs, for decode loops whose buffers stay.  It
goes to the stream that is current when it is called (or to ``stream``, with
the wait above at every call), so it can be bound first and captured in a graph
later; the graph uses its buffers, which live as long as the bound call.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import (CompressedStack, CsfError, MAX_EXPERTS, MXFP4, NVFP4, _check_stack_tensors, _lib, _stream_handle, csf_stack)

BF16, F16, F32 = 0, 1, 2
DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}

EXPORTS = ("csf_rms_norm", "csf_rms_norm_backward_workspace", "csf_rms_norm_backward", "csf_route_workspace",
           "csf_route", "csf_combine_backward", "csf_route_backward", "csf_moe_gated_workspace", "csf_moe_gated",
           "csf_moe_gated_backward")


def declare(lib):
    """ctypes signatures of the layer operators."""
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sp = ctypes.POINTER(csf_stack)
    for name, result, args in (
            ("csf_rms_norm", ctypes.c_int, [i32, vp, vp, vp, i32, i32, vp, vp, i32, i64, f32, vp, vp, vp, vp, vp]),
            ("csf_rms_norm_backward_workspace", i64, [i32, i32]),
            ("csf_rms_norm_backward", ctypes.c_int, [i32, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, i64, vp]),
            ("csf_route_workspace", i64, [i32, i32]),
            ("csf_route", ctypes.c_int, [i32, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp]),
            ("csf_combine_backward", ctypes.c_int, [i32, vp, vp, vp, vp, i32, i32, i32, i64, vp, vp, vp]),
            ("csf_route_backward", ctypes.c_int, [i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]),
            ("csf_moe_gated_workspace", i64, [sp, i32]),
            ("csf_moe_gated", ctypes.c_int, [sp, vp, vp, vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, i64, vp]),
            ("csf_moe_gated_backward", ctypes.c_int, [sp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = result, args
        _functions[name] = fn


class Normed(NamedTuple):
    """Result of ``rms_norm``."""
    out: torch.Tensor                  # [T, D]: the inputs' type, or E4M3 codes (uint8)
    sum: torch.Tensor                  # [T, D]: x + residual (without a residual x itself, not a copy)
    rstd: torch.Tensor                 # float32 [T]
    scales: torch.Tensor | None        # uint8 [T, ceil(D / 32)] (E8M0) with mxfp8


class Routing(NamedTuple):
    """Result of ``route`` (see ``csf_route``)."""
    experts: torch.Tensor              # int32 [T, topk]
    gates: torch.Tensor                # float32 [T, topk]
    expert_start: torch.Tensor         # int32 [E + 1]
    rows: torch.Tensor                 # int32 [T * topk]
    slots: torch.Tensor                # int32 [T, topk]


_functions = {}  # the library's functions by name


class Bound:
    """One checked and marshalled call; calling it enqueues it again, on the
    stream given when it was bound or else on the current one."""
    __slots__ = ("_fn", "_args", "_result", "_name", "_keep", "_dev", "_stream", "_known")

    def __init__(self, name: str, args: tuple, result, keep, dev, stream):
        self._fn, self._name = _functions[name], name
        self._args, self._result, self._keep = args, result, keep
        self._dev, self._stream = dev, stream
        self._known = {_current(dev.index)}  # streams that the tensors' memory waits for when it is freed

    def __call__(self):
        if self._stream is None:
            handle = _current(self._dev.index)
        else:
            handle = _enter(self._stream, self._dev)
        if handle not in self._known:
            self._record(handle)
        status = self._fn(*self._args, handle)
        if status != 0:
            raise CsfError(status, self._name)
        return self._result

    def _record(self, handle):
        """Used on a stream that they were not allocated on, the tensors' memory
        would be handed out again as soon as they are dropped (the inputs of a
        plain call when it returns): it is kept until that stream is done."""
        stream = _stream_of(handle, self._dev)
        inputs, fresh = self._keep
        for t in _tensors((*inputs, *fresh)):
            t.record_stream(stream)
        self._known.add(handle)


# the handle of the current stream, without a Stream object where torch offers that
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _need(where: str, name: str, t, dtypes, dev, numel=None, dim=None, shape=None):
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous {' or '.join(map(str, dtypes))} tensor on {dev}")
    if (numel is not None and t.numel() != numel) or (dim is not None and t.dim() != dim) or (shape is not None and t.shape != shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, which does not match the call")


def _device(where: str, t, name: str):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{where}: {name} must be a GPU tensor")
    return t.device


def _stream_of(handle, dev):
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _enter(stream, dev):
    """The stream's handle; one other than the current stream first waits for that."""
    current = torch.cuda.current_stream(dev)
    handle = _stream_handle(stream, dev)
    if handle != current.cuda_stream:
        _stream_of(handle, dev).wait_stream(current)
    return handle


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _tensors(values):
    """Every tensor among a call's values, a stack's own included."""
    for v in values:
        if isinstance(v, CompressedStack):
            yield from _tensors((v.bases, v.offsets, v.exceptions, v.prefix, v.tile_index))
        elif isinstance(v, torch.Tensor):
            yield v


def _call(name, args, result, dev, inputs, fresh, stream) -> Bound:
    _lib()  # fills _functions
    return Bound(name, args, result, (inputs, fresh), dev, stream)


def _rms_norm(x, weight, residual=None, slots=None, gates=None, eps=1e-6, mxfp8=False, stream=None) -> Bound:
    where = "rms_norm"
    dev = _device(where, x, "x")
    if x.dim() != 2:
        raise ValueError(f"{where}: x must be [T, D]")
    D = x.shape[1]
    if slots is not None:
        _need(where, "x (the experts' outputs)", x, (torch.float32,), dev)
        _need(where, "slots", slots, (torch.int32,), dev, dim=2)
        T, k = slots.shape
        _need(where, "gates", gates, (torch.float32,), dev, shape=(T, k))
        if residual is None:
            raise ValueError(f"{where}: the combination needs the residual")
    else:
        T, k = x.shape[0], 0
        _need(where, "x", x, tuple(DTYPES), dev)
        if gates is not None:
            raise ValueError(f"{where}: gates without slots")
    dtype = x.dtype if residual is None else getattr(residual, "dtype", None)
    if residual is not None:
        _need(where, "residual", residual, tuple(DTYPES) if slots is not None else (x.dtype,), dev, shape=(T, D))
    _need(where, "weight", weight, (torch.float32,), dev, D)
    total = x if residual is None else torch.empty(T, D, dtype=dtype, device=dev)
    out = torch.empty(T, D, dtype=torch.uint8 if mxfp8 else dtype, device=dev)
    scales = torch.empty(T, (D + 31) // 32, dtype=torch.uint8, device=dev) if mxfp8 else None
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    args = (DTYPES[dtype], _ptr(x), _ptr(residual), weight.data_ptr(), T, D, _ptr(slots), _ptr(gates), k,
            x.shape[0], eps, None if residual is None else _ptr(total), _ptr(out), _ptr(scales), _ptr(rstd))
    fresh = (out, scales, rstd, None if residual is None else total)
    return _call("csf_rms_norm", args, Normed(out, total, rstd, scales), dev, (x, weight, residual, slots, gates), fresh, stream)


def _rms_norm_backward(dy, sum, weight, rstd, dsum=None, stream=None) -> Bound:
    where = "rms_norm_backward"
    dev = _device(where, dy, "dy")
    _need(where, "dy", dy, tuple(DTYPES), dev, dim=2)
    T, D = dy.shape
    _need(where, "sum", sum, (dy.dtype,), dev, shape=(T, D))
    _need(where, "weight", weight, (torch.float32,), dev, D)
    _need(where, "rstd", rstd, (torch.float32,), dev, T)
    if dsum is not None:
        _need(where, "dsum", dsum, (dy.dtype,), dev, shape=(T, D))
    dx = torch.empty_like(dy)
    dweight = torch.empty(D, dtype=torch.float32, device=dev)
    need = _lib().csf_rms_norm_backward_workspace(T, D)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    args = (DTYPES[dy.dtype], _ptr(dy), _ptr(sum), weight.data_ptr(), _ptr(rstd), _ptr(dsum), T, D, _ptr(dx),
            dweight.data_ptr(), workspace.data_ptr(), need)
    return _call("csf_rms_norm_backward", args, (dx, dweight), dev, (dy, sum, weight, rstd, dsum), (dx, dweight, workspace), stream)


def _route(logits, topk, renorm=True, stream=None) -> Bound:
    where = "route"
    dev = _device(where, logits, "logits")
    _need(where, "logits", logits, tuple(DTYPES), dev, dim=2)
    T, E = logits.shape
    if not 1 <= topk <= min(E, 64) or E > MAX_EXPERTS:
        raise ValueError(f"{where}: topk must be 1 to min(E, 64), E at most {MAX_EXPERTS}")
    need = _lib().csf_route_workspace(T, E)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    r = Routing(torch.empty(T, topk, dtype=torch.int32, device=dev), torch.empty(T, topk, dtype=torch.float32, device=dev),
                torch.empty(E + 1, dtype=torch.int32, device=dev), torch.empty(T * topk, dtype=torch.int32, device=dev),
                torch.empty(T, topk, dtype=torch.int32, device=dev))
    args = (DTYPES[logits.dtype], _ptr(logits), T, E, topk, int(bool(renorm)), _ptr(r.experts), _ptr(r.gates),
            r.expert_start.data_ptr(), _ptr(r.rows), _ptr(r.slots), _ptr(workspace), need)
    return _call("csf_route", args, r, dev, (logits,), (*r, workspace), stream)


def _combine_backward(dout, y, slots, gates, stream=None) -> Bound:
    where = "combine_backward"
    dev = _device(where, dout, "dout")
    _need(where, "dout", dout, tuple(DTYPES), dev, dim=2)
    T, D = dout.shape
    _need(where, "y", y, (torch.float32,), dev, dim=2)
    _need(where, "slots", slots, (torch.int32,), dev, dim=2)
    k = slots.shape[1]
    if y.shape[1] != D or slots.shape[0] != T or k < 1:
        raise ValueError(f"{where}: y must be [S, {D}] and slots [{T}, k]")
    _need(where, "gates", gates, (torch.float32,), dev, shape=(T, k))
    dy = torch.empty(y.shape, dtype=dout.dtype, device=dev)
    dgates = torch.empty(T, k, dtype=torch.float32, device=dev)
    args = (DTYPES[dout.dtype], _ptr(dout), _ptr(y), _ptr(slots), _ptr(gates), T, k, D, y.shape[0], _ptr(dy), _ptr(dgates))
    return _call("csf_combine_backward", args, (dy, dgates), dev, (dout, y, slots, gates), (dy, dgates), stream)


def _route_backward(dgates, logits, experts, gates, renorm=True, stream=None) -> Bound:
    where = "route_backward"
    dev = _device(where, logits, "logits")
    _need(where, "logits", logits, tuple(DTYPES), dev, dim=2)
    T, E = logits.shape
    _need(where, "experts", experts, (torch.int32,), dev, dim=2)
    k = experts.shape[1]
    if experts.shape[0] != T or not 1 <= k <= min(E, 64) or E > MAX_EXPERTS:
        raise ValueError(f"{where}: experts must be [{T}, topk], topk at most min(E, 64), E at most {MAX_EXPERTS}")
    _need(where, "dgates", dgates, (torch.float32,), dev, shape=(T, k))
    _need(where, "gates", gates, (torch.float32,), dev, shape=(T, k))
    dlogits = torch.empty_like(logits)
    args = (DTYPES[logits.dtype], _ptr(dgates), _ptr(logits), _ptr(experts), _ptr(gates), T, E, k, int(bool(renorm)),
            _ptr(dlogits))
    return _call("csf_route_backward", args, dlogits, dev, (dgates, logits, experts, gates), (dlogits,), stream)


def _gated_shapes(where, scales, weights, alpha, expert_start):
    """Checks what both passes share; returns the device, E, F and K."""
    if not isinstance(scales, CompressedStack) or scales.device.type != "cuda":
        raise ValueError(f"{where}: the scales must be a compressed stack on a GPU")
    dev = scales.device
    _check_stack_tensors(scales, where)
    if scales.R % 2:
        raise ValueError(f"{where}: the stack needs gate and up rows, an even number")
    E, K = scales.E, scales.C * (16 if scales.fmt == NVFP4 else 32)
    _need(where, "weights", weights, (torch.uint8,), dev, E * scales.R * K // 2)
    _need(where, "alpha", alpha, (torch.float32,), dev, E)
    _need(where, "expert_start", expert_start, (torch.int32,), dev, E + 1)
    return dev, E, scales.R // 2, K


def _dense(where, scales, dense_scales, dev):
    _need(where, "dense_scales", dense_scales, (torch.uint8,), dev)
    if dense_scales.numel() < scales.dense_bytes:
        raise ValueError(f"{where}: dense_scales must have the stack's {scales.dense_bytes} bytes")


def _moe_gated(scales, weights, x, alpha, expert_start, rows, x_scales=None, save=False, dense_scales=None,
               stream=None) -> Bound:
    where = "moe_gated"
    dev, E, F, K = _gated_shapes(where, scales, weights, alpha, expert_start)
    if x_scales is None:
        _need(where, "x", x, (torch.bfloat16,), dev, dim=2)
    else:
        _need(where, "x (E4M3 codes)", x, (torch.uint8,), dev, dim=2)
        if scales.fmt != MXFP4:
            raise ValueError(f"{where}: 8-bit activations need MXFP4 weights")
        _need(where, "x_scales", x_scales, (torch.uint8,), dev, shape=(x.shape[0], K // 32))
    T = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"{where}: x must be [T, {K}]")
    _need(where, "rows", rows, (torch.int32,), dev, dim=1)
    S = rows.shape[0]
    if dense_scales is not None:
        _dense(where, scales, dense_scales, dev)
    h = torch.empty(S, F, dtype=torch.bfloat16, device=dev)
    gu = torch.empty(S, 2 * F, dtype=torch.bfloat16, device=dev) if save else None
    d = scales.descriptor()
    need = _lib().csf_moe_gated_workspace(ctypes.byref(d), S)
    if dense_scales is not None:  # the tiles' counters only
        need = min(need, 64)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    args = (ctypes.byref(d), _ptr(dense_scales), weights.data_ptr(), _ptr(x), _ptr(x_scales), T, alpha.data_ptr(),
            expert_start.data_ptr(), _ptr(rows), S, _ptr(h), _ptr(gu), _ptr(workspace), need)
    inputs = (scales, d, weights, x, x_scales, alpha, expert_start, rows, dense_scales)
    return _call("csf_moe_gated", args, (h, gu) if save else h, dev, inputs, (h, gu, workspace), stream)


def _moe_gated_backward(scales, dense_scales, weights, dh, gate_up, alpha, expert_start, stream=None) -> Bound:
    where = "moe_gated_backward"
    dev, E, F, K = _gated_shapes(where, scales, weights, alpha, expert_start)
    _dense(where, scales, dense_scales, dev)
    _need(where, "dh", dh, (torch.bfloat16,), dev, dim=2)
    S = dh.shape[0]
    if dh.shape[1] != F:
        raise ValueError(f"{where}: dh must be [S, {F}]")
    _need(where, "gate_up", gate_up, (torch.bfloat16,), dev, shape=(S, 2 * F))
    dx = torch.empty(S, K, dtype=torch.bfloat16, device=dev)
    dgu = torch.empty(S, 2 * F, dtype=torch.bfloat16, device=dev)
    d = scales.descriptor()
    args = (ctypes.byref(d), dense_scales.data_ptr(), weights.data_ptr(), _ptr(dh), _ptr(gate_up), S, alpha.data_ptr(),
            expert_start.data_ptr(), _ptr(dx), _ptr(dgu))
    inputs = (scales, d, dense_scales, weights, dh, gate_up, alpha, expert_start)
    return _call("csf_moe_gated_backward", args, (dx, dgu), dev, inputs, (dx, dgu), stream)


def rms_norm(x, weight, residual=None, slots=None, gates=None, eps=1e-6, mxfp8=False, stream=None) -> Normed:
    """Enqueue the RMS norm of ``x + residual`` (see ``csf_rms_norm``): bfloat16,
    float16 or float32 [T, D], ``weight`` float32 [D].  With ``slots`` (int32
    [T, k]) and ``gates`` (float32 [T, k]), ``x`` is float32 [S, D], the experts'
    outputs, and their combination takes its place.  ``mxfp8`` gives E4M3 codes
    and E8M0 scales per 32 columns, what ``moe_gated`` reads."""
    return _rms_norm(x, weight, residual, slots, gates, eps, mxfp8, stream)()


def rms_norm_backward(dy, sum, weight, rstd, dsum=None, stream=None):
    """Enqueue the norm's backward pass from ``rms_norm``'s ``sum`` and ``rstd``;
    returns ``(dx, dweight)``: dx serves x and residual alike, ``dsum`` is the
    gradient that reaches the sum itself."""
    return _rms_norm_backward(dy, sum, weight, rstd, dsum, stream)()


def route(logits, topk: int, renorm: bool = True, stream=None) -> Routing:
    """Enqueue the router (see ``csf_route``): the ``topk`` experts of each row of
    ``logits`` [T, E], their gates, and the grouped routing of the T * topk
    choices: ``expert_start`` as the decode and the projections take it, the
    token of each slot (``rows``) and the slot of each choice (``slots``)."""
    return _route(logits, topk, renorm, stream)()


def combine_backward(dout, y, slots, gates, stream=None):
    """Enqueue the backward pass of the routed combination (see
    ``csf_combine_backward``); returns ``(dy, dgates)``."""
    return _combine_backward(dout, y, slots, gates, stream)()


def route_backward(dgates, logits, experts, gates, renorm: bool = True, stream=None):
    """Enqueue the gradient of the router's logits (see ``csf_route_backward``)."""
    return _route_backward(dgates, logits, experts, gates, renorm, stream)()


def moe_gated(scales, weights, x, alpha, expert_start, rows, x_scales=None, save=False, dense_scales=None, stream=None):
    """Enqueue the gated feed-forward half (see ``csf_moe_gated``): ``scales`` is the
    stack of the gate and up rows, ``weights`` uint8 [E, 2F, K/2], ``x`` bfloat16
    [T, K] or E4M3 codes with ``x_scales`` (MXFP4 weights); returns h (bfloat16
    [S, F]), with ``save`` also the gate and up values the backward pass reads.
    ``dense_scales`` are scales decoded beforehand."""
    return _moe_gated(scales, weights, x, alpha, expert_start, rows, x_scales, save, dense_scales, stream)()


def moe_gated_backward(scales, dense_scales, weights, dh, gate_up, alpha, expert_start, stream=None):
    """Enqueue the gated half's backward pass (see ``csf_moe_gated_backward``);
    returns ``(dx, dgate_up)`` per slot.  ``dense_scales`` is a ``decode`` workspace
    filled with the same ``expert_start``."""
    return _moe_gated_backward(scales, dense_scales, weights, dh, gate_up, alpha, expert_start, stream)()


_BINDERS = {rms_norm: _rms_norm, rms_norm_backward: _rms_norm_backward, route: _route,
            combine_backward: _combine_backward, route_backward: _route_backward, moe_gated: _moe_gated,
            moe_gated_backward: _moe_gated_backward}


def bound(function, *args, **kwargs) -> Bound:
    """One call of a layer operator, checked and marshalled once: each call of the
    result enqueues it again on the same buffers and returns the same outputs, on
    the stream then current, or on ``stream`` where one is given here.  Keeps
    references to every tensor; a graph that captured it needs it kept."""
    if function not in _BINDERS:
        raise ValueError("bound() takes one of: " + ", ".join(f.__name__ for f in _BINDERS))
    return _BINDERS[function](*args, **kwargs)
