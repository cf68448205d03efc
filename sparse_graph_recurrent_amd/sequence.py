"""Sequence operators of a text model around the graph recurrence: a short
causal convolution, a selective state space scan and a counter-based dropout.

The layouts are the recurrence's: windows are time first, [T, B, channels].
Sequence tensors may be fp32, bf16 or fp16 (one type per call) and need only
their channels adjacent, so slices of a projection and batch-major storage
(``x.transpose(0, 1)``) are taken as they are; parameters and scan states are
fp32 and contiguous.  ``lengths`` (int32 [B]) cuts each row of a batch of
unequal texts: later steps change nothing, whatever the padding holds, and
give 0.

    y, conv_state = short_conv(x, weight, bias, activation="silu")
    out, state = selective_scan(u, delta, A, B, C, D, z=z, delta_bias=bias, delta_softplus=True)
    h = dropout(out, p, seed, residual=x)

are differentiable; ``*_forward`` / ``*_backward`` are the calls behind them
and ``*_step`` take one token per row, from and to the carried states.
These calls take a ``stream`` to run on instead of the current one; their
inputs have to be ready there, and what they allocate is that stream's memory.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch
from torch.autograd.function import once_differentiable

from . import _check, _on_stream, lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class CkSeq(ctypes.Structure):
    """ck_seq of include/ck.h."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_t", ctypes.c_int64),
                ("stride_b", ctypes.c_int64)]


class ScanShape(ctypes.Structure):
    """ck_scan_shape of include/ck.h."""
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("D", ctypes.c_int64),
                ("N", ctypes.c_int64), ("G", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("delta_softplus", ctypes.c_int32)]


class ScanInputs(ctypes.Structure):
    """ck_scan_inputs of include/ck.h."""
    _fields_ = [(n, CkSeq) for n in ("u", "delta", "b", "c", "z")] + \
               [(n, ctypes.c_void_p) for n in ("a", "d", "delta_bias", "state0", "lengths")]


class ScanGrads(ctypes.Structure):
    """ck_scan_grads of include/ck.h."""
    _fields_ = [(n, CkSeq) for n in ("u", "delta", "b", "c", "z")] + \
               [(n, ctypes.c_void_p) for n in ("a", "d", "delta_bias", "state0")]


class ConvShape(ctypes.Structure):
    """ck_conv_shape of include/ck.h."""
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("D", ctypes.c_int64),
                ("W", ctypes.c_int64), ("dtype", ctypes.c_int32), ("silu", ctypes.c_int32)]


class DropoutShape(ctypes.Structure):
    """ck_dropout_shape of include/ck.h."""
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("D", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("held", ctypes.c_int32), ("p", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("counter", ctypes.c_void_p)]


# The calls fill these structures as packed bytes, several times quicker than
# ctypes fills nested ones (a token's call takes about as long as its kernel).
_SCAN_SHAPE = struct.Struct("=5q2i")
_SCAN_INPUTS = struct.Struct("=20Q")
_SCAN_GRADS = struct.Struct("=19Q")
_CONV_SHAPE = struct.Struct("=4q2i")
_DROP_SHAPE = struct.Struct("=3q2id3Q")
assert _SCAN_SHAPE.size == ctypes.sizeof(ScanShape)
assert _SCAN_INPUTS.size == ctypes.sizeof(ScanInputs)
assert _SCAN_GRADS.size == ctypes.sizeof(ScanGrads)
assert _CONV_SHAPE.size == ctypes.sizeof(ConvShape)
assert _DROP_SHAPE.size == ctypes.sizeof(DropoutShape)

_NONE = (0, 0, 0)  # a ck_seq that is absent


def _declare(L: ctypes.CDLL) -> None:
    """Argument types of the sequence entry points (called once, by ``lib``).
    Structures are passed by address: their packed bytes, or ``ctypes.byref``."""
    p, sz, q = ctypes.c_void_p, ctypes.c_size_t, CkSeq
    szp = ctypes.POINTER(sz)
    L.ck_scan_sizes.argtypes = [p, szp, szp, szp]
    L.ck_scan_forward.argtypes = [p, p, q, p, p, p, sz, p]
    L.ck_scan_backward.argtypes = [p, p, p, q, p, p, p, sz, p]
    L.ck_scan_step.argtypes = [p, p, q, p, p]
    L.ck_conv_sizes.argtypes = [p, szp]
    L.ck_conv_forward.argtypes = [p, q, p, p, p, p, q, p, p]
    L.ck_conv_backward.argtypes = [p, q, p, p, p, p, q, p, q, p, p, p, p, sz, p]
    L.ck_conv_step.argtypes = [p, q, p, p, p, q, p, p]
    L.ck_dropout_forward.argtypes = [p, q, q, q, p]
    L.ck_dropout_backward.argtypes = [p, q, q, p]


def _call(fn, dev: int, args):
    """Runs one entry point with device `dev` current, on its current stream."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(fn, dev, args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


def _adjacent(t: torch.Tensor, last: int) -> bool:
    """True when the last `last` dimensions of t are laid out contiguously."""
    want = 1
    for size, stride in zip(reversed(t.shape[-last:]), reversed(t.stride()[-last:])):
        if size != 1 and stride != want:
            return False
        want *= size
    return True


def _refuse(t, name: str, dtype, dev: int, shape):
    """Raises the error that `t` not being a tensor of this type, device and shape calls for."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _seq(t, name: str, dtype, dev: int, shape, last: int = 1):
    """(address, stride_t, stride_b) of a [T, B, ...] tensor (a step's [B, ...]
    tensor counts as T = 1), checked.  (An empty tensor's address is 0.)"""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape):
        _refuse(t, name, dtype, dev, shape)
    st = t.stride()
    if st[-1] != 1 or last == 2 and st[-2] != shape[-1]:
        if not _adjacent(t, last):  # (sizes of 1 may have any stride)
            raise ValueError(f"{name} must have its last {last} dimension(s) contiguous")
    if len(shape) - last == 1:
        return t.data_ptr(), 0, st[0] if shape[0] > 1 else 0
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0


def _par(t, name: str, dev: int, shape, dtype=torch.float32) -> int:
    """Address of an optional contiguous parameter, state or length vector."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        _refuse(t, name, dtype, dev, shape)
    return t.data_ptr()


def _first(t, name: str, dims) -> int:
    """Checks the tensor that gives a call its type, device and sizes; its device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, "
                         f"got {t.dim()}")
    return t.get_device()


def _fresh(like: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of like's shape and type."""
    # (a copy of a tensor's layout is the quicker of the two calls)
    return torch.empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)


def _dense(shape, inner: int):
    """(stride_t, stride_b) of a contiguous [T, B, ...] tensor, `inner` elements a
    row, or of a step's [B, ...]; 0 where there is but one."""
    if len(shape) == 2:
        return 0, inner if shape[0] > 1 else 0
    return inner * shape[1] if shape[0] > 1 else 0, inner if shape[1] > 1 else 0


# Tells autograd that tensors (a tuple of them) were written: a backward that saved
# what one held before raises, as it does behind torch's own in-place operations.
_written = torch._C._increment_version


def _out_seq(t, name: str, like: torch.Tensor):
    """(tensor, its ck_seq) of an output of like's [.., D] shape: the caller's,
    checked, or a new contiguous one."""
    shape = like.shape
    if t is None:
        t = _fresh(like)
        return t, CkSeq(t.data_ptr(), *_dense(shape, shape[-1]))
    q = CkSeq(*_seq(t, name, like.dtype, like.get_device(), shape))
    _written((t,))
    return t, q


def _out_par(t, name: str, like: torch.Tensor, shape, dtype=torch.float32, model=None):
    """(tensor, its address) of a contiguous output; `model`: a contiguous tensor
    of its shape and type, if there is one (quicker to copy)."""
    if t is not None:
        at = _par(t, name, like.get_device(), shape, dtype)
        _written((t,))
        return t, at
    t = like.new_empty(shape, dtype=dtype) if model is None else torch.empty_like(model)
    return t, t.data_ptr()


def _buffer(buf, nbytes: int, like: torch.Tensor, name: str):
    """(byte buffer, its address, its size): the caller's, checked, or a new one;
    none for 0 bytes."""
    if buf is None:
        if not nbytes:
            return None, None, 0
        buf = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=like.device)
        return buf, buf.data_ptr(), nbytes
    size = buf.numel() * buf.element_size()
    if buf.get_device() != like.get_device() or size < nbytes or not buf.is_contiguous():
        raise ValueError(f"{name} buffer too small, not contiguous or on another device")
    return buf, buf.data_ptr() if size else None, size


# ------------------------------------------------------------ selective scan

def _scan_call(u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus, step=False):
    """(shape, inputs, device, sizes (T, B, D, N, G)) of a scan call, checked."""
    dev = _first(u, "u", (2,) if step else (3,))
    us, dt = u.shape, u.dtype
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [channels, states] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != len(us) + 1:
        raise ValueError(f"B must have {len(us) + 1} dimensions (.., groups, states)")
    T, rows, ch = (1,) + us if step else us
    N, G = A.shape[1], B.shape[-2]
    bs = us[:-1] + (G, N)
    sizes = (T, rows, ch, N, G)
    return _SCAN_SHAPE.pack(*sizes, _DTYPES[dt], 1 if delta_softplus else 0), _SCAN_INPUTS.pack(
        *_seq(u, "u", dt, dev, us), *_seq(delta, "delta", dt, dev, us),
        *_seq(B, "B", dt, dev, bs, 2), *_seq(C, "C", dt, dev, bs, 2),
        *(_NONE if z is None else _seq(z, "z", dt, dev, us)),
        _par(A, "A", dev, (ch, N)), _par(D, "D", dev, (ch,)),
        _par(delta_bias, "delta_bias", dev, (ch,)), _par(state0, "state0", dev, (rows, ch, N)),
        _par(lengths, "lengths", dev, (rows,), torch.int32)), dev, sizes


@functools.lru_cache(maxsize=256)
def _scan_sizes(shape: bytes):
    s, f, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().ck_scan_sizes(shape, ctypes.byref(s), ctypes.byref(f), ctypes.byref(b)))
    return s.value, f.value, b.value


def selective_scan_sizes(T: int, B: int, D: int, N: int, G: int = 1, dtype=torch.float32):
    """(saved_bytes, forward_bytes, backward_bytes) of ``ck_scan_sizes``."""
    return _scan_sizes(_SCAN_SHAPE.pack(T, B, D, N, G, _DTYPES[dtype], 0))


def selective_scan_forward(u, delta, A, B, C, D=None, z=None, delta_bias=None, state0=None,
                           lengths=None, delta_softplus: bool = False, save: bool = True,
                           out=None, state=None, saved=None, workspace=None, stream=None):
    """Run ``ck_scan_forward``; returns (out, state, saved, workspace).

    u, delta, z: [T, B, D]; B, C: [T, B, G, N]; A: [D, N]; D, delta_bias: [D];
    state0 and the returned state: [B, D, N].  ``saved`` is what
    ``selective_scan_backward`` needs (None with save=False)."""
    if stream is not None:
        return _on_stream(stream, selective_scan_forward, u, delta, A, B, C, D, z, delta_bias,
                          state0, lengths, delta_softplus, save, out, state, saved, workspace)
    shape, inputs, dev, (T, rows, ch, N, _) = _scan_call(
        u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus)
    sb, fb, _ = _scan_sizes(shape)
    out, os = _out_seq(out, "out", u)
    state, st = _out_par(state, "state", u, (rows, ch, N), model=state0)
    saved, sp, _ = _buffer(saved, sb, u, "saved") if save or saved is not None else \
        (None, None, 0)
    workspace, wp, wn = _buffer(workspace, fb, u, "workspace")
    _call(lib().ck_scan_forward, dev, (shape, inputs, os, st, sp, wp, wn))
    return out, state, saved, workspace


def selective_scan_backward(u, delta, A, B, C, saved, grad_out, D=None, z=None, delta_bias=None,
                            lengths=None, delta_softplus: bool = False, grad_state=None,
                            grads=None, workspace=None, stream=None) -> dict:
    """Run ``ck_scan_backward``; returns the gradients (overwritten) by the
    names g_u, g_delta, g_A, g_B, g_C, g_D, g_delta_bias, g_state0 and, with a
    gate, g_z."""
    if stream is not None:
        return _on_stream(stream, selective_scan_backward, u, delta, A, B, C, saved, grad_out, D, z,
                          delta_bias, lengths, delta_softplus, grad_state, grads, workspace)
    shape, inputs, dev, (T, rows, ch, N, G) = _scan_call(
        u, delta, A, B, C, D, z, delta_bias, None, lengths, delta_softplus)
    sb, _, wb = _scan_sizes(shape)
    if sb and saved is None:
        raise ValueError("saved is missing")
    _, sp, _ = _buffer(saved, sb, u, "saved")
    ss = (rows, ch, N)
    go = CkSeq(*_seq(grad_out, "grad_out", u.dtype, dev, u.shape))
    gs = _par(grad_state, "grad_state", dev, ss)
    if grads is None:
        g = {"g_u": _fresh(u), "g_delta": _fresh(delta), "g_B": _fresh(B), "g_C": _fresh(C),
             "g_A": torch.empty_like(A), "g_D": D, "g_delta_bias": delta_bias,
             "g_state0": grad_state}
        for name, shape_ in (("g_D", (ch,)), ("g_delta_bias", (ch,)), ("g_state0", ss)):
            like = g[name]
            g[name] = A.new_empty(shape_) if like is None else torch.empty_like(like)
        rows_, bcs = _dense(u.shape, ch), _dense(u.shape, G * N)
        gz = _NONE
        if z is not None:
            g["g_z"] = _fresh(z)
            gz = (g["g_z"].data_ptr(), *rows_)
        out = _SCAN_GRADS.pack(
            g["g_u"].data_ptr(), *rows_, g["g_delta"].data_ptr(), *rows_,
            g["g_B"].data_ptr(), *bcs, g["g_C"].data_ptr(), *bcs, *gz,
            g["g_A"].data_ptr(), g["g_D"].data_ptr(), g["g_delta_bias"].data_ptr(),
            g["g_state0"].data_ptr())
    else:
        g = grads
        out = _SCAN_GRADS.pack(
            *_seq(g["g_u"], "g_u", u.dtype, dev, u.shape),
            *_seq(g["g_delta"], "g_delta", u.dtype, dev, u.shape),
            *_seq(g["g_B"], "g_B", u.dtype, dev, B.shape, 2),
            *_seq(g["g_C"], "g_C", u.dtype, dev, B.shape, 2),
            *(_NONE if z is None else _seq(g["g_z"], "g_z", u.dtype, dev, u.shape)),
            _par(g.get("g_A"), "g_A", dev, A.shape), _par(g.get("g_D"), "g_D", dev, (ch,)),
            _par(g.get("g_delta_bias"), "g_delta_bias", dev, (ch,)),
            _par(g.get("g_state0"), "g_state0", dev, ss))
        _written(tuple(t for t in g.values() if t is not None))
    workspace, wp, wn = _buffer(workspace, wb, u, "workspace")
    _call(lib().ck_scan_backward, dev, (shape, inputs, sp, go, gs, out, wp, wn))
    return g


def selective_scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                        delta_softplus: bool = False, out=None, new_state=None, stream=None):
    """Run ``ck_scan_step``: one token per row.  u, delta, z: [B, D]; B, C:
    [B, G, N]; state: [B, D, N], updated in place unless ``new_state`` is
    given.  Returns (out [B, D], the new state)."""
    if stream is not None:
        return _on_stream(stream, selective_scan_step, state, u, delta, A, B, C, D, z, delta_bias,
                          delta_softplus, out, new_state)
    if state is None:
        raise ValueError("state is missing")
    shape, inputs, dev, (_, rows, ch, N, _) = _scan_call(
        u, delta, A, B, C, D, z, delta_bias, state, None, delta_softplus, step=True)
    new_state = state if new_state is None else new_state
    out, os = _out_seq(out, "out", u)
    _call(lib().ck_scan_step, dev,
          (shape, inputs, os, _par(new_state, "new_state", dev, (rows, ch, N))))
    _written((new_state,))
    return out, new_state


def _rows(t):
    """t itself when its channels are adjacent, else a contiguous copy."""
    return t if t is None or t.numel() == 0 or _adjacent(t, 1) else t.contiguous()


def _groups(t):
    return t if t.numel() == 0 or _adjacent(t, 2) else t.contiguous()


def _cont(t):
    return None if t is None else t.contiguous()


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus,
                recording):
        u, delta, z, B, C = _rows(u), _rows(delta), _rows(z), _groups(B), _groups(C)
        A, D, delta_bias, state0 = (_cont(t) for t in (A, D, delta_bias, state0))
        out, state, saved, _ = selective_scan_forward(
            u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus,
            save=recording and any(ctx.needs_input_grad))
        ctx.softplus = delta_softplus
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, lengths, saved)
        return out, state

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_state):
        u, delta, A, B, C, D, z, delta_bias, lengths, saved = ctx.saved_tensors
        go = torch.zeros_like(u) if grad_out is None else _rows(grad_out)
        g = selective_scan_backward(u, delta, A, B, C, saved, go, D, z, delta_bias, lengths,
                                    ctx.softplus, grad_state=_cont(grad_state))
        return (g["g_u"], g["g_delta"], g["g_A"], g["g_B"], g["g_C"],
                None if D is None else g["g_D"], g.get("g_z"),
                None if delta_bias is None else g["g_delta_bias"],
                g["g_state0"] if ctx.needs_input_grad[8] else None, None, None, None)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, state0=None, lengths=None,
                   delta_softplus: bool = False):
    """The selective scan as one autograd node: returns (out [T, B, D], the
    state after each row's last step [B, D, N]); gradients reach every tensor
    argument but ``lengths``.  Shapes as for ``selective_scan_forward``."""
    # needs_input_grad says nothing of the grad mode, which is off inside the node:
    # without it a prompt would leave the backward's states for nobody
    return _SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, state0, lengths,
                                bool(delta_softplus), torch.is_grad_enabled())


# --------------------------------------------------------- short convolution

def _conv_call(x, weight, bias, activation, step=False):
    """(shape, device, state shape, x's ck_seq, weight, bias) of a convolution call, checked."""
    dev = _first(x, "x", (2,) if step else (3,))
    if activation is not None and activation != "silu":
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [channels, taps] tensor")
    T, rows, ch = (1,) + x.shape if step else x.shape
    W = weight.shape[1]
    return (_CONV_SHAPE.pack(T, rows, ch, W, _DTYPES[x.dtype], 1 if activation else 0), dev,
            (W - 1, rows, ch), CkSeq(*_seq(x, "x", x.dtype, dev, x.shape)),
            _par(weight, "weight", dev, (ch, W)), _par(bias, "bias", dev, (ch,)))


@functools.lru_cache(maxsize=256)
def _conv_sizes(shape: bytes) -> int:
    need = ctypes.c_size_t()
    _check(lib().ck_conv_sizes(shape, ctypes.byref(need)))
    return need.value


def short_conv_forward(x, weight, bias=None, state0=None, lengths=None, activation=None, y=None,
                       state=None, stream=None):
    """Run ``ck_conv_forward``; returns (y, state).  x: [T, B, D]; weight:
    [D, W]; bias: [D]; state0 and the returned state: [W - 1, B, D], the last
    inputs of each row; activation: None or "silu"."""
    if stream is not None:
        return _on_stream(stream, short_conv_forward, x, weight, bias, state0, lengths, activation,
                          y, state)
    shape, dev, ss, xs, w, b = _conv_call(x, weight, bias, activation)
    y, ys = _out_seq(y, "y", x)
    state, st = _out_par(state, "state", x, ss, x.dtype, state0)
    _call(lib().ck_conv_forward, dev,
          (shape, xs, w, b, _par(state0, "state0", dev, ss, x.dtype),
           _par(lengths, "lengths", dev, (ss[1],), torch.int32), ys, st))
    return y, state


def short_conv_backward(x, weight, grad_y, bias=None, state0=None, lengths=None, activation=None,
                        grad_state=None, grads=None, workspace=None, stream=None) -> dict:
    """Run ``ck_conv_backward``; returns the gradients (overwritten) g_x,
    g_weight, g_bias and g_state0."""
    if stream is not None:
        return _on_stream(stream, short_conv_backward, x, weight, grad_y, bias, state0, lengths,
                          activation, grad_state, grads, workspace)
    shape, dev, ss, xs, w, b = _conv_call(x, weight, bias, activation)
    s0 = _par(state0, "state0", dev, ss, x.dtype)
    if grads is None:
        g = {"g_x": _fresh(x), "g_weight": torch.empty_like(weight),
             "g_bias": weight.new_empty(ss[2]) if bias is None else torch.empty_like(bias),
             "g_state0": x.new_empty(ss) if state0 is None else torch.empty_like(state0)}
        gx = CkSeq(g["g_x"].data_ptr(), *_dense(x.shape, ss[2]))
        gw, gb, gs0 = (g[k].data_ptr() for k in ("g_weight", "g_bias", "g_state0"))
    else:
        g = grads
        gx = CkSeq(*_seq(g["g_x"], "g_x", x.dtype, dev, x.shape))
        gw = _par(g["g_weight"], "g_weight", dev, weight.shape)
        gb = _par(g.get("g_bias"), "g_bias", dev, (ss[2],))
        gs0 = _par(g.get("g_state0"), "g_state0", dev, ss, x.dtype)
        _written(tuple(t for t in g.values() if t is not None))
    workspace, wp, wn = _buffer(workspace, _conv_sizes(shape), x, "workspace")
    _call(lib().ck_conv_backward, dev,
          (shape, xs, w, b, s0,
           _par(lengths, "lengths", dev, (ss[1],), torch.int32),
           CkSeq(*_seq(grad_y, "grad_y", x.dtype, dev, x.shape)),
           _par(grad_state, "grad_state", dev, ss, x.dtype), gx, gw, gb, gs0, wp, wn))
    return g


def short_conv_step(state, x, weight, bias=None, activation=None, y=None, new_state=None,
                    stream=None):
    """Run ``ck_conv_step``: one token per row.  x: [B, D]; state: [W - 1, B,
    D], updated in place unless ``new_state`` is given.  Returns (y [B, D],
    the new state)."""
    if stream is not None:
        return _on_stream(stream, short_conv_step, state, x, weight, bias, activation, y, new_state)
    shape, dev, ss, xs, w, b = _conv_call(x, weight, bias, activation, step=True)
    new_state = state if new_state is None else new_state
    y, ys = _out_seq(y, "y", x)
    _call(lib().ck_conv_step, dev,
          (shape, xs, w, b, _par(state, "state", dev, ss, x.dtype), ys,
           _par(new_state, "new_state", dev, ss, x.dtype)))
    if new_state is not None:
        _written((new_state,))
    return y, new_state


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state0, lengths, activation):
        x, weight, bias, state0 = _rows(x), _cont(weight), _cont(bias), _cont(state0)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, state0, lengths)
        return short_conv_forward(x, weight, bias, state0, lengths, activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_state):
        x, weight, bias, state0, lengths = ctx.saved_tensors
        gy = torch.zeros_like(x) if grad_y is None else _rows(grad_y)
        g = short_conv_backward(x, weight, gy, bias, state0, lengths, ctx.activation,
                                grad_state=_cont(grad_state))
        return (g["g_x"], g["g_weight"], None if bias is None else g["g_bias"],
                None if state0 is None else g["g_state0"], None, None)


def short_conv(x, weight, bias=None, state0=None, lengths=None, activation=None):
    """The short causal convolution as one autograd node: returns (y, state);
    gradients reach x, weight, bias and state0.  Shapes as for
    ``short_conv_forward``."""
    return _ShortConv.apply(x, weight, bias, state0, lengths, activation)


# ------------------------------------------------------------------- dropout

def _drop_call(x, name, p, seed, offset, held, counter):
    """(shape, device, x's ck_seq) of a dropout call, checked."""
    dev = _first(x, name, (2, 3))
    T, rows, ch = (1,) + x.shape if x.dim() == 2 else x.shape
    m = 0xFFFFFFFFFFFFFFFF
    return _DROP_SHAPE.pack(T, rows, ch, _DTYPES[x.dtype], 1 if held else 0, p, seed & m,
                            offset & m, _par(counter, "counter", dev, (1,), torch.int64)), dev, \
        CkSeq(*_seq(x, name, x.dtype, dev, x.shape))


def dropout_forward(x, p: float, seed: int, offset: int = 0, residual=None, held: bool = False,
                    counter=None, out=None, stream=None) -> torch.Tensor:
    """Run ``ck_dropout_forward`` on x [T, B, D] (or one step's [B, D]):
    residual + x / (1 - p) where kept, with p rounded to a multiple of 2^-16.
    The mask follows from (seed, offset) alone; held=True gives all steps of a
    window the same mask.  A device ``counter`` (int64 [1]) is added to the
    offset, so that a replayed graph can draw new masks.  ``out`` may be x or
    the residual."""
    if stream is not None:
        return _on_stream(stream, dropout_forward, x, p, seed, offset, residual, held, counter, out)
    shape, dev, xs = _drop_call(x, "x", p, seed, offset, held, counter)
    rs = _NONE if residual is None else _seq(residual, "residual", x.dtype, dev, x.shape)
    out, os = _out_seq(out, "out", x)
    _call(lib().ck_dropout_forward, dev, (shape, xs, CkSeq(*rs), os))
    return out


def dropout_backward(grad_out, p: float, seed: int, offset: int = 0, held: bool = False,
                     counter=None, grad_x=None, stream=None) -> torch.Tensor:
    """Run ``ck_dropout_backward``: the forward's mask and scale on grad_out."""
    if stream is not None:
        return _on_stream(stream, dropout_backward, grad_out, p, seed, offset, held, counter,
                          grad_x)
    shape, dev, gs = _drop_call(grad_out, "grad_out", p, seed, offset, held, counter)
    grad_x, os = _out_seq(grad_x, "grad_x", grad_out)
    _call(lib().ck_dropout_backward, dev, (shape, gs, os))
    return grad_x


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, held, counter):
        # the backward needs the counter's value of now, whatever it becomes
        ctx.args = (p, seed, offset, held)
        ctx.save_for_backward(None if counter is None else counter.clone())
        return dropout_forward(_rows(x), p, seed, offset, _rows(residual), held, counter)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        p, seed, offset, held = ctx.args
        gx = None
        if ctx.needs_input_grad[0]:
            gx = dropout_backward(_rows(grad_out), p, seed, offset, held, ctx.saved_tensors[0])
        return gx, grad_out if ctx.needs_input_grad[1] else None, None, None, None, None, None


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, held: bool = False,
            counter=None) -> torch.Tensor:
    """Dropout as one autograd node that stores no mask; gradients reach x and
    the residual.  Arguments as for ``dropout_forward``."""
    return _Dropout.apply(x, residual, float(p), int(seed), int(offset), bool(held), counter)


__all__ = ["selective_scan", "selective_scan_sizes", "selective_scan_forward",
           "selective_scan_backward", "selective_scan_step", "short_conv", "short_conv_forward",
           "short_conv_backward", "short_conv_step", "dropout", "dropout_forward",
           "dropout_backward"]
