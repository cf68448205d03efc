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
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _byte_buffer, _check, _dev, _ptr, lib

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


def _declare(L: ctypes.CDLL) -> None:
    """Argument types of the sequence entry points (called once, by ``lib``)."""
    p, sz, q = ctypes.c_void_p, ctypes.c_size_t, CkSeq
    szp = ctypes.POINTER(sz)
    scan, conv, drop = (ctypes.POINTER(s) for s in (ScanShape, ConvShape, DropoutShape))
    inp, grads = ctypes.POINTER(ScanInputs), ctypes.POINTER(ScanGrads)
    L.ck_scan_sizes.argtypes = [scan, szp, szp, szp]
    L.ck_scan_forward.argtypes = [scan, inp, q, p, p, p, sz, p]
    L.ck_scan_backward.argtypes = [scan, inp, p, q, p, grads, p, sz, p]
    L.ck_scan_step.argtypes = [scan, inp, q, p, p]
    L.ck_conv_sizes.argtypes = [conv, szp]
    L.ck_conv_forward.argtypes = [conv, q, p, p, p, p, q, p, p]
    L.ck_conv_backward.argtypes = [conv, q, p, p, p, p, q, p, q, p, p, p, p, sz, p]
    L.ck_conv_step.argtypes = [conv, q, p, p, p, q, p, p]
    L.ck_dropout_forward.argtypes = [drop, q, q, q, p]
    L.ck_dropout_backward.argtypes = [drop, q, q, p]


class _On:
    """The device and stream of a call: makes the tensors' device current while
    the library runs, and keeps the memory of tensors made here from being
    reused while a stream other than the current one still works on them."""

    def __init__(self, device: torch.device, stream):
        self.device = device
        self.stream = stream

    def __call__(self, fn, *args, made=()):
        with torch.cuda.device(self.device):
            s = torch.cuda.current_stream() if self.stream is None else self.stream
            _check(fn(*args, ctypes.c_void_p(s.cuda_stream)))
            if self.stream is not None:
                for t in made:
                    if t is not None:
                        t.record_stream(s)


def _adjacent(t: torch.Tensor, last: int) -> bool:
    """True when the last `last` dimensions of t are laid out contiguously."""
    want = 1
    for size, stride in zip(reversed(t.shape[-last:]), reversed(t.stride()[-last:])):
        if size != 1 and stride != want:
            return False
        want *= size
    return True


def _seq(t: torch.Tensor, name: str, like: torch.Tensor, shape, last: int = 1) -> CkSeq:
    """The ck_seq of a [T, B, ...] tensor (a step's [B, ...] tensor counts as T = 1)."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() == 0:
        return CkSeq(None, 0, 0)
    if not _adjacent(t, last):
        raise ValueError(f"{name} must have its last {last} dimension(s) contiguous")
    st = t.stride()
    lead = t.dim() - last  # [T, B] or [B]
    return CkSeq(t.data_ptr(), st[0] if lead == 2 and t.shape[0] > 1 else 0,
                 st[lead - 1] if t.shape[lead - 1] > 1 else 0)


def _par(t, name: str, like: torch.Tensor, shape, dtype=torch.float32):
    """Pointer of an optional contiguous parameter, state or length vector."""
    if t is None:
        return None
    _dev(t, name, dtype, shape)
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    return t.data_ptr() if t.numel() else None


def _first(t, name: str, dims) -> torch.Tensor:
    """The tensor that gives a call its type, device and sizes."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, "
                         f"got {t.dim()}")
    return t


def _into(t, name: str, like: torch.Tensor, shape, dtype=None):
    """(tensor, was made here) of an output: the caller's, or a new one."""
    if t is not None:
        return t, False
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device), True


def _buffer(buf, nbytes: int, like: torch.Tensor, name: str):
    """A byte buffer of the caller's (checked) or a new one; None for 0 bytes."""
    if buf is None:
        return _byte_buffer(nbytes, like.device) if nbytes else None
    if buf.device != like.device or buf.numel() * buf.element_size() < nbytes:
        raise ValueError(f"{name} buffer too small or on another device")
    return buf


def _bytes(buf) -> int:
    return 0 if buf is None else buf.numel() * buf.element_size()


# ------------------------------------------------------------ selective scan

def _scan_call(u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus, step=False):
    """(shape, inputs) structures of a scan call, checked."""
    _first(u, "u", (2,) if step else (3,))
    lead = tuple(u.shape[:-1])
    ch = u.shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [channels, states] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != u.dim() + 1:
        raise ValueError(f"B must have {u.dim() + 1} dimensions (.., groups, states)")
    N, G = A.shape[1], B.shape[-2]
    T, rows = (1,) + lead if step else lead
    shape = ScanShape(T, rows, ch, N, G, _DTYPES[u.dtype], 1 if delta_softplus else 0)
    none = CkSeq(None, 0, 0)
    return shape, ScanInputs(
        _seq(u, "u", u, lead + (ch,)), _seq(delta, "delta", u, lead + (ch,)),
        _seq(B, "B", u, lead + (G, N), 2), _seq(C, "C", u, lead + (G, N), 2),
        none if z is None else _seq(z, "z", u, lead + (ch,)),
        _par(A, "A", u, (ch, N)), _par(D, "D", u, (ch,)),
        _par(delta_bias, "delta_bias", u, (ch,)), _par(state0, "state0", u, (rows, ch, N)),
        _par(lengths, "lengths", u, (rows,), torch.int32))


def selective_scan_sizes(T: int, B: int, D: int, N: int, G: int = 1, dtype=torch.float32):
    """(saved_bytes, forward_bytes, backward_bytes) of ``ck_scan_sizes``."""
    s, f, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    shape = ScanShape(int(T), int(B), int(D), int(N), int(G), _DTYPES[dtype], 0)
    _check(lib().ck_scan_sizes(ctypes.byref(shape), ctypes.byref(s), ctypes.byref(f),
                               ctypes.byref(b)))
    return s.value, f.value, b.value


def _scan_sizes(shape):
    s, f, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().ck_scan_sizes(ctypes.byref(shape), ctypes.byref(s), ctypes.byref(f),
                               ctypes.byref(b)))
    return s.value, f.value, b.value


def selective_scan_forward(u, delta, A, B, C, D=None, z=None, delta_bias=None, state0=None,
                           lengths=None, delta_softplus: bool = False, save: bool = True,
                           out=None, state=None, saved=None, workspace=None, stream=None):
    """Run ``ck_scan_forward``; returns (out, state, saved, workspace).

    u, delta, z: [T, B, D]; B, C: [T, B, G, N]; A: [D, N]; D, delta_bias: [D];
    state0 and the returned state: [B, D, N].  ``saved`` is what
    ``selective_scan_backward`` needs (None with save=False)."""
    shape, inp = _scan_call(u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus)
    sb, fb, _ = _scan_sizes(shape)
    out, m0 = _into(out, "out", u, u.shape)
    state, m1 = _into(state, "state", u, (shape.B, shape.D, shape.N), torch.float32)
    m2, m3 = saved is None, workspace is None
    saved = _buffer(saved, sb, u, "saved") if save or not m2 else None
    workspace = _buffer(workspace, fb, u, "workspace")
    o = _seq(out, "out", u, u.shape)
    st = _par(state, "state", u, (shape.B, shape.D, shape.N))
    _On(u.device, stream)(
        lib().ck_scan_forward, ctypes.byref(shape), ctypes.byref(inp), o, st, _ptr(saved),
        _ptr(workspace), _bytes(workspace),
        made=(out if m0 else None, state if m1 else None, saved if m2 else None,
              workspace if m3 else None))
    return out, state, saved, workspace


def selective_scan_backward(u, delta, A, B, C, saved, grad_out, D=None, z=None, delta_bias=None,
                            lengths=None, delta_softplus: bool = False, grad_state=None,
                            grads=None, workspace=None, stream=None) -> dict:
    """Run ``ck_scan_backward``; returns the gradients (overwritten) by the
    names g_u, g_delta, g_A, g_B, g_C, g_D, g_delta_bias, g_state0 and, with a
    gate, g_z."""
    shape, inp = _scan_call(u, delta, A, B, C, D, z, delta_bias, None, lengths, delta_softplus)
    sb, _, wb = _scan_sizes(shape)
    saved = _buffer(saved, sb, u, "saved") if sb else None
    if sb and saved is None:
        raise ValueError("saved is missing")
    go = _seq(grad_out, "grad_out", u, u.shape)
    state = (shape.B, shape.D, shape.N)
    gs = _par(grad_state, "grad_state", u, state)
    m0, m1 = grads is None, workspace is None
    if m0:
        f = dict(dtype=torch.float32, device=u.device)
        grads = {"g_u": torch.empty(u.shape, dtype=u.dtype, device=u.device),
                 "g_delta": torch.empty(u.shape, dtype=u.dtype, device=u.device),
                 "g_A": torch.empty(A.shape, **f),
                 "g_B": torch.empty(B.shape, dtype=u.dtype, device=u.device),
                 "g_C": torch.empty(B.shape, dtype=u.dtype, device=u.device),
                 "g_D": torch.empty(shape.D, **f), "g_delta_bias": torch.empty(shape.D, **f),
                 "g_state0": torch.empty(state, **f)}
        if z is not None:
            grads["g_z"] = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    g = grads
    out = ScanGrads(
        _seq(g["g_u"], "g_u", u, u.shape), _seq(g["g_delta"], "g_delta", u, u.shape),
        _seq(g["g_B"], "g_B", u, B.shape, 2), _seq(g["g_C"], "g_C", u, B.shape, 2),
        CkSeq(None, 0, 0) if z is None else _seq(g["g_z"], "g_z", u, u.shape),
        _par(g["g_A"], "g_A", u, A.shape), _par(g.get("g_D"), "g_D", u, (shape.D,)),
        _par(g.get("g_delta_bias"), "g_delta_bias", u, (shape.D,)),
        _par(g.get("g_state0"), "g_state0", u, state))
    workspace = _buffer(workspace, wb, u, "workspace")
    _On(u.device, stream)(
        lib().ck_scan_backward, ctypes.byref(shape), ctypes.byref(inp), _ptr(saved), go, gs,
        ctypes.byref(out), _ptr(workspace), _bytes(workspace),
        made=(tuple(grads.values()) if m0 else ()) + ((workspace,) if m1 else ()))
    return grads


def selective_scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                        delta_softplus: bool = False, out=None, new_state=None, stream=None):
    """Run ``ck_scan_step``: one token per row.  u, delta, z: [B, D]; B, C:
    [B, G, N]; state: [B, D, N], updated in place unless ``new_state`` is
    given.  Returns (out [B, D], the new state)."""
    shape, inp = _scan_call(u, delta, A, B, C, D, z, delta_bias, state, None, delta_softplus,
                            step=True)
    if state is None:
        raise ValueError("state is missing")
    new_state = state if new_state is None else new_state
    out, made = _into(out, "out", u, u.shape)
    o = _seq(out, "out", u, u.shape)
    st = _par(new_state, "new_state", u, (shape.B, shape.D, shape.N))
    _On(u.device, stream)(lib().ck_scan_step, ctypes.byref(shape), ctypes.byref(inp), o, st,
                          made=(out,) if made else ())
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
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus):
        u, delta, z, B, C = _rows(u), _rows(delta), _rows(z), _groups(B), _groups(C)
        A, D, delta_bias, state0 = (_cont(t) for t in (A, D, delta_bias, state0))
        out, state, saved, _ = selective_scan_forward(
            u, delta, A, B, C, D, z, delta_bias, state0, lengths, delta_softplus,
            save=any(ctx.needs_input_grad))
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
                g["g_state0"] if ctx.needs_input_grad[8] else None, None, None)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, state0=None, lengths=None,
                   delta_softplus: bool = False):
    """The selective scan as one autograd node: returns (out [T, B, D], the
    state after each row's last step [B, D, N]); gradients reach every tensor
    argument but ``lengths``.  Shapes as for ``selective_scan_forward``."""
    return _SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, state0, lengths,
                                bool(delta_softplus))


# --------------------------------------------------------- short convolution

def _conv_call(x, weight, bias, activation, step=False):
    _first(x, "x", (2,) if step else (3,))
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [channels, taps] tensor")
    T, rows, ch = (1,) + tuple(x.shape) if step else tuple(x.shape)
    W = weight.shape[1]
    shape = ConvShape(T, rows, ch, W, _DTYPES[x.dtype], 1 if activation else 0)
    return (shape, (W - 1, rows, ch), _seq(x, "x", x, x.shape),
            _par(weight, "weight", x, (ch, W)), _par(bias, "bias", x, (ch,)))


def short_conv_forward(x, weight, bias=None, state0=None, lengths=None, activation=None, y=None,
                       state=None, stream=None):
    """Run ``ck_conv_forward``; returns (y, state).  x: [T, B, D]; weight:
    [D, W]; bias: [D]; state0 and the returned state: [W - 1, B, D], the last
    inputs of each row; activation: None or "silu"."""
    shape, sshape, xs, w, b = _conv_call(x, weight, bias, activation)
    s0 = _par(state0, "state0", x, sshape, x.dtype)
    ln = _par(lengths, "lengths", x, (shape.B,), torch.int32)
    y, m0 = _into(y, "y", x, x.shape)
    state, m1 = _into(state, "state", x, sshape)
    ys, st = _seq(y, "y", x, x.shape), _par(state, "state", x, sshape, x.dtype)
    _On(x.device, stream)(lib().ck_conv_forward, ctypes.byref(shape), xs, w, b, s0, ln, ys, st,
                          made=(y if m0 else None, state if m1 else None))
    return y, state


def short_conv_backward(x, weight, grad_y, bias=None, state0=None, lengths=None, activation=None,
                        grad_state=None, grads=None, workspace=None, stream=None) -> dict:
    """Run ``ck_conv_backward``; returns the gradients (overwritten) g_x,
    g_weight, g_bias and g_state0."""
    shape, sshape, xs, w, b = _conv_call(x, weight, bias, activation)
    s0 = _par(state0, "state0", x, sshape, x.dtype)
    ln = _par(lengths, "lengths", x, (shape.B,), torch.int32)
    gy = _seq(grad_y, "grad_y", x, x.shape)
    gs = _par(grad_state, "grad_state", x, sshape, x.dtype)
    need = ctypes.c_size_t()
    _check(lib().ck_conv_sizes(ctypes.byref(shape), ctypes.byref(need)))
    m0, m1 = grads is None, workspace is None
    if m0:
        f = dict(dtype=torch.float32, device=x.device)
        grads = {"g_x": torch.empty(x.shape, dtype=x.dtype, device=x.device),
                 "g_weight": torch.empty(weight.shape, **f), "g_bias": torch.empty(shape.D, **f),
                 "g_state0": torch.empty(sshape, dtype=x.dtype, device=x.device)}
    workspace = _buffer(workspace, need.value, x, "workspace")
    gx = _seq(grads["g_x"], "g_x", x, x.shape)
    gw = _par(grads["g_weight"], "g_weight", x, weight.shape)
    gb = _par(grads.get("g_bias"), "g_bias", x, (shape.D,))
    gs0 = _par(grads.get("g_state0"), "g_state0", x, sshape, x.dtype)
    _On(x.device, stream)(
        lib().ck_conv_backward, ctypes.byref(shape), xs, w, b, s0, ln, gy, gs, gx, gw, gb, gs0,
        _ptr(workspace), _bytes(workspace),
        made=(tuple(grads.values()) if m0 else ()) + ((workspace,) if m1 else ()))
    return grads


def short_conv_step(state, x, weight, bias=None, activation=None, y=None, new_state=None,
                    stream=None):
    """Run ``ck_conv_step``: one token per row.  x: [B, D]; state: [W - 1, B,
    D], updated in place unless ``new_state`` is given.  Returns (y [B, D],
    the new state)."""
    shape, sshape, xs, w, b = _conv_call(x, weight, bias, activation, step=True)
    s0 = _par(state, "state", x, sshape, x.dtype)
    new_state = state if new_state is None else new_state
    y, made = _into(y, "y", x, x.shape)
    ys, st = _seq(y, "y", x, x.shape), _par(new_state, "new_state", x, sshape, x.dtype)
    _On(x.device, stream)(lib().ck_conv_step, ctypes.byref(shape), xs, w, b, s0, ys, st,
                          made=(y,) if made else ())
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
    _first(x, name, (2, 3))
    T, rows, ch = (1,) + tuple(x.shape) if x.dim() == 2 else tuple(x.shape)
    m = 0xFFFFFFFFFFFFFFFF
    shape = DropoutShape(T, rows, ch, _DTYPES[x.dtype], 1 if held else 0, float(p), int(seed) & m,
                         int(offset) & m, _par(counter, "counter", x, (1,), torch.int64))
    return shape, _seq(x, name, x, x.shape)


def dropout_forward(x, p: float, seed: int, offset: int = 0, residual=None, held: bool = False,
                    counter=None, out=None, stream=None) -> torch.Tensor:
    """Run ``ck_dropout_forward`` on x [T, B, D] (or one step's [B, D]):
    residual + x / (1 - p) where kept, with p rounded to a multiple of 2^-16.
    The mask follows from (seed, offset) alone; held=True gives all steps of a
    window the same mask.  A device ``counter`` (int64 [1]) is added to the
    offset, so that a replayed graph can draw new masks.  ``out`` may be x or
    the residual."""
    shape, xs = _drop_call(x, "x", p, seed, offset, held, counter)
    rs = CkSeq(None, 0, 0) if residual is None else _seq(residual, "residual", x, x.shape)
    out, made = _into(out, "out", x, x.shape)
    o = _seq(out, "out", x, x.shape)
    _On(x.device, stream)(lib().ck_dropout_forward, ctypes.byref(shape), xs, rs, o,
                          made=(out,) if made else ())
    return out


def dropout_backward(grad_out, p: float, seed: int, offset: int = 0, held: bool = False,
                     counter=None, grad_x=None, stream=None) -> torch.Tensor:
    """Run ``ck_dropout_backward``: the forward's mask and scale on grad_out."""
    shape, gs = _drop_call(grad_out, "grad_out", p, seed, offset, held, counter)
    grad_x, made = _into(grad_x, "grad_x", grad_out, grad_out.shape)
    o = _seq(grad_x, "grad_x", grad_out, grad_out.shape)
    _On(grad_out.device, stream)(lib().ck_dropout_backward, ctypes.byref(shape), gs, o,
                                 made=(grad_x,) if made else ())
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
