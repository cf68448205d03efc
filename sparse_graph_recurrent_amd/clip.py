"""The norm of a model's gradients and their scaling to a limit, as a training
step runs them between its backward and its optimizer:

    grads = [p.grad for p in model.parameters() if p.grad is not None]
    norm, _ = clip_grad_norm(grads, 1.0)

Backpropagation through a window of the recurrence multiplies by its steps'
derivatives once a microstep; a limit on the whole gradient's norm keeps one
steep window from undoing what many have learned.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _check, _on_stream, lib
from .sequence import _DTYPES, _buffer, _call, _written


class ClipTensor(ctypes.Structure):
    """ck_clip_tensor of include/ck.h."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


@functools.lru_cache(maxsize=64)
def _table(count: int) -> struct.Struct:
    """`count` ck_clip_tensor as packed bytes."""
    return struct.Struct("=" + "2Qqi4x" * count)


assert _table(1).size == ctypes.sizeof(ClipTensor)


def _declare(L: ctypes.CDLL) -> None:
    p, sz = ctypes.c_void_p, ctypes.c_size_t
    L.ck_clip_sizes.argtypes = [ctypes.c_int64, ctypes.POINTER(sz)]
    L.ck_clip_grad_norm.argtypes = [p, ctypes.c_int64, ctypes.c_double, p, p, sz, p]


@functools.lru_cache(maxsize=64)
def _sizes(count: int) -> int:
    need = ctypes.c_size_t()
    _check(lib().ck_clip_sizes(count, ctypes.byref(need)))
    return need.value


def _dense(t: torch.Tensor) -> bool:
    """True when t's elements fill its memory without gaps, in any order of dimensions."""
    want = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != want:
            return t.numel() == 0
        want *= size
    return True


def _refuse(t, name: str, dev: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} has gaps between its elements, or some that are one")


def _run(grads, outs, max_norm: float, norm, workspace, device):
    """One call; outs: the tensors that are written (None: none)."""
    count = len(grads)
    if count:
        if not isinstance(grads[0], torch.Tensor) or not grads[0].is_cuda:
            raise TypeError("gradient 0 must be a CUDA (HIP) tensor")
        dev = grads[0].get_device()
    else:
        dev = torch.device("cuda" if device is None else device).index
        dev = torch.cuda.current_device() if dev is None else dev
    args, last, code = [], None, None
    same = outs is grads
    for k, t in enumerate(grads):
        dtype = t.dtype if isinstance(t, torch.Tensor) else None
        if dtype is not last:
            last, code = dtype, _DTYPES.get(dtype)
        if code is None or t.get_device() != dev or not (t.is_contiguous() or _dense(t)):
            _refuse(t, f"gradient {k}", dev)
        at = t.data_ptr()
        to = at if same else 0
        if not same and outs is not None:
            o = outs[k]
            if not (isinstance(o, torch.Tensor) and o.dtype is dtype and o.shape == t.shape
                    and o.get_device() == dev and (o.stride() == t.stride() or o.is_contiguous()
                                                   and t.is_contiguous())):
                raise ValueError(f"output {k} must be on cuda:{dev}, with its gradient's type, "
                                 "shape and strides")
            to = o.data_ptr()
        args += (at, to, t.numel(), code)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=f"cuda:{dev}")
    elif not (isinstance(norm, torch.Tensor) and norm.dtype is torch.float32
              and norm.shape == (1,) and norm.get_device() == dev):
        raise ValueError(f"norm must be fp32 [1] on cuda:{dev}")
    else:
        _written((norm,))
    workspace, wp, wn = _buffer(workspace, _sizes(count), norm, "workspace")
    _call(lib().ck_clip_grad_norm, dev,
          (_table(count).pack(*args) if count else None, count, max_norm, norm.data_ptr(), wp, wn))
    if outs:
        _written(tuple(outs))
    return norm


def _streamed(stream, tensors):
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.device != stream.device:
            raise ValueError(f"a tensor is on {t.device}, the stream on {stream.device}")


def grad_norm(grads, norm=None, workspace=None, stream=None) -> torch.Tensor:
    """The norm (fp32 [1], on the device) of all tensors in ``grads`` together,
    by ``ck_clip_grad_norm``; nothing is scaled."""
    grads = list(grads)
    if stream is not None:
        _streamed(stream, grads)
        return _on_stream(stream, grad_norm, grads, norm, workspace)
    return _run(grads, None, float("inf"), norm, workspace, None)


def clip_grad_norm(grads, max_norm: float, out=None, norm=None, workspace=None, stream=None):
    """Run ``ck_clip_grad_norm``: scales the tensors of ``grads`` (fp32, bf16 or
    fp16, mixed as they come; each without gaps) so that their norm together is
    at most ``max_norm``.  In place, or into ``out``, a tensor for each.
    Returns (the norm before, fp32 [1] on the device; the scaled tensors).  A
    norm that is not finite scales nothing.  (``torch.nn.utils.clip_grad_norm_``
    takes parameters, leaves out those without a gradient, adds 1e-6 to the norm
    that it divides by, and scales by a norm that is not finite as well.)"""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(grads)} gradients, {len(outs)} outputs")
    if stream is not None:
        _streamed(stream, grads + outs)
        return _on_stream(stream, clip_grad_norm, grads, max_norm, None if out is None else outs,
                          norm, workspace)
    norm = _run(grads, outs, float(max_norm), norm, workspace, None)
    return norm, tuple(outs)


__all__ = ["clip_grad_norm", "grad_norm"]
