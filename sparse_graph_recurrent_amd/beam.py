"""Beam search's step, for a model that answers with several beams a text: the
selection of the best continuations, and the reordering of the states that the
beams carry (the convolution's, the scans', the recurrence's).

    scores, parents, tokens, finished = beam_select(logits, scores, finished, eos)
    beam_reorder([conv_state.transpose(0, 1), scan_state, node_state], parents)

Row b K + k of a state is beam k of text b.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _check, _on_stream, lib
from .sequence import CkSeq, _DTYPES, _buffer, _call, _first, _par, _seq, _written


class BeamShape(ctypes.Structure):
    """ck_beam_shape of include/ck.h."""
    _fields_ = [("B", ctypes.c_int64), ("K", ctypes.c_int64), ("V", ctypes.c_int64),
                ("eos", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class BeamState(ctypes.Structure):
    """ck_beam_state of include/ck.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("segments", "bytes", "in_row", "in_segment",
                                              "out_row", "out_segment")]


_SHAPE = struct.Struct("=4qi4x")
assert _SHAPE.size == ctypes.sizeof(BeamShape)


@functools.lru_cache(maxsize=64)
def _states(count: int) -> struct.Struct:
    """`count` ck_beam_state as packed bytes."""
    return struct.Struct("=" + "2Q6q" * count)


assert _states(1).size == ctypes.sizeof(BeamState)


def _declare(L: ctypes.CDLL) -> None:
    p, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
    L.ck_beam_sizes.argtypes = [p, ctypes.POINTER(sz)]
    L.ck_beam_select.argtypes = [p, CkSeq, p, p, p, p, p, p, p, sz, p]
    L.ck_beam_reorder.argtypes = [p, i64, p, i64, i64, p]


@functools.lru_cache(maxsize=64)
def _sizes(shape: bytes) -> int:
    need = ctypes.c_size_t()
    _check(lib().ck_beam_sizes(shape, ctypes.byref(need)))
    return need.value


def beam_select(logits, scores, finished=None, eos=None, out=None, workspace=None, stream=None):
    """Run ``ck_beam_select``: the K best continuations of each text, best first.

    logits: [B, K, V] (fp32, bf16 or fp16; adjacent tokens, any other strides);
    scores: fp32 [B, K]; finished: bool [B, K], beams that go on with the token
    ``eos`` alone.  Returns (scores fp32, parents int64, tokens int64, finished
    bool or None without eos), each [B, K]; ``out``: such a tuple to write."""
    if stream is not None:
        for t in out or ():
            if t is not None and t.device != stream.device:
                raise ValueError(f"a tensor is on {t.device}, the stream on {stream.device}")
        return _on_stream(stream, beam_select, logits, scores, finished, eos, out, workspace)
    dev = _first(logits, "logits", (3,))
    B, K, V = logits.shape
    if finished is not None and eos is None:
        raise ValueError("finished beams go on with an end token: eos is missing")
    if eos is not None and not 0 <= eos < V:
        raise ValueError(f"eos must be in [0, {V}), got {eos}")
    shape = _SHAPE.pack(B, K, V, -1 if eos is None else eos, _DTYPES[logits.dtype])
    need = _sizes(shape)
    bk = (B, K)
    x = CkSeq(*_seq(logits, "logits", logits.dtype, dev, logits.shape))
    if scores is None:
        raise ValueError("scores are missing")
    sp = _par(scores, "scores", dev, bk)
    fp = _par(finished, "finished", dev, bk, torch.bool)
    if out is None:
        new = torch.empty_like(scores)
        parents = torch.empty(bk, dtype=torch.int64, device=logits.device)
        tokens = torch.empty_like(parents)
        ends = None if eos is None else torch.empty(bk, dtype=torch.bool, device=logits.device)
        ptrs = (new.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                0 if ends is None else ends.data_ptr())
    else:
        new, parents, tokens, ends = out
        if new is None or parents is None or tokens is None:
            raise ValueError("out must hold scores, parents and tokens")
        ptrs = (_par(new, "out scores", dev, bk), _par(parents, "out parents", dev, bk, torch.int64),
                _par(tokens, "out tokens", dev, bk, torch.int64),
                _par(ends, "out finished", dev, bk, torch.bool))
        _written(tuple(t for t in out if t is not None))
    workspace, wp, wn = _buffer(workspace, need, logits, "workspace")
    _call(lib().ck_beam_select, dev, (shape, x, sp, fp, *ptrs, wp, wn))
    return new, parents, tokens, ends


def _pieces(t: torch.Tensor):
    """(segments, elements, row stride, segment stride) of a state's rows, in elements."""
    if t.is_contiguous():
        n = t.numel() // t.shape[0]
        return 1, n, n, 0
    inner, segs, seg = 1, 1, 0
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size == 1:
            continue
        if segs == 1 and stride == inner:
            inner *= size
        elif segs == 1:
            segs, seg = size, stride
        elif stride == segs * seg:
            segs *= size
        else:
            raise ValueError("a state's row must be pieces of adjacent elements that lie "
                             "equally far apart")
    return segs, inner, t.stride(0) if t.shape[0] > 1 else 0, seg


def beam_reorder(states, parents, out=None, stream=None):
    """Run ``ck_beam_reorder``: row b K + j of every state becomes what row
    b K + parents[b, j] was.  states: tensors of any type whose first dimension
    is B K (pass ``conv_state.transpose(0, 1)`` for one that has its rows
    second); parents: int64 [B, K] in [0, K).  In place, or into ``out``, a
    tensor for each state that does not overlap it.  Returns the new states."""
    states = tuple(states)
    outs = states if out is None else tuple(out)
    if len(outs) != len(states):
        raise ValueError(f"{len(states)} states, {len(outs)} outputs")
    if stream is not None:
        for t in states + outs:
            if isinstance(t, torch.Tensor) and t.device != stream.device:
                raise ValueError(f"a tensor is on {t.device}, the stream on {stream.device}")
        return _on_stream(stream, beam_reorder, states, parents, None if out is None else outs)
    if not isinstance(parents, torch.Tensor) or not parents.is_cuda or parents.dim() != 2:
        raise TypeError("parents must be a CUDA (HIP) int64 tensor [texts, beams]")
    dev = parents.get_device()
    B, K = parents.shape
    pp = _par(parents, "parents", dev, (B, K), torch.int64)
    args = []
    for n, (t, o) in enumerate(zip(states, outs)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() < 1:
            raise TypeError(f"state {n} must be a CUDA (HIP) tensor")
        if t.get_device() != dev:
            raise ValueError(f"state {n} is on {t.device}, not on cuda:{dev}")
        if t.shape[0] != B * K:
            raise ValueError(f"state {n} must have {B * K} rows, got {t.shape[0]}")
        if t.numel() == 0:
            continue
        segs, inner, row, seg = _pieces(t)
        o_segs, o_inner, o_row, o_seg = segs, inner, row, seg
        if o is not t:
            if not (isinstance(o, torch.Tensor) and o.dtype is t.dtype and o.shape == t.shape
                    and o.get_device() == dev):
                raise ValueError(f"output {n} must have its state's type, shape and device")
            o_segs, o_inner, o_row, o_seg = _pieces(o)
            if o_inner != inner:  # the longer pieces as some of the shorter
                if segs == 1:
                    segs, inner, seg = o_segs, o_inner, o_inner
                elif o_segs == 1:
                    o_segs, o_inner, o_seg = segs, inner, inner
                if o_inner != inner:
                    raise ValueError(f"output {n} must have its state's layout within a row")
        e = t.element_size()
        args += (t.data_ptr(), o.data_ptr(), segs, inner * e, row * e, seg * e, o_row * e,
                 o_seg * e)
    count = len(args) // 8
    _call(lib().ck_beam_reorder, dev,
          (_states(count).pack(*args) if count else None, count, pp, B, K))
    if outs:
        _written(outs)
    return outs


__all__ = ["beam_select", "beam_reorder"]
