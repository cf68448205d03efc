"""Calls of the gated scan whose outputs lie over what they read or over one another are
refused before any device work, where addresses, sizes and strides show it."""
import ctypes
import os

import pytest

import sparse_graph_recurrent_amd as sgr
from sparse_graph_recurrent_amd.sequence import CkSeq, GatedGrads, GatedInputs, GatedShape

BAD_VALUE = 12
T, B, D = 40, 2, 65     # bf16: the last group of channels shares one with the group before
ROW, STEP = D, B * D    # strides of a contiguous tensor, in elements
SIZE = 1 << 24          # apart from one another: never read or written, every call fails
NONE = CkSeq(None, 0, 0)
NAMES = ("x", "f", "i", "z", "go", "out", "gx", "gf", "gi", "gz", "state0", "state", "gstate",
         "gstate0", "f_bias", "i_bias", "gf_bias", "gi_bias", "lengths", "saved", "ws")
AT = {n: SIZE * (k + 1) for k, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sgr.LIB_PATH):
        from sparse_graph_recurrent_amd import build
        build.build()
    return sgr.lib()


def seq(at):
    return at if isinstance(at, CkSeq) else CkSeq(at, STEP, ROW)


def inputs(a, state0=True, lengths=True):
    return ctypes.byref(GatedInputs(seq(a["x"]), seq(a["f"]), seq(a["i"]), seq(a["z"]), a["f_bias"],
                                    a["i_bias"], a["state0"] if state0 else None,
                                    a["lengths"] if lengths else None))


def shape(steps=T, dtype=1):
    return ctypes.byref(GatedShape(steps, B, D, dtype))


def forward(L, **kw):
    a = {**AT, **kw}
    return L.ck_gated_forward(shape(), inputs(a), seq(a["out"]), a["state"], a["saved"], a["ws"],
                              2**40, None)


def backward(L, **kw):
    a = {**AT, **kw}
    g = ctypes.byref(GatedGrads(seq(a["gx"]), seq(a["gf"]), seq(a["gi"]), seq(a["gz"]),
                                a["gf_bias"], a["gi_bias"], a["gstate0"]))
    return L.ck_gated_backward(shape(), inputs(a), a["saved"], seq(a["go"]), a["gstate"], g,
                               a["ws"], 2**40, None)


def step(L, dtype=1, **kw):
    a = {**AT, **kw}
    return L.ck_gated_step(shape(1, dtype), inputs(a, lengths=False), seq(a["out"]), a["state"],
                           None)


def refused(L, status, *names):
    assert status == BAD_VALUE
    text = L.ck_last_error().decode()
    assert "must not lie over" in text and all(n in text for n in names), text


@pytest.mark.parametrize("over", ["x", "f", "i", "z"])
def test_forward_output_over_an_input(L, over):
    a = AT[over]
    for out in (a, a + 2, a + 2 * (T * STEP - 1), a - 2 * (T * STEP - 1),
                CkSeq(a, 4 * STEP, 4 * ROW), CkSeq(a + 64, D, T * D)):
        refused(L, forward(L, out=out), "out", over)


def test_forward_slices_of_one_tensor(L):
    wide = 4 * D    # of a projection: x is its first slice
    x = CkSeq(AT["x"], B * wide, wide)
    for by in (1, D - 1, -1):
        refused(L, forward(L, x=x, out=CkSeq(AT["x"] + 2 * by, B * wide, wide)), "out", "x")
    refused(L, forward(L, x=x, out=CkSeq(AT["x"] + 2 * (7 * B * wide + D - 1), B * wide, wide)),
            "out", "x")
    # x the same at every step and row
    refused(L, forward(L, x=CkSeq(AT["out"] + 2 * (T * STEP - 1), 0, 0)), "out", "x")


def test_forward_states_and_buffers(L):
    row = 4 * D
    refused(L, forward(L, state=AT["state0"]), "state", "state0")
    refused(L, forward(L, state=AT["state0"] + row), "state", "state0")    # a row into it
    refused(L, forward(L, state=AT["out"]), "state", "out")
    refused(L, forward(L, state=AT["f_bias"] + 4 * D - 4), "state", "f_bias")
    refused(L, forward(L, state=AT["lengths"]), "state", "lengths")
    refused(L, forward(L, saved=AT["z"]), "saved", "z")
    refused(L, forward(L, saved=AT["out"]), "saved", "out")
    refused(L, forward(L, lengths=AT["out"]), "out", "lengths")


@pytest.mark.parametrize("grad", ["gx", "gf", "gi", "gz"])
def test_backward_gradients(L, grad):
    for over in ("x", "f", "i", "z", "go"):
        refused(L, backward(L, **{grad: AT[over]}), over if over != "go" else "grad_out")
    for other in {"gx", "gf", "gi", "gz"} - {grad}:
        refused(L, backward(L, **{grad: AT[other] + 2}), "gradient of")
    refused(L, backward(L, **{grad: AT["saved"]}), "saved")


def test_backward_states_and_biases(L):
    refused(L, backward(L, gstate0=AT["gstate"]), "state0", "grad_state")
    refused(L, backward(L, gstate0=AT["gstate"] + 4 * D), "state0", "grad_state")
    refused(L, backward(L, gf_bias=AT["f_bias"]), "f_bias")
    refused(L, backward(L, gf_bias=AT["gi_bias"]), "gradient of f_bias", "gradient of i_bias")
    refused(L, backward(L, gi_bias=AT["i_bias"] + 4), "i_bias")
    refused(L, backward(L, gf_bias=AT["gx"] + 4), "gradient")


def test_step_in_place_but_no_other_way(L):
    refused(L, step(L, out=AT["x"] + 2), "out", "x")
    refused(L, step(L, out=CkSeq(AT["x"], 0, 2 * D)), "out", "x")
    refused(L, step(L, state=AT["state0"] + 4), "state", "state0")
    refused(L, step(L, state=AT["state0"] - 4 * D), "state", "state0")
    refused(L, step(L, dtype=0, out=AT["state"]), "out", "state")
    refused(L, step(L, out=AT["f_bias"]), "out", "f_bias")
