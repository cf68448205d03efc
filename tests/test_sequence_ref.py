"""The fp64 definitions the GPU tests of the sequence operators compare with:
gradient formulas against central differences, the generator against its
published test vectors, and host-side refusals of the entry points (checked
before any device work)."""
import ctypes
import os

import numpy as np
import pytest

import sequence_ref as ref
import sparse_graph_recurrent_amd as sgr
from sparse_graph_recurrent_amd.sequence import (CkSeq, ConvShape, DropoutShape, ScanGrads,
                                                 ScanInputs, ScanShape)


def _differences(f, x, loss, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        hi = loss(f())
        x[i] = old - eps
        lo = loss(f())
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("gate,softplus,lengths", [(True, True, None), (False, False, None),
                                                   (True, True, [0, 3, 5])])
def test_scan_gradient_formulas_against_differences(gate, softplus, lengths):
    r = np.random.default_rng(3)
    T, B, D, N, G = 5, 3, 4, 3, 2
    p = {"u": r.standard_normal((T, B, D)), "delta": 0.5 + 0.3 * r.standard_normal((T, B, D)),
         "A": -r.uniform(0.2, 2, (D, N)), "B": r.standard_normal((T, B, G, N)),
         "C": r.standard_normal((T, B, G, N)), "D": r.standard_normal(D),
         "z": r.standard_normal((T, B, D)) if gate else None,
         "delta_bias": 0.1 * r.standard_normal(D), "state0": r.standard_normal((B, D, N)),
         "lengths": None if lengths is None else np.array(lengths), "softplus": softplus}
    go, gs = r.standard_normal((T, B, D)), r.standard_normal((B, D, N))
    got = ref.scan({**p, "go": go, "gstate": gs})
    loss = lambda o: (o["out"] * go).sum() + (o["state"] * gs).sum()
    for k in ("u", "delta", "A", "B", "C", "D", "delta_bias", "state0") + (("z",) if gate else ()):
        want = _differences(lambda: ref.scan(p), p[k], loss)
        # central differences of a smooth function: about 1e-9 of the values
        np.testing.assert_allclose(got["g_" + k], want, rtol=1e-6, atol=1e-7, err_msg=k)


@pytest.mark.parametrize("silu,W,lengths", [(True, 4, None), (False, 3, [0, 1, 6]),
                                            (True, 1, None)])
def test_conv_gradient_formulas_against_differences(silu, W, lengths):
    r = np.random.default_rng(4)
    T, B, D = 6, 3, 2
    p = {"x": r.standard_normal((T, B, D)), "weight": r.standard_normal((D, W)),
         "bias": r.standard_normal(D), "state0": r.standard_normal((W - 1, B, D)), "silu": silu,
         "lengths": None if lengths is None else np.array(lengths)}
    gy, gs = r.standard_normal((T, B, D)), r.standard_normal((W - 1, B, D))
    got = ref.conv({**p, "gy": gy, "gstate": gs})
    loss = lambda o: (o["y"] * gy).sum() + (o["state"] * gs).sum()
    for k in ("x", "weight", "bias", "state0"):
        want = _differences(lambda: ref.conv(p), p[k], loss)
        np.testing.assert_allclose(got["g_" + k], want, rtol=1e-6, atol=1e-7, err_msg=k)


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_published_vectors(counter, key, want):
    got = ref.philox(np.array(counter, np.uint64), key)
    assert tuple(int(v) for v in got) == want


def test_keep_fraction():
    m, scale = ref.keep(50, 4, 1000, 0.3, 5, 9, False)
    n = m.size  # the fraction's standard deviation is sqrt(p (1 - p) / n)
    assert abs(m.mean() - 0.7) < 5 * np.sqrt(0.21 / n)
    assert scale == 65536 / (65536 - 19661)


# ------------------------------------------------------- refusals (no device)

NULL_ARG, BAD_SIZE, TOO_LARGE, WORKSPACE, BAD_VALUE = 1, 2, 5, 6, 12
FAKE = 0x10000  # never dereferenced: validation fails before any device work
SEQ, NONE = CkSeq(FAKE, 64, 64), CkSeq(None, 0, 0)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sgr.LIB_PATH):
        from sparse_graph_recurrent_amd import build
        build.build()
    return sgr.lib()


def _scan(**kw):
    return ctypes.byref(ScanShape(*[kw.get(k, v) for k, v in dict(
        T=8, B=2, D=64, N=16, G=1, dtype=1, delta_softplus=1).items()]))


def _inputs(**kw):
    v = dict(u=SEQ, delta=SEQ, b=SEQ, c=SEQ, z=NONE, a=FAKE, d=None, delta_bias=None, state0=None,
             lengths=None)
    v.update(kw)
    return ctypes.byref(ScanInputs(*v.values()))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD_SIZE), (dict(B=0), BAD_SIZE), (dict(D=0), BAD_SIZE), (dict(N=0), BAD_SIZE),
    (dict(N=65), BAD_SIZE), (dict(G=0), BAD_SIZE), (dict(G=3), BAD_SIZE), (dict(G=128), BAD_SIZE),
    (dict(T=2**31), TOO_LARGE), (dict(B=2**31), TOO_LARGE), (dict(D=2**31), TOO_LARGE),
    (dict(B=2**30, D=2**10), TOO_LARGE), (dict(D=2**28, N=1), TOO_LARGE),
    (dict(D=2**26, G=2**26, N=16), TOO_LARGE), (dict(T=2**30, B=2**20, D=64), TOO_LARGE),
    (dict(dtype=3), BAD_VALUE), (dict(dtype=-1), BAD_VALUE)])
def test_scan_shape_refusals(L, kw, status):
    s = ctypes.c_size_t()
    assert L.ck_scan_sizes(_scan(**kw), ctypes.byref(s), None, None) == status
    assert L.ck_scan_forward(_scan(**kw), _inputs(), SEQ, None, None, None, 0, None) == status
    assert L.ck_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(u=NONE), NULL_ARG), (dict(delta=NONE), NULL_ARG), (dict(b=NONE), NULL_ARG),
    (dict(c=NONE), NULL_ARG), (dict(a=None), NULL_ARG),
    (dict(u=CkSeq(FAKE + 1, 64, 64)), BAD_VALUE), (dict(z=CkSeq(FAKE, -64, 64)), BAD_VALUE),
    (dict(delta=CkSeq(FAKE, 64, -1)), BAD_VALUE), (dict(c=CkSeq(FAKE, 2**24, 64)), BAD_VALUE)])
def test_scan_input_refusals(L, kw, status):
    assert L.ck_scan_forward(_scan(), _inputs(**kw), SEQ, None, None, FAKE, 2**40, None) == status
    assert L.ck_scan_step(_scan(T=1), _inputs(**kw), SEQ, FAKE, None) == status


def test_sizes_beyond_the_kernels_counts_are_refused(L):
    """32-bit steps and channels need room for a tile's or workgroup's end, and a
    launch has fewer than 2^32 threads: sizes that were taken until they did not
    launch, or wrapped."""
    s = ctypes.c_size_t()
    end = 2**31 - 8
    for kw in (dict(T=end, B=1, D=1), dict(T=1, B=2**24, D=64), dict(T=1, B=2**18, D=64 * 64, G=64)):
        assert L.ck_scan_sizes(_scan(N=1, **kw), ctypes.byref(s), None, None) == TOO_LARGE, kw
    assert L.ck_scan_sizes(_scan(N=1, T=1, B=2**24 - 1), ctypes.byref(s), None, None) == 0
    for kw in (dict(T=end, B=1, D=1), dict(T=1, B=1, D=end), dict(T=1, B=2**24, D=2**11)):
        assert L.ck_conv_sizes(_conv(**kw), ctypes.byref(s)) == TOO_LARGE, kw
    assert L.ck_conv_sizes(_conv(T=1, B=2**22, D=2**11), ctypes.byref(s)) == 0
    for T, D in ((end, 1), (1, end)):
        d = ctypes.byref(DropoutShape(T, 1, D, 1, 0, 0.5, 1, 0, None))
        assert L.ck_dropout_forward(d, NONE, NONE, NONE, None) == TOO_LARGE


def test_step_strides_a_call_takes(L):
    """Long strides are refused only where a kernel's offsets end.  (What is taken is
    seen by the next refusal, the workspace's: nothing runs.)"""
    far = lambda stride: CkSeq(FAKE, stride, 64)
    grads = lambda q: ctypes.byref(ScanGrads(q, q, SEQ, SEQ, q, FAKE, None, None, None))

    def scan(q, bc, **kw):
        return L.ck_scan_backward(_scan(**kw), _inputs(u=q, delta=q, b=bc, c=bc, z=q), FAKE, q,
                                  None, grads(q), FAKE, 0, None)

    many, cut = dict(T=40, B=400), dict(T=200, B=2)   # a workgroup each; chunks
    for kw in (many, cut):
        for dtype, last in ((0, 2**26), (1, 2**27), (2, 2**27)):
            assert scan(far(last), far(last), dtype=dtype, **kw) == WORKSPACE
            assert scan(far(8 * last), SEQ, dtype=dtype, **kw) == BAD_VALUE
            assert scan(SEQ, far(8 * last), dtype=dtype, **kw) == BAD_VALUE
    assert scan(far(2**24 - 1), far(2**24 - 1)) == WORKSPACE      # several tiles a workgroup
    assert scan(far(2**24), SEQ) == BAD_VALUE and scan(SEQ, far(2**24)) == BAD_VALUE
    # the gradients of B and C are written row by row
    g = ctypes.byref(ScanGrads(SEQ, SEQ, far(2**40), far(2**40), NONE, FAKE, None, None, None))
    assert L.ck_scan_backward(_scan(), _inputs(), FAKE, SEQ, None, g, FAKE, 0, None) == WORKSPACE

    def conv(q):
        return L.ck_conv_backward(_conv(), q, FAKE, None, None, None, q, None, q, FAKE, None, None,
                                  FAKE, 0, None)

    assert conv(far(2**24)) == WORKSPACE and conv(far(2**30 - 1)) == WORKSPACE
    assert conv(far(2**30)) == BAD_VALUE


@pytest.mark.parametrize("st,sb", [(0, 64), (64, 0), (63, 64), (128, 63)])
def test_outputs_over_one_another_are_refused(L, st, sb):
    """An output that is the same memory at several steps or rows (a broadcast
    tensor) has no one value; inputs may be broadcast."""
    q = CkSeq(FAKE, st, sb)
    s, one, i = _scan(), _scan(T=1), _inputs()
    assert L.ck_scan_forward(s, i, q, None, None, FAKE, 2**40, None) == BAD_VALUE
    for k in range(5):
        v = [SEQ] * 5
        v[k] = q if k not in (2, 3) else CkSeq(FAKE, st // 4, sb // 4)  # 16 values a row
        g = ctypes.byref(ScanGrads(*v, FAKE, None, None, None))
        assert L.ck_scan_backward(s, _inputs(z=q), FAKE, q, None, g, FAKE, 0, None) == BAD_VALUE
    g = ctypes.byref(ScanGrads(*[SEQ] * 5, FAKE, None, None, None))
    assert L.ck_scan_backward(s, _inputs(u=q, b=q, z=q), FAKE, q, None, g, FAKE, 0,
                              None) == WORKSPACE
    assert L.ck_conv_forward(_conv(), SEQ, FAKE, None, None, None, q, None, None) == BAD_VALUE
    back = lambda gy, gx: L.ck_conv_backward(_conv(), q, FAKE, None, None, None, gy, None, gx,
                                             FAKE, None, None, FAKE, 0, None)
    assert back(q, q) == BAD_VALUE and back(q, SEQ) == WORKSPACE
    d = ctypes.byref(DropoutShape(8, 2, 64, 1, 0, 0.5, 1, 0, None))
    assert L.ck_dropout_forward(d, SEQ, NONE, q, None) == BAD_VALUE
    assert L.ck_dropout_backward(d, SEQ, q, None) == BAD_VALUE
    if sb < 64:  # a step has no stride between steps
        assert L.ck_scan_step(one, i, q, FAKE, None) == BAD_VALUE
        assert L.ck_conv_step(_conv(T=1), SEQ, FAKE, None, None, q, FAKE, None) == BAD_VALUE


def test_scan_call_refusals(L):
    g = ctypes.byref(ScanGrads(SEQ, SEQ, SEQ, SEQ, NONE, FAKE, None, None, None))
    s, i = _scan(), _inputs()
    assert L.ck_scan_sizes(None, None, None, None) == NULL_ARG
    assert L.ck_scan_forward(s, None, SEQ, None, None, None, 0, None) == NULL_ARG
    assert L.ck_scan_forward(s, i, NONE, None, None, FAKE, 2**40, None) == NULL_ARG
    assert L.ck_scan_forward(s, i, SEQ, None, FAKE + 16, FAKE, 2**40, None) == BAD_VALUE
    assert L.ck_scan_backward(s, i, None, SEQ, None, g, FAKE, 2**40, None) == NULL_ARG
    assert L.ck_scan_backward(s, i, FAKE, SEQ, None, None, FAKE, 2**40, None) == NULL_ARG
    assert L.ck_scan_backward(s, i, FAKE, NONE, None, g, FAKE, 2**40, None) == NULL_ARG
    assert L.ck_scan_backward(s, i, FAKE, SEQ, None, g, None, 0, None) == NULL_ARG
    assert L.ck_scan_backward(s, i, FAKE, SEQ, None, g, FAKE, 16, None) == WORKSPACE
    assert L.ck_scan_backward(s, i, FAKE, SEQ, None, g, FAKE + 16, 2**40, None) == BAD_VALUE
    # a gate's gradient is required when there is a gate
    assert L.ck_scan_backward(s, _inputs(z=SEQ), FAKE, SEQ, None, g, FAKE, 2**40, None) == NULL_ARG
    assert L.ck_scan_step(s, i, SEQ, FAKE, None) == BAD_SIZE
    assert L.ck_scan_step(_scan(T=1), i, SEQ, None, None) == NULL_ARG
    assert L.ck_scan_step(_scan(T=1), _inputs(lengths=FAKE), SEQ, FAKE, None) == BAD_VALUE


def _conv(**kw):
    return ctypes.byref(ConvShape(*[kw.get(k, v) for k, v in dict(
        T=8, B=2, D=64, W=4, dtype=1, silu=1).items()]))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD_SIZE), (dict(B=0), BAD_SIZE), (dict(D=-2), BAD_SIZE), (dict(W=0), BAD_SIZE),
    (dict(W=9), BAD_SIZE), (dict(T=2**31), TOO_LARGE), (dict(T=2**30, B=2**20), TOO_LARGE),
    (dict(dtype=7), BAD_VALUE)])
def test_conv_shape_refusals(L, kw, status):
    s = ctypes.c_size_t()
    assert L.ck_conv_sizes(_conv(**kw), ctypes.byref(s)) == status
    assert L.ck_conv_forward(_conv(**kw), SEQ, FAKE, None, None, None, SEQ, None, None) == status
    if "T" not in kw:
        assert L.ck_conv_step(_conv(**{"T": 1, **kw}), SEQ, FAKE, None, None, SEQ, FAKE,
                              None) == status


def test_conv_call_refusals(L):
    s, one = _conv(), _conv(T=1)
    assert L.ck_conv_sizes(None, None) == NULL_ARG
    assert L.ck_conv_forward(s, SEQ, None, None, None, None, SEQ, None, None) == NULL_ARG
    assert L.ck_conv_forward(s, NONE, FAKE, None, None, None, SEQ, None, None) == NULL_ARG
    assert L.ck_conv_forward(s, SEQ, FAKE, None, None, None, NONE, None, None) == NULL_ARG
    assert L.ck_conv_forward(s, SEQ, FAKE, None, FAKE + 1, None, SEQ, None, None) == BAD_VALUE
    back = lambda gy, gx, gw, ws, n: L.ck_conv_backward(s, SEQ, FAKE, None, None, None, gy, None,
                                                        gx, gw, None, None, ws, n, None)
    assert back(NONE, SEQ, FAKE, FAKE, 2**40) == NULL_ARG
    assert back(SEQ, NONE, FAKE, FAKE, 2**40) == NULL_ARG
    assert back(SEQ, SEQ, None, FAKE, 2**40) == NULL_ARG
    assert back(SEQ, SEQ, FAKE, None, 0) == NULL_ARG
    assert back(SEQ, SEQ, FAKE, FAKE, 16) == WORKSPACE
    assert back(SEQ, SEQ, FAKE, FAKE + 64, 2**40) == BAD_VALUE
    assert L.ck_conv_step(s, SEQ, FAKE, None, None, SEQ, FAKE, None) == BAD_SIZE
    assert L.ck_conv_step(one, SEQ, FAKE, None, None, SEQ, None, None) == NULL_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD_SIZE), (dict(B=0), BAD_SIZE), (dict(p=-0.1), BAD_VALUE),
    (dict(p=1.5), BAD_VALUE), (dict(p=float("nan")), BAD_VALUE), (dict(dtype=5), BAD_VALUE),
    (dict(T=2**20, B=2**12), TOO_LARGE)])
def test_dropout_refusals(L, kw, status):
    s = ctypes.byref(DropoutShape(*[kw.get(k, v) for k, v in dict(
        T=8, B=2, D=64, dtype=1, held=0, p=0.5, seed=1, offset=0, counter=None).items()]))
    assert L.ck_dropout_forward(s, SEQ, NONE, SEQ, None) == status
    assert L.ck_dropout_backward(s, SEQ, SEQ, None) == status


def test_dropout_call_refusals(L):
    s = ctypes.byref(DropoutShape(8, 2, 64, 1, 0, 0.5, 1, 0, None))
    assert L.ck_dropout_forward(None, SEQ, NONE, SEQ, None) == NULL_ARG
    assert L.ck_dropout_forward(s, NONE, NONE, SEQ, None) == NULL_ARG
    assert L.ck_dropout_forward(s, SEQ, NONE, NONE, None) == NULL_ARG
    assert L.ck_dropout_forward(s, SEQ, CkSeq(FAKE + 1, 0, 0), SEQ, None) == BAD_VALUE
    assert L.ck_dropout_backward(s, SEQ, CkSeq(FAKE, 0, -8), None) == BAD_VALUE


@pytest.mark.parametrize("mode", ["grad", "no_grad", "inference", "no leaf"])
def test_scan_saves_states_for_a_backward_alone(monkeypatch, mode):
    """Without a backward to come (grad mode off, or nothing that requires a
    gradient) the node does not have the forward leave its states."""
    import torch

    from sparse_graph_recurrent_amd import sequence
    asked = []

    def forward(u, delta, A, B, C, *args, save=True, **kw):
        asked.append(save)
        return torch.zeros_like(u), u.new_zeros(u.shape[1:] + A.shape[1:]), None, None

    monkeypatch.setattr(sequence, "selective_scan_forward", forward)
    A = torch.ones(4, 2, requires_grad=mode != "no leaf")
    x, b = torch.ones(3, 1, 4), torch.ones(3, 1, 1, 2)
    with {"no_grad": torch.no_grad, "inference": torch.inference_mode}.get(
            mode, torch.enable_grad)():
        out, _ = sgr.selective_scan(x, x, A, b, b)
    assert asked == [mode == "grad"]
    assert out.requires_grad == (mode == "grad")
