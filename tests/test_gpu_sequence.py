"""The sequence operators (short convolution, selective scan, dropout) against
their fp64 definitions, at the sizes, lengths, strides and types where such
kernels go wrong.

Tolerances.  Every output is held to

    |got - want| <= (eps / 2) (|want| + err) + err,   err = k 2^-24 m

where eps / 2 is the one rounding to the output's type, m the sum of the
magnitudes of the output's terms (``sequence_ref``, magnitude=True) and k the
count of fp32 roundings on a term's way: about 8 a step through the
recurrence's products and hardware functions (the decay's error, relative
8 |dt A|, is largest where dt A exp(dt A) is, at 3 / 8 of that), once more in
the gradients, whose terms hold a state and an adjoint, and the additions
across channels, rows and steps.
"""
import ctypes

import numpy as np
import pytest
import torch

import sequence_ref as ref
import sparse_graph_recurrent_amd as sgr
from gpu_helpers import log
from sparse_graph_recurrent_amd import sequence

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def close(got, want, mag, k, name):
    got_t = got.detach()
    fi = torch.finfo(got_t.dtype)
    g = got_t.double().cpu().numpy()
    assert g.shape == want.shape, name
    err = k * ref.U32 * mag
    tol = fi.eps / 2 * (np.abs(want) + err) + err + fi.smallest_normal * fi.eps
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                           f"{np.nanmax(np.abs(g - want) / tol):.3g} times it, "
                           f"{np.isnan(g).sum()} NaN, first at {np.argwhere(bad)[0]}")


def place(a, dtype, layout, pad_nan=None):
    """The fp64 array [T, B, ...] on the device: "time" contiguous, "batch"
    batch outermost, "slice" a slice of a wider tensor (odd offset, odd row
    stride).  Returns (tensor, its exact values in fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype)
    val = t.double().numpy()
    if pad_nan is not None:
        t[torch.from_numpy(~pad_nan)] = float("nan")
    T, B = t.shape[:2]
    inner = t.shape[2:]
    n = int(np.prod(inner))
    if layout == "batch":
        s = torch.empty((B, T) + tuple(inner), dtype=dtype, device="cuda").transpose(0, 1)
    elif layout == "slice":
        s = torch.full((T, B, n + 5), 7.0, dtype=dtype, device="cuda")[:, :, 3:3 + n]
        s = s.unflatten(2, tuple(inner)) if n else s.reshape((T, B) + tuple(inner))
    else:
        s = torch.empty(t.shape, dtype=dtype, device="cuda")
    s.copy_(t)
    return s, val


def _f32(a):
    t = torch.from_numpy(np.ascontiguousarray(a)).float()
    return t.cuda(), t.double().numpy()


def scan_problem(seed, T, B, D, N, G, dtype, gate, softplus, lengths, layout, state0=True,
                 extras=True, nan=True):
    """(GPU arguments, fp64 problem) with the same values."""
    r = np.random.default_rng(seed)
    ok = ref.valid(T, B, None if lengths is None else np.array(lengths))
    pad = ok if nan and lengths is not None else None
    raw = {"u": r.standard_normal((T, B, D)),
           "delta": (r.standard_normal((T, B, D)) - 2 if softplus else
                     r.uniform(0.0, 0.5, (T, B, D))),
           "B": r.standard_normal((T, B, G, N)), "C": r.standard_normal((T, B, G, N)),
           "go": r.standard_normal((T, B, D))}
    if gate:
        raw["z"] = 2 * r.standard_normal((T, B, D))
    gpu, p = {}, {"softplus": softplus, "lengths": None if lengths is None else np.array(lengths)}
    for k, a in raw.items():
        gpu[k], p[k] = place(a, DT[dtype], layout, pad)
    par = {"A": -np.exp(r.uniform(np.log(0.05), np.log(16), (D, N))),
           "gstate": r.standard_normal((B, D, N))}
    if extras:
        par.update(D=r.standard_normal(D),
                   delta_bias=0.2 * (r.standard_normal(D) if softplus else r.random(D)))
    if state0:
        par["state0"] = r.standard_normal((B, D, N))
    for k, a in par.items():
        gpu[k], p[k] = _f32(a)
    gpu["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                               device="cuda")
    return gpu, p


def scan_run(g, softplus, stream=None, **kw):
    args = (g["u"], g["delta"], g["A"], g["B"], g["C"])
    opt = dict(D=g.get("D"), z=g.get("z"), delta_bias=g.get("delta_bias"), lengths=g["lengths"],
               delta_softplus=softplus, stream=stream)
    out, state, saved, _ = sgr.selective_scan_forward(*args, state0=g.get("state0"), **opt, **kw)
    grads = sgr.selective_scan_backward(*args, saved, g["go"], grad_state=g["gstate"], **opt)
    return out, state, grads


def scan_check(g, p, softplus, got=None):
    T, B, D = g["u"].shape
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    out, state, grads = got or scan_run(g, softplus)
    torch.cuda.synchronize()
    k = 32 + 8 * T
    close(out, want["out"], mag["out"], k, "out")
    close(state, want["state"], mag["state"], k, "state")
    k = 64 + 16 * T + B + 64
    for name, t in grads.items():
        if name in ("g_D", "g_delta_bias") and name not in want:
            continue
        close(t, want[name], mag[name], k, name)


SCAN = [  # T, B, D, N, G, dtype, gate, softplus, lengths, layout
    (1, 1, 1, 1, 1, "fp32", False, False, None, "time"),
    (16, 2, 64, 16, 1, "fp32", True, True, None, "time"),
    (15, 2, 63, 16, 1, "bf16", True, True, None, "slice"),
    (17, 3, 65, 13, 5, "fp16", True, True, None, "batch"),
    (33, 2, 130, 4, 2, "fp32", False, True, None, "batch"),
    (40, 1, 96, 8, 3, "bf16", True, False, None, "time"),
    (100, 2, 70, 16, 7, "fp32", True, True, None, "slice"),
    (19, 2, 64, 17, 1, "fp32", True, True, None, "time"),
    (21, 2, 48, 32, 2, "fp16", False, True, None, "time"),
    (11, 2, 33, 33, 1, "fp32", True, True, None, "batch"),
    (13, 2, 32, 64, 1, "bf16", True, True, None, "time"),
    (50, 6, 66, 16, 2, "fp32", True, True, [0, 50, 1, 16, 17, 33], "time"),
    (50, 5, 40, 3, 1, "bf16", True, True, [49, 0, 32, 2, 48], "batch"),
    (9, 4, 20, 40, 4, "fp32", False, True, [0, 9, 4, 5], "slice"),
    (20, 4, 24, 16, 1, "fp16", True, True, [-3, 25, 20, 7], "time"),
    (200, 1, 128, 16, 1, "fp32", True, True, None, "time"),
    (1500, 1, 16, 16, 1, "fp32", True, True, None, "time"),
    (700, 3, 40, 16, 2, "fp32", True, True, [700, 333, 0], "batch"),
    # enough rows for a workgroup each without cutting the window, and for
    # several tiles a workgroup over a long one
    (20, 400, 64, 16, 1, "bf16", True, True, None, "time"),
    (25, 390, 40, 16, 1, "fp32", False, True, [(7 * b) % 26 for b in range(390)], "time"),
    (131, 210, 64, 12, 1, "fp32", True, True, None, "time"),
    (10, 390, 48, 24, 1, "fp32", True, True, None, "time"),
    # cut windows with more than 16 states, and with groups that end in a workgroup
    (200, 1, 40, 33, 1, "fp32", True, True, None, "time"),
    (150, 2, 66, 20, 3, "bf16", False, True, [150, 77], "batch"),
]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan(case):
    log(f"scan {case}")
    g, p = scan_problem(1, *case)
    scan_check(g, p, case[7])


# Windows cut where neither all workgroups run at once nor few chunks are read, so
# that a launch joins the chunks; and short windows of few rows, cut finely.
JOINED = [
    (520, 130, 16, 16, 1, "fp32", True, True, None, "time"),
    (521, 131, 20, 5, 1, "bf16", True, True, [(37 * b) % 522 for b in range(131)], "batch"),
    (515, 130, 6, 20, 2, "fp32", False, True, None, "time"),
    (514, 130, 3, 33, 1, "fp16", False, True, [514 - 3 * b for b in range(130)], "time"),
    (97, 2, 40, 16, 1, "fp32", True, True, [97, 40], "time"),
    (129, 3, 64, 16, 1, "bf16", False, True, None, "slice"),
]


# Up to 8 states, which have a layout of their own: uncut, several tiles a
# workgroup over long and short windows, and cut.
NARROW = [
    (20, 400, 64, 7, 1, "bf16", True, True, None, "time"),
    (131, 210, 64, 6, 1, "fp32", True, True, None, "time"),
    (70, 3, 96, 8, 2, "fp16", True, True, [70, 0, 33], "batch"),
    (333, 2, 70, 8, 1, "fp32", True, False, None, "slice"),
    (333, 3, 40, 2, 2, "bf16", False, True, [333, 100, 1], "time"),
]


@pytest.mark.parametrize("case", NARROW, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_few_states(case):
    log(f"scan few states {case[:8]}")
    g, p = scan_problem(13, *case)
    scan_check(g, p, case[7])


@pytest.mark.parametrize("case", JOINED, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_chunks(case):
    log(f"scan chunks {case[:8]}")
    g, p = scan_problem(12, *case)
    scan_check(g, p, case[7])


# around the length from which few rows are cut
@pytest.mark.parametrize("T", [63, 64, 65, 66, 95])
@pytest.mark.parametrize("rest", [(2, 70, 16, 1, "bf16", True, True, [64, 40], "slice"),
                                  (3, 40, 6, 2, "fp32", False, True, None, "time"),
                                  (2, 24, 20, 1, "fp16", True, True, None, "batch")],
                         ids=lambda c: "-".join(map(str, c[:5])))
def test_scan_short_windows(T, rest):
    case = (T,) + rest
    log(f"scan short {case[:6]}")
    g, p = scan_problem(16, *case)
    scan_check(g, p, case[7])


def test_scan_without_optional_inputs():
    g, p = scan_problem(2, 20, 2, 64, 16, 1, "fp32", False, True, None, "time", state0=False,
                        extras=False)
    out, state, grads = scan_run(g, True)
    scan_check(g, p, True, (out, state, grads))


def test_scan_empty_window_passes_the_state():
    g, p = scan_problem(3, 0, 2, 33, 5, 1, "fp32", True, True, None, "time")
    out, state, saved, _ = sgr.selective_scan_forward(
        g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["delta_bias"], g["state0"],
        delta_softplus=True)
    gr = sgr.selective_scan_backward(g["u"], g["delta"], g["A"], g["B"], g["C"], saved, g["go"],
                                     g["D"], g["z"], g["delta_bias"], delta_softplus=True,
                                     grad_state=g["gstate"])
    torch.cuda.synchronize()
    assert out.shape == (0, 2, 33)
    assert torch.equal(state, g["state0"]) and torch.equal(gr["g_state0"], g["gstate"])
    for k in ("g_A", "g_D", "g_delta_bias"):
        assert not gr[k].any(), k


def test_scan_broadcast_inputs_and_windows():
    """u the same at every row and step (strides 0); a window cut in two gives
    the whole window's outputs through the carried state."""
    g, p = scan_problem(4, 37, 3, 64, 16, 1, "fp32", True, True, None, "time")
    g["u"] = g["u"][:1, :1].expand(37, 3, 64)
    p["u"] = np.broadcast_to(p["u"][:1, :1], p["u"].shape)
    out, state, grads = scan_run(g, True)
    scan_check(g, p, True, (out, state, grads))
    part = lambda a, b, s: sgr.selective_scan_forward(
        *(g[k][a:b] if k != "A" else g[k] for k in ("u", "delta", "A", "B", "C")), D=g["D"],
        z=g["z"][a:b], delta_bias=g["delta_bias"], state0=s, delta_softplus=True, save=False)
    o1, s1, saved, _ = part(0, 20, g["state0"])
    o2, s2, _, _ = part(20, 37, s1)
    assert saved is None
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    close(torch.cat([o1, o2]), want["out"], mag["out"], 32 + 8 * 37, "out")
    close(s2, want["state"], mag["state"], 32 + 8 * 37, "state")


def test_scan_extremes():
    """Large and infinite inputs: softplus and the gate saturate as the
    definition does, and an infinite step forgets the state."""
    T, D, N = 4, 8, 16
    g, p = scan_problem(5, T, 1, D, N, 1, "fp32", True, True, None, "time")
    for i, v in enumerate((-200.0, -30.0, 30.0, 300.0)):
        g["delta"][:, :, i] = v
        p["delta"][:, :, i] = v
        g["z"][:, :, 4 + i] = v
        p["z"][:, :, 4 + i] = v
    scan_check(g, p, True)
    g["delta"][2, 0, 0] = float("inf")
    out, state, _, _ = sgr.selective_scan_forward(
        g["u"], g["delta"], g["A"], g["B"], g["C"], state0=g["state0"], delta_softplus=True)
    assert not torch.isfinite(out[2, 0, 0])          # inf * u * B
    assert torch.isfinite(out[:, 0, 1:]).all()       # other channels do not see it
    assert torch.isfinite(out[:2, 0, 0]).all()       # nor do earlier steps


# windows that end inside a tile, on each of the ways over the chip: several tiles a
# workgroup, uncut, cut and folded, cut and joined; every number of padded states
FORGETS = [
    (13, 2, 40, 16, 1, "fp32", True, True, [13, 6], "time"),
    (77, 210, 16, 5, 1, "fp32", False, True, None, "time"),
    (21, 390, 20, 16, 1, "bf16", True, True, [(5 * b) % 22 for b in range(390)], "time"),
    (203, 2, 70, 16, 2, "fp32", True, True, [203, 58], "batch"),
    (203, 1, 40, 33, 1, "fp32", False, True, None, "time"),
    (517, 130, 6, 7, 2, "fp32", True, True, [(29 * b) % 518 for b in range(130)], "time"),
    (515, 130, 6, 20, 2, "fp16", True, True, None, "time"),
]


@pytest.mark.parametrize("case", FORGETS, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_state_that_forgets_everything(case):
    """A = -inf, as -exp(log_a) overflows to: each step's decay is 0, and the steps
    past a row's end still change nothing.  The definition's own limit is taken at
    -1e30, where exp(dt A) is 0 as well."""
    log(f"scan forgets {case[:6]}")
    g, p = scan_problem(22, *case)
    g["A"][::3, ::2] = g["A"][1, -1] = float("-inf")
    p["A"][::3, ::2] = p["A"][1, -1] = -1e30
    scan_check(g, p, case[7])


def test_scan_step_of_a_state_that_forgets_everything():
    g, p = scan_problem(23, 1, 3, 20, 5, 1, "fp32", True, True, None, "time")
    g["A"][::3], p["A"][::3] = float("-inf"), -1e30
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    o, s = sgr.selective_scan_step(g["state0"], g["u"][0], g["delta"][0], g["A"], g["B"][0],
                                   g["C"][0], g["D"], g["z"][0], g["delta_bias"], True)
    close(o[None], want["out"], mag["out"], 40, "out")
    close(s, want["state"], mag["state"], 40, "state")


def growing(seed, case, rate, zero):
    """A problem whose states grow by exp(|dt A|) a step, |dt A| up to `rate`, A
    positive or dt negative.  zero: u is 0 before the last two steps and the outputs'
    gradient behind the first two, so that states and adjoints are 0 in between;
    else everything starts at 1e-15 and stays in range over the rows' lengths."""
    T, B, D, N, G, _, gate, positive, lengths, layout = case
    g, p = scan_problem(seed, T, B, D, N, G, "fp32", gate, False, lengths, layout,
                        extras=False, nan=False)
    r = np.random.default_rng(seed + 1)
    sign = 1.0 if positive else -1.0
    g["A"], p["A"] = _f32(sign * rate * r.uniform(0.9, 1.0, (D, N)))
    g["delta"], p["delta"] = place(sign * r.uniform(0.95, 1.0, (T, B, D)), torch.float32, layout)
    for k in ("u", "go", "state0", "gstate"):
        a = p[k].copy() if zero else 1e-15 * p[k]
        if zero:
            a[{"u": slice(0, T - 2), "go": slice(2, T)}.get(k, slice(None))] = 0.0
        g[k], p[k] = place(a, torch.float32, layout) if a.ndim == 3 and k in ("u", "go") else _f32(a)
    return g, p


GROWS = [  # T, B, D, N, G, dtype, gate, A positive (else dt negative), lengths, layout
    (40, 2, 40, 16, 1, "fp32", False, True, None, "time"),
    (40, 2, 40, 16, 1, "fp32", True, False, None, "time"),
    (77, 210, 16, 5, 1, "fp32", False, True, None, "time"),
    (131, 210, 16, 12, 1, "fp32", False, False, None, "time"),
    (203, 2, 70, 16, 2, "fp32", True, True, None, "batch"),
    (203, 1, 40, 33, 1, "fp32", False, False, None, "time"),
    (517, 130, 6, 7, 2, "fp32", False, True, None, "time"),
    (515, 130, 6, 20, 2, "fp32", False, False, None, "time"),
]


def growing_check(g, p, rate):
    # A step's decay is off by 4 |dt A| roundings for its exponent and 4 more; the
    # other 8 (16 in the gradients) a step are scan_check's.
    T, B, _ = g["u"].shape
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    out, state, grads = scan_run(g, False)
    torch.cuda.synchronize()
    k = 32 + (12 + 4 * rate) * T
    close(out, want["out"], mag["out"], k, "out")
    close(state, want["state"], mag["state"], k, "state")
    for name, t in grads.items():
        if name in want:
            close(t, want[name], mag[name], 2 * k + B + 64, name)


@pytest.mark.parametrize("case", GROWS, ids=lambda c: "-".join(map(str, c[:5])))
def test_scan_keeps_zero_states_where_decays_overflow(case):
    """Over a tile or chunk the decay is far beyond fp32, each step's is not: a
    zero state (adjoint) stays zero."""
    log(f"scan grows {case[:5]}")
    g, p = growing(24, case, 16.0, True)
    growing_check(g, p, 16.0)


@pytest.mark.parametrize("case,rate", [
    ((9, 2, 40, 16, 1, "fp32", False, True, None, "time"), 12.0),
    ((9, 3, 70, 6, 1, "fp32", True, False, None, "time"), 12.0),
    ((203, 2, 70, 16, 2, "fp32", False, True, [26, 25], "time"), 4.2),
    ((517, 130, 6, 20, 2, "fp32", False, False, [64 + b % 24 for b in range(130)], "time"), 1.3),
], ids=lambda c: "-".join(map(str, c[:5])) if isinstance(c, tuple) else str(c))
def test_scan_small_states_grow_past_a_decay_beyond_range(case, rate):
    """A tile's or chunk's decay overflows fp32, the states it is applied to do not."""
    log(f"scan grows {case[:5]}")
    g, p = growing(26, case, rate, False)
    growing_check(g, p, rate)


def test_scan_values_of_one_step_stay_in_it():
    """An infinite or undefined B, C or u reaches no earlier step and no other row."""
    for k in ("B", "C", "u"):
        g, _ = scan_problem(15, 12, 2, 20, 16, 1, "fp32", True, True, None, "time")
        clean, _, _, _ = sgr.selective_scan_forward(
            g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["delta_bias"],
            g["state0"], delta_softplus=True)
        g[k][6, 0] = float("nan")
        out, state, _, _ = sgr.selective_scan_forward(
            g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["delta_bias"],
            g["state0"], delta_softplus=True)
        assert torch.equal(out[:6], clean[:6]) and torch.equal(out[:, 1], clean[:, 1]), k
        assert torch.isnan(out[6, 0]).all(), k
        # C enters no state: the steps behind are clean again
        assert torch.equal(out[7:, 0], clean[7:, 0]) == (k == "C"), k


def test_scan_same_bits_every_time_and_on_another_stream():
    g, p = scan_problem(6, 70, 2, 130, 16, 1, "bf16", True, True, [70, 41], "time")
    a = scan_run(g, True)
    b = scan_run(g, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = scan_run(g, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for o in (b, c):
        assert torch.equal(a[0], o[0]) and torch.equal(a[1], o[1])
        for k in a[2]:
            assert torch.equal(a[2][k], o[2][k]), k


@pytest.mark.parametrize("dtype,B,D,N,G", [("fp32", 1, 1, 1, 1), ("bf16", 3, 70, 16, 7),
                                           ("fp16", 5, 64, 13, 1), ("bf16", 2, 130, 33, 2),
                                           ("fp32", 4, 66, 64, 2), ("fp32", 2, 36, 6, 3)])
def test_scan_step_walks_the_window(dtype, B, D, N, G):
    """Single tokens, state in place, against the definition of the window."""
    T = 6
    g, p = scan_problem(7, T, B, D, N, G, dtype, True, True, None, "slice")
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    state = g["state0"].clone()
    outs = []
    for t in range(T):
        o, s = sgr.selective_scan_step(state, g["u"][t], g["delta"][t], g["A"], g["B"][t],
                                       g["C"][t], g["D"], g["z"][t], g["delta_bias"], True)
        assert s is state
        outs.append(o)
    close(torch.stack(outs), want["out"], mag["out"], 32 + 8 * T, "out")
    close(state, want["state"], mag["state"], 32 + 8 * T, "state")
    keep = g["state0"].clone()
    o, s = sgr.selective_scan_step(g["state0"], g["u"][0], g["delta"][0], g["A"], g["B"][0],
                                   g["C"][0], g["D"], g["z"][0], g["delta_bias"], True,
                                   new_state=torch.empty_like(keep))
    assert torch.equal(o, outs[0]) and torch.equal(g["state0"], keep)


def test_scan_autograd_with_shared_inputs():
    """Gradients through the autograd node where one tensor feeds several
    inputs and B, C come from a broadcast, against fp64 autograd of the
    definition written step by step."""
    T, B, D, N = 12, 2, 24, 4
    r = np.random.default_rng(8)
    x0 = torch.from_numpy(r.standard_normal((T, B, D))).float()
    bc0 = torch.from_numpy(r.standard_normal((T, 1, 1, N))).float()
    a0 = torch.from_numpy(-r.uniform(0.1, 2, (D, N))).float()

    def loss_of(x, bc, a, fn):
        out, state = fn(x, 0.3 * x - 1, a, bc.expand(T, B, 1, N), bc.expand(T, B, 1, N), x)
        return (out * out).sum() + state.sum()

    def define(u, d, a, Bm, Cm, z):
        h, outs = torch.zeros(B, D, N, dtype=u.dtype), []
        for t in range(T):
            dt = torch.nn.functional.softplus(d[t]).unsqueeze(-1)
            h = torch.exp(dt * a) * h + dt * u[t].unsqueeze(-1) * Bm[t]
            outs.append((h * Cm[t]).sum(-1) * z[t] * torch.sigmoid(z[t]))
        return torch.stack(outs), h

    lw = [t.double().requires_grad_() for t in (x0, bc0, a0)]
    loss_of(*lw, define).backward()
    lg = [t.cuda().requires_grad_() for t in (x0, bc0, a0)]
    loss_of(*lg, lambda u, d, a, Bm, Cm, z: sgr.selective_scan(
        u, d, a, Bm, Cm, z=z, delta_softplus=True)).backward()
    for w, g, name in zip(lw, lg, ("x", "bc", "a")):
        # rounding of sums of some hundred terms: 1e-5 of the largest gradient
        scale = w.grad.abs().max().item()
        assert (g.grad.double().cpu() - w.grad).abs().max().item() <= 1e-5 * scale, name


# several tiles a workgroup, a workgroup each, cut; rows and states that fill nothing
GIVEN = [
    (21, 3, 70, 13, 7, "bf16", True, True, [21, 0, 10], "time"),
    (13, 390, 9, 5, 1, "fp32", False, True, None, "batch"),
    (140, 2, 66, 20, 3, "fp16", True, True, [140, 77], "time"),
]


def given(like, fill=7.0):
    """(a tensor of like's shape inside a wider storage of another order, batch
    outermost and one element past an aligned address; that storage)"""
    T, B = like.shape[:2]
    n = like[0, 0].numel()
    store = torch.full((B, T + 1, n + 3), fill, dtype=like.dtype, device="cuda")
    return store[:, :T, 1:1 + n].transpose(0, 1).unflatten(2, like.shape[2:]), store


def untouched(store, n, fill=7.0):
    return bool((store[:, -1] == fill).all() and (store[..., 0] == fill).all() and
                (store[..., 1 + n:] == fill).all())


@pytest.mark.parametrize("case", GIVEN, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_into_given_tensors(case):
    """The caller's outputs, gradients (strided), saved states and workspaces get the
    bits that tensors made by the calls get, and nothing beside them is written."""
    g, p = scan_problem(31, *case)
    softplus = case[7]
    args = (g["u"], g["delta"], g["A"], g["B"], g["C"])
    opt = dict(D=g["D"], z=g.get("z"), delta_bias=g["delta_bias"], lengths=g["lengths"],
               delta_softplus=softplus)
    scan_check(g, p, softplus)
    want = sgr.selective_scan_forward(*args, state0=g["state0"], **opt)
    wg = sgr.selective_scan_backward(*args, want[2], g["go"], grad_state=g["gstate"], **opt)
    sb, fb, bb = sgr.selective_scan_sizes(*g["u"].shape, case[3], case[4], g["u"].dtype)
    out, so = given(g["u"])
    state = torch.full_like(g["state0"], 7.0)
    buf = lambda n: torch.full((max(n, 1) + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    saved, fw, bw = buf(sb), buf(fb), buf(bb)
    r = sgr.selective_scan_forward(*args, state0=g["state0"], out=out, state=state, saved=saved,
                                   workspace=fw, **opt)
    assert r[0] is out and r[1] is state and r[2] is saved and r[3] is fw
    assert torch.equal(out, want[0]) and torch.equal(state, want[1])
    assert untouched(so, case[2])
    for b, n in ((saved, sb), (fw, fb)):
        assert bool((b[n:] == 0x5A).all())
    grads, stores = {}, {}
    for k, t in wg.items():
        if k in ("g_u", "g_delta", "g_B", "g_C", "g_z"):
            grads[k], stores[k] = given(t)
        else:
            grads[k] = torch.full_like(t, 7.0)
    assert sgr.selective_scan_backward(*args, saved, g["go"], grad_state=g["gstate"], grads=grads,
                                       workspace=bw, **opt) is grads
    for k, t in wg.items():
        assert torch.equal(grads[k], t), k
    for k, s in stores.items():
        assert untouched(s, wg[k][0, 0].numel()), k
    assert bool((bw[bb:] == 0x5A).all())
    # gradients that are not wanted
    some = {k: v for k, v in grads.items() if k not in ("g_D", "g_delta_bias", "g_state0")}
    sgr.selective_scan_backward(*args, saved, g["go"], grad_state=g["gstate"], grads=some, **opt)
    assert all(torch.equal(some[k], wg[k]) for k in some)
    for kw in (dict(saved=saved[:sb - 1]), dict(workspace=fw[:fb - 1] if fb else fw[::2]),
               dict(out=out[:-1]), dict(state=state[:, :, :-1]),
               dict(out=g["u"].new_empty(1, *g["u"].shape[1:]).expand_as(g["u"]))):
        with pytest.raises((ValueError, sgr.CkError)):
            sgr.selective_scan_forward(*args, state0=g["state0"], **kw, **opt)
    for kw in (dict(workspace=bw[:bb - 1]), dict(grads=dict(grads, g_A=g["A"][:, :-1])),
               dict(grads=dict(grads, g_B=grads["g_B"][:-1])), dict(saved=saved[:sb - 1])):
        s = kw.pop("saved", saved)
        with pytest.raises(ValueError):
            sgr.selective_scan_backward(*args, s, g["go"], **kw, **opt)


@pytest.mark.parametrize("case", GIVEN, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_autograd_reaches_every_input(case):
    """The node's gradients of all inputs, with lengths, against the definition's;
    parameters in another order of storage."""
    T, B, D, N, G, dtype, gate, softplus, lengths, _ = case
    g, p = scan_problem(32, *case, nan=False)
    leaf = lambda t: t.detach().clone().requires_grad_()
    turned = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2).detach().requires_grad_()
    names = ["u", "delta", "A", "B", "C", "D", "delta_bias", "state0"] + (["z"] if gate else [])
    t = {k: (turned if k in ("A", "state0", "B") else leaf)(g[k]) for k in names}
    out, state = sgr.selective_scan(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"], t.get("z"),
                                    t["delta_bias"], t["state0"], g["lengths"], softplus)
    got = torch.autograd.grad((out, state), [t[k] for k in names], (g["go"], g["gstate"]))
    want, mag = ref.scan(p), ref.scan(p, magnitude=True)
    close(out, want["out"], mag["out"], 32 + 8 * T, "out")
    for k, gr in zip(names, got):
        close(gr, want["g_" + k], mag["g_" + k], 64 + 16 * T + B + 64, k)
    # the state alone, and out alone
    def run(no):
        o, s = sgr.selective_scan(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"], t.get("z"),
                                  t["delta_bias"], t["state0"], g["lengths"], softplus)
        return torch.autograd.grad(*((s, t["state0"], g["gstate"]) if no == "out" else
                                     (o, t["state0"], g["go"])))[0]
    for no, zero in (("out", "go"), ("state", "gstate")):
        q = dict(p, **{zero: np.zeros_like(p[zero])})
        close(run(no), ref.scan(q)["g_state0"], ref.scan(q, magnitude=True)["g_state0"],
              128 + 16 * T + B, no)


# --------------------------------------------------------------- convolution

def conv_problem(seed, T, B, D, W, dtype, silu, lengths, layout, state0=True, bias=True):
    r = np.random.default_rng(seed)
    ok = ref.valid(T, B, None if lengths is None else np.array(lengths))
    pad = None if lengths is None else ok
    gpu, p = {}, {"silu": silu, "lengths": None if lengths is None else np.array(lengths)}
    gpu["x"], p["x"] = place(r.standard_normal((T, B, D)), DT[dtype], layout, pad)
    gpu["gy"], p["gy"] = place(r.standard_normal((T, B, D)), DT[dtype], layout, pad)
    gpu["weight"], p["weight"] = _f32(r.standard_normal((D, W)))
    gpu["bias"] = gpu["state0"] = None
    if bias:
        gpu["bias"], p["bias"] = _f32(r.standard_normal(D))
    for k in ("state0", "gstate") if state0 else ("gstate",):
        t = torch.from_numpy(r.standard_normal((W - 1, B, D))).to(DT[dtype])
        gpu[k], p[k] = t.cuda(), t.double().numpy()
    gpu["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                               device="cuda")
    return gpu, p


def conv_run(g, silu, stream=None):
    kw = dict(bias=g["bias"], state0=g["state0"], lengths=g["lengths"],
              activation="silu" if silu else None, stream=stream)
    y, state = sgr.short_conv_forward(g["x"], g["weight"], **kw)
    return y, state, sgr.short_conv_backward(g["x"], g["weight"], g["gy"],
                                             grad_state=g["gstate"], **kw)


CONV = [  # T, B, D, W, dtype, silu, lengths, layout
    (1, 1, 1, 4, "fp32", True, None, "time"),
    (0, 2, 16, 4, "fp32", True, None, "time"),
    (2, 3, 64, 4, "bf16", True, None, "time"),
    (16, 2, 256, 4, "bf16", True, None, "time"),
    (17, 2, 72, 3, "fp16", False, None, "batch"),
    (33, 3, 1025, 4, "bf16", True, None, "time"),
    (65, 2, 520, 2, "fp32", True, None, "batch"),
    (40, 2, 64, 1, "fp32", True, None, "time"),
    (40, 2, 64, 8, "bf16", True, None, "time"),
    (70, 1, 24, 7, "fp32", True, None, "slice"),
    (35, 2, 40, 5, "fp16", True, None, "time"),
    (35, 2, 41, 6, "fp32", False, None, "batch"),
    (50, 7, 64, 4, "bf16", True, [0, 1, 2, 3, 50, 32, 33], "time"),
    (50, 6, 37, 4, "fp32", True, [0, 1, 2, 49, 16, 17], "batch"),
    (4, 3, 16, 8, "fp32", False, [0, 3, 4], "time"),
    (20, 4, 16, 4, "fp16", True, [-1, 21, 20, 5], "slice"),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c[:5])))
@pytest.mark.parametrize("full", [True, False])
def test_conv(case, full):
    T, B, D, W, dtype, silu, lengths, layout = case
    log(f"conv {case} full={full}")
    g, p = conv_problem(1, *case, state0=full, bias=full)
    want, mag = ref.conv(p), ref.conv(p, magnitude=True)
    y, state, grads = conv_run(g, silu)
    torch.cuda.synchronize()
    close(y, want["y"], mag["y"], 16 + 2 * W, "y")
    # the state is a copy of inputs
    assert np.array_equal(state.double().cpu().numpy(), want["state"])
    # sums over all steps and rows in runs and pieces of them
    for k, n in (("g_x", W), ("g_state0", W), ("g_weight", T * B), ("g_bias", T * B)):
        close(grads[k], want[k], mag[k], 24 + 2 * W + n, k)


# Backward runs longer than the 16 steps that few rows get: T, B, D, W, dtype, silu,
# and the run that these sizes select (no shorter one gives as few workgroups); T
# ends inside a run.
LONG_RUNS = [
    (81, 19558, 5, 4, "fp32", True, 20),
    (101, 39116, 3, 4, "bf16", True, 24),
    (121, 13004, 7, 7, "bf16", True, 28),
    (201, 13004, 6, 8, "fp32", True, 44),
    (221, 39116, 1, 3, "fp16", False, 48),
]


@pytest.mark.parametrize("case", LONG_RUNS, ids=lambda c: "-".join(map(str, c)))
def test_conv_long_runs(case):
    T, B, D, W, dtype, silu, run = case
    log(f"conv long runs {case}")
    # the workspace has a row of partial sums for each of the backward's workgroups along
    # time and rows: 256 threads, one run of 4 channels each
    def workgroups(run):
        return -(-B * -(-T // run) // (256 // -(-D // 4)))
    need = ctypes.c_size_t()
    sgr.lib().ck_conv_sizes(ctypes.byref(sequence.ConvShape(
        T, B, D, W, sequence._DTYPES[DT[dtype]], int(silu))), ctypes.byref(need))
    assert need.value == workgroups(run) * D * (W + 1) * 4
    assert workgroups(run) not in {workgroups(shorter) for shorter in range(16, run, 4)}
    # texts that end at a run's end, within W - 1 steps of it, anywhere and nowhere
    r = np.random.default_rng(7)
    ends = np.array([run * k + e for k in range(1, T // run + 1) for e in range(-W, W + 1)])
    lengths = np.where(r.random(B) < 0.5, r.choice(ends, B), r.integers(0, T + 1, B))
    lengths[::3] = T
    g, p = conv_problem(7, T, B, D, W, dtype, silu, np.minimum(lengths, T).tolist(), "time")
    want, mag = ref.conv(p), ref.conv(p, magnitude=True)
    _, state, grads = conv_run(g, silu)
    torch.cuda.synchronize()
    assert np.array_equal(state.double().cpu().numpy(), want["state"])
    # sums: a run's steps, a workgroup's 256 runs, an eighth of the workgroups, eight eighths
    n = 48 + 256 + workgroups(run) // 8 + 8
    for k, m in (("g_x", W), ("g_state0", W), ("g_weight", n), ("g_bias", n)):
        close(grads[k], want[k], mag[k], 24 + 2 * W + m, k)


# rows that end within a group of channels, at the end of a workgroup's or short of one
@pytest.mark.parametrize("D", [2, 3, 5, 6, 7, 254, 257, 259])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_conv_row_ends(D, dtype):
    test_conv((35, 3, D, 4, dtype, True, [35, 0, 20], "slice"), True)


@pytest.mark.parametrize("dtype,B,D,W", [("fp32", 1, 1, 4), ("bf16", 3, 64, 4),
                                         ("fp16", 2, 37, 3), ("fp32", 2, 20, 1),
                                         ("bf16", 2, 2048, 8)])
def test_conv_step_walks_the_window(dtype, B, D, W):
    T = 2 * W + 1
    g, p = conv_problem(2, T, B, D, W, dtype, True, None, "slice")
    want, mag = ref.conv(p), ref.conv(p, magnitude=True)
    state, ys = g["state0"].clone(), []
    for t in range(T):
        y, s = sgr.short_conv_step(state, g["x"][t], g["weight"], g["bias"], "silu")
        assert s is state
        ys.append(y)
    close(torch.stack(ys), want["y"], mag["y"], 16 + 2 * W, "y")
    assert np.array_equal(state.double().cpu().numpy(), want["state"])
    keep = g["state0"].clone()
    y, s = sgr.short_conv_step(g["state0"], g["x"][0], g["weight"], g["bias"], "silu",
                               new_state=torch.empty_like(keep))
    assert torch.equal(y, ys[0]) and torch.equal(g["state0"], keep)


def test_conv_autograd():
    """Through the autograd node, against fp64 differences along random
    directions of the definition."""
    g, p = conv_problem(3, 30, 2, 24, 4, "fp32", True, [30, 17], "time")
    x = torch.nan_to_num(g["x"]).requires_grad_()
    leaves = [x] + [g[k].clone().requires_grad_() for k in ("weight", "bias", "state0")]
    y, state = sgr.short_conv(leaves[0], leaves[1], leaves[2], leaves[3], g["lengths"], "silu")
    gy = torch.nan_to_num(g["gy"])
    ((y * gy).sum() + (state * g["gstate"]).sum()).backward()
    r = np.random.default_rng(9)
    names = ("x", "weight", "bias", "state0")
    q = {k: v for k, v in p.items() if k not in ("gy", "gstate")}
    loss = lambda o: (o["y"] * ref.cut(p["gy"], ref.valid(30, 2, p["lengths"]))).sum() + \
        (o["state"] * p["gstate"]).sum()
    for leaf, k in zip(leaves, names):
        d = r.standard_normal(p[k].shape)
        e = 1e-6
        hi, lo = (loss(ref.conv({**q, k: p[k] + s * e * d})) for s in (1, -1))
        slope = (leaf.grad.double().cpu().numpy() * d).sum()
        size = np.abs(leaf.grad.double().cpu().numpy() * d).sum()
        # the difference is good to about 1e-8, the fp32 gradient to 100 roundings
        assert abs(slope - (hi - lo) / (2 * e)) <= (100 * ref.U32 + 1e-7) * size, k


def rows_alone(p, lengths):
    """The definition with each row a window of its own length: nothing behind a
    row's text enters any sum."""
    T, B, D = p["x"].shape
    W = p["weight"].shape[1]
    r = {"y": np.zeros((T, B, D)), "g_x": np.zeros((T, B, D)), "state": np.zeros((W - 1, B, D)),
         "g_state0": np.zeros((W - 1, B, D)), "g_weight": np.zeros((D, W)), "g_bias": np.zeros(D)}
    for b, n in enumerate(lengths):
        q = {k: v[:n, b:b + 1] if k in ("x", "gy") else v[:, b:b + 1] if k in ("state0", "gstate")
             else v for k, v in p.items() if k != "lengths"}
        with np.errstate(all="ignore"):
            one = ref.conv(q)
            for k in ("g_weight", "g_bias"):
                r[k] += one[k]
        for k in ("y", "g_x"):
            r[k][:n, b] = one[k][:, 0]
        for k in ("state", "g_state0"):
            r[k][:, b] = one[k][:, 0]
    return r


@pytest.mark.parametrize("D", [3, 12, 66])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_conv_infinite_last_input_reaches_its_own_taps_alone(D, dtype):
    """Behind a row's end there are no steps: an infinite last input reaches the
    gradient of the tap that saw it, not those that would see it later."""
    lengths = [5, 16, 17, 0, 40, 36, 31, 33]
    g, p = conv_problem(5, 40, 8, D, 4, dtype, False, lengths, "time")
    for b, n in enumerate(lengths[:7]):
        if n:
            g["x"][n - 1, b, b % D] = float("inf")
            p["x"][n - 1, b, b % D] = np.inf
    want = rows_alone(p, lengths)
    _, _, grads = conv_run(g, False)
    torch.cuda.synchronize()
    p["x"] = np.where(np.isinf(p["x"]), 0.0, p["x"])
    mag = ref.conv(p, magnitude=True)
    for k in ("g_x", "g_weight", "g_bias", "g_state0"):
        fine = np.isfinite(want[k])
        got = grads[k].double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), fine), k
        close(torch.where(torch.from_numpy(fine).cuda(), grads[k], 0), np.where(fine, want[k], 0.0),
              mag[k], 24 + 8 + 320, k)
    assert np.isfinite(want["g_weight"][:, :3]).all() and not np.isfinite(want["g_weight"]).all()


def test_conv_overflow_behind_the_text_reaches_nothing():
    """With silu: the pre-activation overflows only at steps behind the text."""
    lengths = [5, 16, 17, 40, 20]
    g, p = conv_problem(6, 40, 5, 10, 4, "fp32", True, lengths, "batch")
    for k, w in (("weight", torch.tensor([2.0, 2.0, 2.0, 1e-30], device="cuda")),):
        g[k][:] = w
        p[k][:] = w.double().cpu().numpy()
    for b, n in enumerate(lengths):
        if n < 40:
            g["x"][n - 1, b], p["x"][n - 1, b] = 3e38, float(np.float32(3e38))
            g["gy"][n - 1, b], p["gy"][n - 1, b] = 0.0625, 0.0625
    want = rows_alone(p, lengths)
    y, state, grads = conv_run(g, True)
    torch.cuda.synchronize()
    for k, t in grads.items():
        assert np.isfinite(want[k]).all() and torch.isfinite(t).all(), k
        # every term's roundings, against the largest terms: the huge input's own
        size = np.abs(want[k]).max() if k == "g_weight" else np.maximum(np.abs(want[k]), 20.0)
        assert (np.abs(t.double().cpu().numpy() - want[k]) <= 400 * ref.U32 * size).all(), k


@pytest.mark.parametrize("T,B,D,W,dtype", [(37, 3, 41, 4, "bf16"), (20, 2, 3, 8, "fp32"),
                                           (5, 4, 260, 2, "fp16")])
def test_conv_into_given_tensors(T, B, D, W, dtype):
    g, p = conv_problem(33, T, B, D, W, dtype, True, [T] + [T // 2] * (B - 1), "slice")
    kw = dict(bias=g["bias"], state0=g["state0"], lengths=g["lengths"], activation="silu")
    y, state, wg = conv_run(g, True)
    oy, sy = given(y)
    os = torch.full_like(state, 7.0)
    r = sgr.short_conv_forward(g["x"], g["weight"], y=oy, state=os, **kw)
    assert r[0] is oy and r[1] is os and torch.equal(oy, y) and torch.equal(os, state)
    gx, sx = given(y)
    grads = dict({k: torch.full_like(v, 7.0) for k, v in wg.items()}, g_x=gx)
    need = sequence._conv_sizes(sequence._CONV_SHAPE.pack(T, B, D, W, sequence._DTYPES[DT[dtype]],
                                                          1))
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    assert sgr.short_conv_backward(g["x"], g["weight"], g["gy"], grad_state=g["gstate"],
                                   grads=grads, workspace=ws, **kw) is grads
    assert all(torch.equal(grads[k], wg[k]) for k in wg)
    assert untouched(sy, D) and untouched(sx, D) and bool((ws[need:] == 0x5A).all())
    some = {k: grads[k] for k in ("g_x", "g_weight")}
    sgr.short_conv_backward(g["x"], g["weight"], g["gy"], grad_state=g["gstate"], grads=some, **kw)
    assert all(torch.equal(some[k], wg[k]) for k in some)
    for bad in (dict(y=oy[:-1]), dict(state=os[:-1]), dict(y=oy.float() if dtype != "fp32" else
                                                          oy.bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            sgr.short_conv_forward(g["x"], g["weight"], **bad, **kw)
    for bad in (dict(workspace=ws[:need - 1]), dict(grads=dict(grads, g_x=gx[:-1])),
                dict(grads=dict(grads, g_weight=g["weight"].t().contiguous().t()))):
        with pytest.raises(ValueError):
            sgr.short_conv_backward(g["x"], g["weight"], g["gy"], **bad, **kw)


def test_conv_same_bits_every_time():
    g, _ = conv_problem(4, 100, 3, 200, 4, "bf16", True, [100, 50, 7], "time")
    a, b = conv_run(g, True), conv_run(g, True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(a[2][k], b[2][k]) for k in a[2])


# ------------------------------------------------------------------- dropout

@pytest.mark.parametrize("T,B,D,dtype,layout", [
    (1, 1, 1, "fp32", "time"), (5, 3, 64, "bf16", "time"), (9, 2, 37, "fp16", "batch"),
    (17, 2, 1000, "fp32", "time"), (8, 3, 40, "bf16", "slice"), (0, 2, 8, "fp32", "time")])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(T, B, D, dtype, layout, held, p):
    r = np.random.default_rng(10)
    x, xv = place(r.standard_normal((T, B, D)), DT[dtype], layout)
    res, rv = place(r.standard_normal((T, B, D)), DT[dtype], layout)
    seed, offset = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    m, scale = ref.keep(T, B, D, p, seed, offset, held)
    kw = dict(p=p, seed=seed, offset=offset, held=held)
    for got, want in ((sgr.dropout_forward(x, **kw), m * xv * scale),
                      (sgr.dropout_backward(x, **kw), m * xv * scale),
                      (sgr.dropout_forward(x, residual=res, **kw), rv + m * xv * scale)):
        # one product, one sum, the scale's own rounding
        close(got, want, np.abs(rv) + np.abs(xv) * scale, 3, "out")
    out = sgr.dropout_forward(x, **kw)
    assert np.array_equal((out != 0).cpu().numpy(), m & (xv != 0))


@pytest.mark.parametrize("D", [2, 3, 4, 5, 6, 7, 9, 10, 11, 12, 14, 15, 518])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_dropout_row_ends(D, dtype):
    test_dropout(6, 3, D, dtype, "slice", True, 0.3)
    test_dropout(6, 3, D, dtype, "time", False, 0.3)
    # nothing past a row's end is written
    wide = torch.full((6, 3, D + 3), 5.0, dtype=DT[dtype], device="cuda")
    sgr.dropout_forward(torch.randn(6, 3, D, device="cuda").to(DT[dtype]), 0.3, seed=1,
                        out=wide[:, :, 1:1 + D])
    assert bool((wide[:, :, 0] == 5).all()) and bool((wide[:, :, 1 + D:] == 5).all())


def test_dropout_nan_counter_in_place_and_autograd():
    x = torch.randn(6, 4, 100, device="cuda")
    m, scale = ref.keep(6, 4, 100, 0.4, 7, 3, True)
    keep = torch.from_numpy(m.copy()).cuda()
    bad = torch.where(keep, x, torch.full_like(x, float("nan")))
    ok = sgr.dropout_forward(bad, 0.4, 7, 3, held=True)
    assert torch.isfinite(ok).all() and not ok[~keep].any()
    # the counter adds to the offset
    c = torch.tensor([3], dtype=torch.int64, device="cuda")
    assert torch.equal(sgr.dropout_forward(x, 0.4, 7, 0, held=True, counter=c),
                       sgr.dropout_forward(x, 0.4, 7, 3, held=True))
    y = x.clone()
    assert sgr.dropout_forward(y, 0.4, 7, 3, held=True, out=y) is y
    assert torch.equal(y, sgr.dropout_forward(x, 0.4, 7, 3, held=True))
    leaf, res = x.clone().requires_grad_(), torch.randn_like(x).requires_grad_()
    out = sgr.dropout(leaf, 0.4, 7, 0, residual=res, held=True, counter=c)
    c += 5  # a later step's value does not change this step's mask
    go = torch.randn_like(x)
    out.backward(go)
    assert torch.equal(leaf.grad, sgr.dropout_backward(go, 0.4, 7, 3, held=True))
    assert torch.equal(res.grad, go)
    # one step's rows, as in a token's path
    assert torch.equal(sgr.dropout_forward(x[0], 0.4, 7, 3), sgr.dropout_forward(x[:1], 0.4, 7, 3)[0])


def test_a_write_into_a_saved_tensor_is_seen():
    """What a call writes into, a pending backward may have saved: it raises, as
    behind torch's in-place operations, and does not use the new values."""
    x = torch.randn(5, 2, 8, device="cuda")
    w = torch.randn(8, 4, device="cuda", requires_grad=True)
    A, b = -torch.ones(8, 2, device="cuda"), torch.randn(5, 2, 1, 2, device="cuda")
    h = torch.zeros(2, 8, 2, device="cuda")

    def fresh():
        s0 = torch.randn(3, 2, 8, device="cuda")
        y, _ = sgr.short_conv(x, w, state0=s0)
        return y.sum(), s0

    def pending(shape):
        t = torch.randn(shape, device="cuda")
        return (t * torch.ones_like(t).requires_grad_()).sum(), t

    def cases():
        loss, s0 = fresh()
        yield loss, lambda: sgr.short_conv_step(s0, x[0], w.detach())
        loss, t = pending((2, 8, 2))
        yield loss, lambda: sgr.selective_scan_step(t, x[0], x[0], A, b[0], b[0])
        for call in (lambda t: sgr.dropout_forward(t, 0.5, 1, out=t),
                     lambda t: sgr.dropout_backward(t, 0.5, 1, grad_x=t),
                     lambda t: sgr.short_conv_forward(x, w.detach(), y=t),
                     lambda t: sgr.selective_scan_forward(x, x, A, b, b, out=t),
                     lambda t: sgr.short_conv_step(fresh()[1], x[0], w.detach(), y=t[0])):
            loss, t = pending((5, 2, 8))
            yield loss, lambda: call(t)
        loss, t = pending((2, 8, 2))
        yield loss, lambda: sgr.selective_scan_forward(x, x, A, b, b, state=t)
        loss, t = pending((5, 2, 8))
        g = sgr.short_conv_backward(x, w.detach(), x)
        yield loss, lambda: sgr.short_conv_backward(x, w.detach(), x, grads=dict(g, g_x=t))
        loss, t = pending((8, 2))
        f = sgr.selective_scan_forward(x, x, A, b, b)
        g = sgr.selective_scan_backward(x, x, A, b, b, f[2], x)
        yield loss, lambda: sgr.selective_scan_backward(x, x, A, b, b, f[2], x,
                                                        grads=dict(g, g_A=t))

    for i, (loss, write) in enumerate(cases()):
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
            pytest.fail(f"case {i}")


# --------------------------------------------------- large offsets and graphs

def test_offsets_past_32_bits():
    """Rows of one storage more than 2^31 elements apart."""
    far = 2 ** 31 + 64
    T, D, N = 18, 64, 16
    g, p = scan_problem(11, T, 2, D, N, 1, "bf16", True, True, None, "time")
    store = torch.zeros(far + 4 * T * D, dtype=torch.bfloat16, device="cuda")
    def spread(t, at):
        v = store.as_strided((T, 2, D), (D, far, 1), at * T * D)
        v.copy_(t)
        return v
    for i, k in enumerate(("u", "delta", "z", "go")):
        g[k] = spread(g[k], i)
    scan_check(g, p, True)
    conv, q = conv_problem(12, T, 2, D, 4, "bf16", True, None, "time")
    conv["x"], conv["gy"] = spread(conv["x"], 0), spread(conv["gy"], 1)
    y, state, grads = conv_run(conv, True)
    want, mag = ref.conv(q), ref.conv(q, magnitude=True)
    close(y, want["y"], mag["y"], 24, "y")
    close(grads["g_x"], want["g_x"], mag["g_x"], 36, "g_x")
    x = spread(conv["x"], 2)
    out = spread(torch.zeros(T, 2, D, dtype=torch.bfloat16, device="cuda"), 3)
    sgr.dropout_forward(x, 0.5, 1, out=out)
    assert torch.equal(out, sgr.dropout_forward(x.contiguous(), 0.5, 1))


def test_long_step_strides():
    """Steps 2^24 elements and more apart, as in a window of many wide rows."""
    def far(t, stride, fill=None):
        T = t.shape[0]
        v = torch.empty((T - 1) * stride + t[0].numel(), dtype=t.dtype, device="cuda")
        v = v.as_strided(t.shape, (stride,) + tuple(t[0].stride()), 0)
        return v.copy_(t) if fill is None else v.fill_(fill)

    x = torch.randn(5, 3, 70, device="cuda").bfloat16()
    r = torch.randn_like(x)
    for stride in (2**24, 2**31 + 2):
        out = sgr.dropout_forward(far(x, stride), 0.3, 5, residual=far(r, stride),
                                  out=far(x, stride, 0))
        assert torch.equal(out, sgr.dropout_forward(x, 0.3, 5, residual=r)), stride
    g, p = conv_problem(14, 22, 2, 70, 4, "bf16", True, [22, 9], "time")
    want = conv_run(g, True)
    f = dict(g, x=far(g["x"], 2**27 + 6), gy=far(g["gy"], 2**27 + 6))
    y = far(g["x"], 2**27 + 6, 0)
    sgr.short_conv_forward(f["x"], f["weight"], f["bias"], f["state0"], f["lengths"], "silu", y=y)
    got = conv_run(f, True)
    assert torch.equal(y, want[0]) and torch.equal(got[0], want[0])
    assert all(torch.equal(got[2][k], want[2][k]) for k in want[2])
    # the scan: a workgroup each; cut
    for T, B, D, far_by in ((9, 400, 20, 2**26 + 2), (100, 2, 40, 2**25)):
        g, p = scan_problem(24, T, B, D, 16, 1, "bf16", True, True, None, "time")
        want = scan_run(g, True)
        f = dict(g, **{k: far(g[k], far_by) for k in ("u", "delta", "z", "go")})
        f.update({k: far(g[k], 2**24 + 2) for k in ("B", "C")})
        got = scan_run(f, True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(got[2][k], want[2][k]) for k in want[2])
    del f, y, out
    torch.cuda.empty_cache()  # (some 30 GB of it)


def test_more_workgroups_than_a_grid_dimension_holds():
    """Launches that go on in the grid's second dimension (from 2^22 workgroups on)."""
    # dropout, 2^20 + 1024 rows of 8192 channels, in place
    T, B, D = 1025, 1024, 8192
    x = torch.ones(T, B, D, dtype=torch.bfloat16, device="cuda")
    sgr.dropout_forward(x, 0.25, 7, 3, out=x)
    for t, b in ((0, 0), (1023, 1023), (1024, 0), (1024, 1023)):
        ctr = np.zeros((D // 8, 4), np.uint64)
        ctr[:, 0], ctr[:, 1], ctr[:, 2] = np.arange(D // 8), t * B + b, 3
        w = ref.philox(ctr, (7, 0))
        r = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(D)
        want = torch.from_numpy(np.where(r >= 16384, 65536 / 49152, 0.0)).bfloat16()
        assert torch.equal(x[t, b].cpu(), want), (t, b)
    del x
    # sums of the gradients of B and C, 4097 x 256 x 64 groups; rows are independent
    T, B, D = 4097, 256, 64
    mk = lambda *shape: torch.randn(*shape, device="cuda").bfloat16()
    u, go = mk(T, B, D), mk(T, B, D)
    bm, cm = mk(T, B, D, 1), mk(T, B, D, 1)
    delta, A = 0.1 * u.abs() + 0.1, -torch.ones(D, 1, device="cuda")

    def grads(rows):
        a = (u[:, rows], delta[:, rows], A, bm[:, rows], cm[:, rows])
        saved = sgr.selective_scan_forward(*a)[2]
        return sgr.selective_scan_backward(*a, saved, go[:, rows])

    whole = grads(slice(0, B))
    for rows in (slice(0, 8), slice(B - 8, B)):
        few = grads(rows)
        for k in ("g_B", "g_C", "g_u"):
            assert torch.equal(whole[k][:, rows], few[k]), (k, rows)
    assert torch.isfinite(whole["g_A"]).all()
    del u, go, bm, cm, delta, whole, few
    # single tokens: 2^28 + 1024 channels, 2^32 + 4096 channels
    B, D = 2**18 + 1, 1024
    a = [mk(B, D), mk(B, D), -torch.ones(D, 1, device="cuda"), mk(B, 1, 1), mk(B, 1, 1)]
    state = torch.randn(B, D, 1, device="cuda")
    out, new = sgr.selective_scan_step(state, *a, new_state=torch.empty_like(state))
    for rows in (slice(0, 2), slice(B - 2, B)):
        one, s1 = sgr.selective_scan_step(state[rows].clone(), a[0][rows], a[1][rows], a[2],
                                          a[3][rows], a[4][rows])
        assert torch.equal(out[rows], one) and torch.equal(new[rows], s1), rows
    del a, state, out, new
    B, D = 2**20 + 1, 4096
    x = torch.empty(B, D, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    w, state = torch.randn(D, 2, device="cuda"), x.unsqueeze(0) * 0.5
    y, new = sgr.short_conv_step(state, x, w, new_state=torch.empty_like(state))
    for rows in (slice(0, 2), slice(B - 2, B)):
        one, s1 = sgr.short_conv_step(state[:, rows].contiguous(), x[rows], w)
        assert torch.equal(y[rows], one) and torch.equal(new[:, rows], s1), rows
    del x, state, y, new
    torch.cuda.empty_cache()


def test_captured_graph_replays():
    """Forward, backward and tokens in one HIP graph: every replay equals the
    eager result on the inputs of that moment, with eager work between."""
    g, p = scan_problem(13, 40, 2, 64, 16, 1, "fp32", True, True, [40, 23], "time", nan=False)
    w = torch.randn(64, 4, device="cuda")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    step_state = torch.zeros(2, 64, 16, device="cuda")

    def work():
        x, _ = sgr.short_conv_forward(g["u"], w, activation="silu")
        h = dict(g, u=x)
        out, state, grads = scan_run(h, True)
        cg = sgr.short_conv_backward(g["u"], w, grads["g_u"], activation="silu")
        tok, _ = sgr.selective_scan_step(step_state, x[0], g["delta"][0], g["A"], g["B"][0],
                                         g["C"][0], new_state=torch.empty_like(step_state))
        dr = sgr.dropout_forward(out, 0.3, 5, residual=x, counter=counter)
        return [out, state, cg["g_x"], cg["g_weight"], tok, dr] + list(grads.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = work()
    for i in range(4):
        g["u"].copy_(torch.randn_like(g["u"]))
        counter.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(res, work())):
            assert torch.equal(a, b), (i, k)


def test_binding_refusals():
    g, _ = scan_problem(14, 4, 2, 8, 4, 1, "fp32", True, True, None, "time")
    args = lambda **kw: [{**g, **kw}[k] for k in ("u", "delta", "A", "B", "C")]
    for kw, err in ((dict(u=g["u"].double()), TypeError), (dict(u=g["u"].cpu()), TypeError),
                    (dict(delta=g["delta"].bfloat16()), TypeError),
                    (dict(delta=g["delta"][:2]), ValueError),
                    (dict(B=g["B"][:, :, :, :2]), ValueError),
                    (dict(A=g["A"].bfloat16()), TypeError),
                    (dict(u=g["u"].transpose(0, 2).contiguous().transpose(0, 2)), ValueError)):
        with pytest.raises(err):
            sgr.selective_scan_forward(*args(**kw))
    with pytest.raises(ValueError):
        sgr.selective_scan_forward(*args(), lengths=torch.zeros(3, dtype=torch.int32,
                                                                device="cuda"))
    with pytest.raises(TypeError):
        sgr.selective_scan_forward(*args(), lengths=torch.zeros(2, dtype=torch.int64,
                                                                device="cuda"))
    with pytest.raises(ValueError):
        sgr.selective_scan_backward(*args(), None, g["go"][:2])
    with pytest.raises(ValueError):
        sgr.short_conv_forward(g["u"], torch.ones(8, 4, device="cuda"), activation="tanh")
    with pytest.raises(sgr.CkError):
        sgr.short_conv_forward(g["u"], torch.ones(8, 9, device="cuda"))
    with pytest.raises(sgr.CkError):
        sgr.dropout_forward(g["u"], 1.5, 1)
    # the autograd node takes what the calls refuse for its layout alone
    u = g["u"].transpose(0, 2).contiguous().transpose(0, 2)
    a, _ = sgr.selective_scan(*args(u=u))
    assert torch.equal(a, sgr.selective_scan(*args())[0])


# ------------------------------------------------------------------- streams

def _flat(res):
    return [t for r in res for t in (r.values() if isinstance(r, dict) else
                                     r if isinstance(r, tuple) else (r,)) if t is not None]


def _ranges(res):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in _flat(res)]


@pytest.mark.parametrize("op", ["scan", "conv", "dropout", "steps"])
def test_a_call_on_another_stream_takes_no_memory_of_the_current_one(op):
    """What a call with stream= allocates is that stream's memory: blocks freed on
    the current stream, which work queued there may still read, are not among it."""
    side = torch.cuda.Stream()
    g, _ = scan_problem(21, 40, 8, 256, 16, 1, "fp32", True, True, None, "time")
    w, x, state = torch.randn(256, 4, device="cuda"), g["u"], torch.zeros(3, 8, 256, device="cuda")

    def work(stream):
        if op == "scan":
            a = (g["u"], g["delta"], g["A"], g["B"], g["C"])
            o = dict(D=g["D"], z=g["z"], delta_bias=g["delta_bias"], stream=stream)
            f = sgr.selective_scan_forward(*a, **o)
            return f, sgr.selective_scan_backward(*a, f[2], g["go"], **o)
        if op == "conv":
            return (sgr.short_conv_forward(x, w, stream=stream),
                    sgr.short_conv_backward(x, w, g["go"], stream=stream))
        if op == "dropout":
            return (sgr.dropout_forward(x, 0.5, 1, stream=stream),
                    sgr.dropout_backward(x, 0.5, 1, stream=stream))
        return (sgr.selective_scan_step(g["state0"], g["u"][0], g["delta"][0], g["A"], g["B"][0],
                                        g["C"][0], stream=stream)[0],
                sgr.short_conv_step(state, x[0], w, stream=stream)[0])

    # the current stream's free blocks: one of every size that the call makes, twice
    old = [work(None), work(None)]
    torch.cuda.synchronize()
    freed = _ranges(old[0]) + _ranges(old[1])
    del old
    res = work(side)
    torch.cuda.current_stream().wait_stream(side)
    made = _ranges(res)
    assert made
    for lo, hi in made:
        assert not any(lo < b and a < hi for a, b in freed), (lo, hi)
    want = work(None)
    torch.cuda.synchronize()
    if op == "steps":  # (the states have moved on)
        return
    for i, (a, b) in enumerate(zip(_flat(res), _flat(want))):
        # bit for bit: the steps' negative dt makes states outgrow fp32 here
        if a.dtype == torch.float32:
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), i


def test_a_call_on_another_stream_leaves_the_current_one_current():
    """The current stream is the caller's again behind a call, also one that raises."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = torch.randn(4, 2, 8, device="cuda")
    before = torch.cuda.current_stream()
    sgr.dropout_forward(x, 0.5, 1, stream=side)
    assert torch.cuda.current_stream() == before
    with pytest.raises(sgr.CkError):
        sgr.dropout_forward(x, 1.5, 1, stream=side)
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
