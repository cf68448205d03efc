"""The gated scan against its fp64 definition, at the sizes, lengths, strides and
types where such kernels go wrong.  Every output is held to

    |got - want| <= (eps / 2) (|want| + err) + err

where eps / 2 is the one rounding to the output's type and err the running bound of
``gated_ref``."""
import numpy as np
import pytest
import torch

import gated_ref as ref
import sparse_graph_recurrent_amd as sgr
from gpu_helpers import log
from sequence_ref import valid

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def close(got, want, name):
    want, err = want
    fi = torch.finfo(got.dtype)
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.shape, name
    tol = fi.eps / 2 * (np.abs(want) + err) + err + fi.smallest_normal * fi.eps
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                           f"{np.nanmax(np.abs(g - want) / tol):.3g} times it, "
                           f"{np.isnan(g).sum()} NaN, first at {np.argwhere(bad)[0]}")


def place(a, dtype, layout, pad=None):
    """(the array on the device in a storage, its exact values): "time" contiguous,
    "batch" batch outermost, "slice" of a wider tensor (odd offset and strides); `pad`:
    where it holds NaN instead."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype])
    val = t.double().numpy()
    if pad is not None:
        t[torch.from_numpy(pad)] = float("nan")
    T, B, D = t.shape
    if layout == "batch":
        s = torch.empty((B, T, D), dtype=t.dtype, device="cuda").transpose(0, 1)
    elif layout == "slice":
        s = torch.full((T, B, D + 5), 7.0, dtype=t.dtype, device="cuda")[:, :, 3:3 + D]
    else:
        s = torch.empty(t.shape, dtype=t.dtype, device="cuda")
    s.copy_(t)
    return s, val


def problem(seed, T, B, D, dtype, own, z, lengths, layout, bias=True, state0=True, spread=2.0):
    """(device tensors, the same values in fp64)."""
    r = np.random.default_rng(seed)
    pad = None if lengths is None else ~valid(T, B, np.array(lengths))
    p = {"lengths": None if lengths is None else np.array(lengths)}
    g = {"lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                              device="cuda")}
    for k, on in (("x", True), ("f", True), ("i", own), ("z", z), ("go", True)):
        g[k] = p[k] = None
        if on:
            a = r.standard_normal((T, B, D)) * (spread if k in "fi" else 1.0)
            g[k], p[k] = place(a, dtype, layout, pad)
    for k, on, shape in (("f_bias", bias, (D,)), ("i_bias", bias and own, (D,)),
                         ("state0", state0, (B, D)), ("gstate", True, (B, D))):
        g[k] = p[k] = None
        if on:
            t = torch.from_numpy(r.standard_normal(shape) + (2.0 if k == "f_bias" else 0.0)).float()
            g[k], p[k] = t.cuda(), t.double().numpy()
    return g, p


def run(g, stream=None):
    kw = dict(i=g["i"], z=g["z"], f_bias=g["f_bias"], i_bias=g["i_bias"], lengths=g["lengths"],
              stream=stream)
    out, state, saved, _ = sgr.gated_scan_forward(g["x"], g["f"], state0=g["state0"], **kw)
    return out, state, sgr.gated_scan_backward(g["x"], g["f"], saved, g["go"],
                                               grad_state=g["gstate"], **kw)


def check(g, p, got=None):
    want = ref.gated(p)
    out, state, grads = got or run(g)
    torch.cuda.synchronize()
    close(out, want["out"], "out")
    close(state, want["state"], "state")
    assert set(grads) >= {k for k in want if k.startswith("g_")}
    for k, t in grads.items():
        close(t, want[k], k)


CASES = [  # T, B, D, dtype, own input gate, output gate, lengths, layout
    (1, 1, 1, "fp32", False, False, None, "time"),
    (1, 1, 1, "bf16", True, True, None, "time"),
    (9, 3, 1, "fp16", True, True, [9, 0, 4], "slice"),
    (8, 2, 64, "bf16", True, True, None, "time"),
    (7, 2, 65, "fp16", False, True, None, "slice"),
    (16, 1, 32, "fp32", True, False, None, "time"),
    (17, 3, 33, "fp32", False, False, [17, 16, 1], "batch"),
    (31, 2, 63, "bf16", True, False, [8, 31], "slice"),
    (33, 2, 129, "bf16", False, True, None, "batch"),
    (64, 5, 96, "fp32", True, True, [64, 63, 0, 7, 9], "time"),
    (65, 1, 2, "fp16", True, True, None, "time"),
    (255, 2, 40, "bf16", True, True, [255, 100], "batch"),
    (256, 1, 66, "fp32", False, True, None, "slice"),
    (257, 3, 70, "fp16", True, False, [257, 256, 255], "time"),
    (300, 4, 3, "bf16", False, False, [-1, 301, 300, 8], "slice"),
]
CUT = [  # few rows: every window of 128 steps is a workgroup, runs of eight windows
    (129, 1, 64, "fp32", True, True, [129], "time"),
    (1024, 5, 33, "fp16", False, False, [1024, 1023, 897, 896, 128], "time"),
    (1025, 4, 64, "bf16", True, False, [1025, 1024, 0, 129], "slice"),
    (2200, 5, 31, "fp32", True, True, [2200, 2049, 2048, 2047, 1], "batch"),
    (513, 1, 64, "bf16", True, True, None, "time"),
    (1000, 1, 63, "fp32", True, True, None, "slice"),
    (1025, 2, 65, "fp16", False, True, [1025, 511], "batch"),
    (2049, 1, 1, "bf16", True, False, None, "time"),
    (3000, 3, 34, "bf16", True, True, [0, 1600, 3000], "batch"),
    (2048, 8, 40, "fp32", False, False, None, "time"),
    (4099, 1, 130, "bf16", True, True, [4000], "slice"),
]


@pytest.mark.parametrize("case", CASES + CUT, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan(case):
    log(f"gated {case}")
    check(*problem(1, *case))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_columns(dtype):
    """More columns than CUs."""
    check(*problem(2, 150, 40, 1030, dtype, True, True, None, "batch"))


LENS = [900, 0, 1, 127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 512, 513, 640] * 2


@pytest.mark.parametrize("own,z", [(True, True), (False, False)])
@pytest.mark.parametrize("lengths", [None, LENS])
def test_a_column_a_cu(own, z, lengths):
    """As many columns as CUs: workgroups that go through all windows of one."""
    check(*problem(20, 900, 32, 256, "fp32", own, z, lengths, "time"))
    check(*problem(21, 300, 8, 2048, "bf16", own, z, lengths and lengths[:8], "slice"))


@pytest.mark.parametrize("own", [True, False])
def test_without_optional_inputs(own):
    check(*problem(3, 40, 2, 70, "fp32", own, False, None, "time", bias=False, state0=False))


@pytest.mark.parametrize("dtype,spread", [("fp32", 12.0), ("bf16", 30.0)])
def test_gates_that_are_shut_or_open(dtype, spread):
    """Gates far out on both sides: what passes them is still held to its own size."""
    check(*problem(4, 100, 2, 64, dtype, True, True, None, "time", bias=False, spread=spread))
    check(*problem(5, 600, 1, 64, dtype, False, True, [590], "time", bias=False, spread=spread))


def test_infinite_gates():
    """+inf keeps a state (or lets an input in) as it is, -inf forgets it."""
    T, B, D = 40, 2, 34
    for own in (True, False):
        g, p = problem(6, T, B, D, "fp32", own, False, None, "time", bias=False)
        for k in ("f", "i") if own else ("f",):
            for t, b, d, v in ((0, 0, 0, np.inf), (20, 1, 33, -np.inf), (39, 0, 5, np.inf),
                               (39, 1, 5, -np.inf), (8, 0, 7, -np.inf), (15, 0, 7, np.inf)):
                g[k][t, b, d] = v
                p[k][t, b, d] = np.copysign(1e4, v)   # the same to fp64, without 0 * inf
        check(g, p)


def test_a_long_memory_is_kept():
    """Gates that keep all but 2^-20 of a state a step: the rounding of a decay next to 1
    would by itself change a state by T 2^-25 of it."""
    T = 5000
    g, p = problem(7, T, 1, 64, "fp32", True, False, None, "time", bias=False)
    v = float(np.float32(20 * np.log(2.0)))
    g["f"].fill_(v), g["i"].fill_(-200.0)
    p["f"][:], p["i"][:] = v, -200.0
    want = p["state0"] * np.exp(-T * np.log1p(np.exp(-v)))
    out, state, _ = run(g)
    # a step rounds the state once, at random: T^0.5 half steps, and the gate by 32 U of q
    got = state.double().cpu().numpy()
    assert np.abs(got / want - 1).max() <= 8 * T ** 0.5 * 2.0 ** -24
    check(g, p)


def test_empty_window_passes_the_state():
    g, _ = problem(8, 1, 3, 40, "bf16", True, True, None, "time")
    for k in ("x", "f", "i", "z", "go"):
        g[k] = g[k][:0]
    out, state, grads = run(g)
    assert out.shape == (0, 3, 40) and torch.equal(state, g["state0"])
    assert torch.equal(grads["g_state0"], g["gstate"])
    for k in ("g_f_bias", "g_i_bias"):
        assert not grads[k].any()


def test_padding_is_written_and_not_read():
    """Outputs behind a row's text are 0 whatever they held; NaN inputs there reach nothing."""
    g, p = problem(9, 300, 3, 65, "bf16", True, True, [300, 0, 131], "time")
    out = torch.full((300, 3, 65), float("nan"), dtype=torch.bfloat16, device="cuda")
    grads = {k: torch.full_like(out, float("nan")) for k in ("g_x", "g_f", "g_i", "g_z")}
    kw = dict(i=g["i"], z=g["z"], f_bias=g["f_bias"], i_bias=g["i_bias"], lengths=g["lengths"])
    _, state, saved, _ = sgr.gated_scan_forward(g["x"], g["f"], state0=g["state0"], out=out, **kw)
    sgr.gated_scan_backward(g["x"], g["f"], saved, g["go"], grad_state=g["gstate"], grads=grads,
                            **kw)
    want = ref.gated(p)
    close(out, want["out"], "out")
    for k, t in grads.items():
        close(t, want[k], k)


def test_windows_follow_one_another():
    """A window in two parts, the state carried, is the window (and its gradients)."""
    g, p = problem(10, 200, 2, 70, "fp32", True, True, None, "time")
    want = ref.gated(p)
    cut = lambda a, b: {k: g[k][a:b] for k in ("x", "f", "i", "z")}
    kw = dict(f_bias=g["f_bias"], i_bias=g["i_bias"])
    first, second = cut(0, 77), cut(77, 200)
    o1, s1, v1, _ = sgr.gated_scan_forward(**first, state0=g["state0"], **kw)
    o2, s2, v2, _ = sgr.gated_scan_forward(**second, state0=s1, **kw)
    close(torch.cat([o1, o2]), want["out"], "out")
    close(s2, want["state"], "state")
    b2 = sgr.gated_scan_backward(saved=v2, grad_out=g["go"][77:], grad_state=g["gstate"], **second,
                                 **kw)
    b1 = sgr.gated_scan_backward(saved=v1, grad_out=g["go"][:77], grad_state=b2["g_state0"],
                                 **first, **kw)
    close(b1["g_state0"], want["g_state0"], "g_state0")
    for k in ("g_x", "g_f", "g_i", "g_z"):
        close(torch.cat([b1[k], b2[k]]), want[k], k)


@pytest.mark.parametrize("dtype,B,D", [("fp32", 1, 1), ("bf16", 3, 65), ("fp16", 2, 1),
                                       ("bf16", 70, 64)])
@pytest.mark.parametrize("own,z", [(True, True), (False, False)])
def test_step_walks_the_window(dtype, B, D, own, z):
    T = 6
    g, p = problem(11, T, B, D, dtype, own, z, None, "slice")
    want = ref.gated(p)
    state, outs = g["state0"].clone(), []
    at = lambda k, t: None if g[k] is None else g[k][t]
    for t in range(T):
        kw = dict(f_bias=g["f_bias"], i_bias=g["i_bias"])
        if t % 2:
            old, new = state, torch.empty_like(state)
            out, state = sgr.gated_scan_step(old, at("x", t), at("f", t), at("i", t), at("z", t),
                                             new_state=new, **kw)
            assert state is new
        else:
            out, same = sgr.gated_scan_step(state, at("x", t), at("f", t), at("i", t), at("z", t),
                                            **kw)
            assert same is state
        outs.append(out)
    close(torch.stack(outs), want["out"], "out")
    close(state, want["state"], "state")


def test_autograd_reaches_every_input():
    g, p = problem(12, 70, 2, 66, "fp32", True, True, [70, 33], "batch")
    names = ("x", "f", "i", "z", "f_bias", "i_bias", "state0")
    leaf = {k: torch.nan_to_num(g[k]).requires_grad_() for k in names}
    args = [leaf[k] for k in names] + [g["lengths"]]
    out, state = sgr.gated_scan(*args)
    go = torch.nan_to_num(g["go"])
    got = torch.autograd.grad([out, state], [leaf[k] for k in names], [go, g["gstate"]])
    want = ref.gated(p)
    for k, t in zip(names, got):
        close(t, want["g_" + k], k)
    # one of the two outputs alone
    out, state = sgr.gated_scan(*args)
    close(torch.autograd.grad(state, leaf["state0"], g["gstate"])[0],
          ref.gated(dict(p, go=0 * p["go"]))["g_state0"], "state alone")
    out, state = sgr.gated_scan(*args)
    close(torch.autograd.grad(out, leaf["x"], go)[0],
          ref.gated(dict(p, gstate=0 * p["gstate"]))["g_x"], "out alone")


def test_autograd_adds_up_broadcast_and_shared_inputs():
    """One tensor as input and gate, a gate the same at every step: their gradients add up."""
    r = np.random.default_rng(13)
    T, B, D = 30, 2, 36
    x = torch.from_numpy(r.standard_normal((T, B, D))).float().cuda().requires_grad_()
    f = torch.from_numpy(r.standard_normal((1, 1, D))).float().cuda().requires_grad_()
    go = torch.from_numpy(r.standard_normal((T, B, D))).float().cuda()
    out, _ = sgr.gated_scan(x, f.expand(T, B, D), x)
    gx, gf = torch.autograd.grad(out, [x, f], go)
    xv = x.detach().double().cpu().numpy()
    want = ref.gated({"x": xv, "f": np.broadcast_to(f.detach().double().cpu().numpy(), (T, B, D)),
                      "i": xv, "z": None, "go": go.double().cpu().numpy(),
                      "gstate": np.zeros((B, D))})
    close(gx, tuple(a + b for a, b in zip(want["g_x"], want["g_i"])), "x")
    v, e = (a.sum((0, 1))[None, None] for a in want["g_f"])
    close(gf, (v, e + T * B * 2.0 ** -24 * np.abs(want["g_f"][0]).sum((0, 1))), "f")


def test_no_states_are_left_without_a_backward(monkeypatch):
    g, _ = problem(14, 20, 2, 8, "fp32", True, True, None, "time")
    asked = []
    forward = sgr.sequence.gated_scan_forward

    def spy(*a, save=True, **kw):
        asked.append(save)
        return forward(*a, save=save, **kw)

    monkeypatch.setattr(sgr.sequence, "gated_scan_forward", spy)
    x = g["x"].requires_grad_()
    sgr.gated_scan(x, g["f"])
    with torch.no_grad():
        sgr.gated_scan(x, g["f"])
    sgr.gated_scan(x.detach(), g["f"])
    assert asked == [True, False, False]


def test_same_bits_every_time_and_on_another_stream():
    g, _ = problem(15, 1500, 1, 130, "bf16", True, True, [1490], "time")
    first = run(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (run(g), run(g, stream=side)):
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*first[:2], *first[2].values()), (*got[:2], *got[2].values())):
            assert torch.equal(a, b)


def test_calls_side_by_side():
    """Windows wait for one another within their call alone: several calls at once, with
    other work, come to the bits of one after the other; the workspace may hold anything."""
    probs = [problem(22 + k, 1500 + 100 * k, 2, 500, "bf16", True, True, None, "time")[0]
             for k in range(3)]
    want = [run(g) for g in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    ws = [torch.randint(0, 256, (8 << 20,), dtype=torch.uint8, device="cuda") for _ in probs]
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    got = [[] for _ in probs]
    for _ in range(5):
        for k, (g, st) in enumerate(zip(probs, streams)):
            kw = dict(i=g["i"], z=g["z"], f_bias=g["f_bias"], i_bias=g["i_bias"],
                      workspace=ws[k], stream=st)
            out, state, saved, _ = sgr.gated_scan_forward(g["x"], g["f"], state0=g["state0"], **kw)
            grads = sgr.gated_scan_backward(g["x"], g["f"], saved, g["go"],
                                            grad_state=g["gstate"], **kw)
            got[k].append((out, state, *grads.values()))
        busy = busy @ busy * 1e-3
    torch.cuda.synchronize()
    for w, rounds in zip(want, got):
        w = (w[0], w[1], *w[2].values())
        for res in rounds:
            assert all(map(torch.equal, w, res))


@pytest.mark.parametrize("T,stride", [(40, (1 << 26) - 1), (1000, (1 << 21) + 3)])
def test_long_strides_and_offsets_past_32_bits(T, stride):
    """The longest strides, and such as leave a window fewer waves; rows that end past
    2^32 bytes."""
    D = 40
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    far = torch.empty((T - 1) * stride + 2 * D, dtype=torch.float32, device="cuda")
    x = far.as_strided((T, 2, D), (stride, D, 1))
    g, p = problem(16, T, 2, D, "fp32", True, True, [T, T - 3], "time")
    near = run(g)
    for k in ("x", "f", "i", "z", "go"):
        x.copy_(g[k])
        check(g, p, run(dict(g, **{k: x})))
    kw = dict(i=g["i"], z=g["z"], f_bias=g["f_bias"], i_bias=g["i_bias"], lengths=g["lengths"])
    _, _, saved, _ = sgr.gated_scan_forward(g["x"], g["f"], state0=g["state0"], out=x, **kw)
    close(x, ref.gated(p)["out"], "out")
    for k in ("g_x", "g_f", "g_i", "g_z"):
        grads = {n: torch.empty_like(g["x"]) for n in ("g_x", "g_f", "g_i", "g_z")}
        grads[k] = x
        sgr.gated_scan_backward(g["x"], g["f"], saved, g["go"], grad_state=g["gstate"],
                                grads=grads, **kw)
        close(x, ref.gated(p)[k], k)
    check(g, p, near)


def test_captured_graph_replays():
    """A training pass and a token's step in a graph, replayed on new values with eager
    work between."""
    g, _ = problem(17, 1030, 1, 70, "bf16", True, True, [1000], "time")
    tok, _ = problem(18, 1, 4, 70, "bf16", True, True, None, "time")

    def work():
        out, state, grads = run(g)
        o, s = sgr.gated_scan_step(tok["state0"], tok["x"][0], tok["f"][0], tok["i"][0],
                                   tok["z"][0], new_state=torch.empty_like(tok["state0"]))
        return [out, state, *grads.values(), o, s]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(4):
        g["x"].copy_(torch.nan_to_num(g["x"]) * 0.5 + 0.1 * k)
        tok["x"].mul_(0.7)
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), k


def test_autograd_in_a_captured_graph():
    """Gradients asked for within a capture, of windows that wait for one another."""
    g, _ = problem(20, 700, 2, 70, "bf16", True, True, None, "time")
    leaves = [g[k].requires_grad_() for k in ("x", "f", "i", "z", "f_bias", "i_bias", "state0")]

    def work():
        out, state = sgr.gated_scan(*leaves)
        return torch.autograd.grad([out, state], leaves, [g["go"], g["gstate"]])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(3):
        with torch.no_grad():
            g["x"].mul_(0.5).add_(0.1 * k)
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        assert all(map(torch.equal, held, want)), k


def test_binding_refusals():
    g, _ = problem(19, 5, 2, 8, "fp32", True, True, None, "time")
    x, f = g["x"], g["f"]
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(x=x[0]), dict(f=f[:4]),
                dict(f=f.half()), dict(i=f[:, :, :4]), dict(z=f.transpose(1, 2)),
                dict(f_bias=g["f_bias"][:4]), dict(f_bias=g["f_bias"].double()),
                dict(i_bias=g["i_bias"]), dict(state0=g["state0"].t()),
                dict(lengths=torch.ones(2, dtype=torch.int64, device="cuda")),
                dict(out=torch.empty(5, 2, 9, device="cuda")), dict(saved=g["f_bias"]),
                dict(out=x[:1].expand(5, 2, 8))):
        with pytest.raises((TypeError, ValueError, sgr.CkError)):
            sgr.gated_scan_forward(**{**dict(x=x, f=f), **bad})
    with pytest.raises(ValueError):
        sgr.gated_scan_backward(x, f, None, g["go"])
    with pytest.raises(ValueError):
        sgr.gated_scan_step(None, x[0], f[0])
