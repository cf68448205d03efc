"""The sequence operators that stand before and behind the graph recurrence in
a text model, as measured cases: the short causal convolution, the selective
state space scan and the counter-based dropout.

Each case is one pass of one operator.  ``run`` computes it in the plain form
(elementary torch operations in 32 bits) while ``own`` is false and through
the package's entry points while it is true; ``exact`` evaluates the
definition in 64 bits.  Tensors are time first ([T, B, channels]), as the
recurrence's own drives and states are.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases

def _scan(name, op, T, B, D, N, G, dtype, gated, ragged, layout):
    return {"name": name, "op": op, "T": T, "B": B, "D": D, "N": N, "G": G, "dtype": dtype,
            "gated": gated, "ragged": ragged, "layout": layout}


def _conv(name, op, T, B, D, W, dtype, silu, ragged, layout):
    return {"name": name, "op": op, "T": T, "B": B, "D": D, "W": W, "dtype": dtype,
            "silu": silu, "ragged": ragged, "layout": layout}


def _drop(name, T, B, D, dtype, p, held, residual):
    return {"name": name, "op": "dropout_train", "T": T, "B": B, "D": D, "dtype": dtype,
            "p": p, "held": held, "residual": residual}


def listed():
    return [
        # training on the FlyGPT window (64 steps, batch 32) with a scan over
        # its 256 input channels, in the recurrence's own type
        _scan("scan_train_window", "scan_train", 64, 32, 256, 16, 1, "fp32", False, False, "time"),
        # training on long texts: gated, the gate and the input halves of one projection
        _scan("scan_train_text", "scan_train", 2048, 8, 2048, 16, 1, "bf16", True, False, "proj"),
        # training on texts of unequal length with odd sizes and several B/C groups
        _scan("scan_train_ragged", "scan_train", 777, 5, 1001, 13, 7, "fp16", True, True, "batch"),
        # one long prompt read before answering: a single row, so the time axis has to be split
        _scan("scan_prompt_long", "scan_prompt", 16384, 1, 2048, 16, 1, "bf16", True, False, "proj"),
        # a batch of prompts of unequal length
        _scan("scan_prompt_ragged", "scan_prompt", 1023, 16, 1024, 16, 2, "bf16", True, True, "time"),
        # answering, one token for one text: the smallest call
        _scan("scan_token_one", "scan_token", 1, 1, 256, 16, 1, "bf16", True, False, "proj"),
        # answering, one token for each of many texts
        _scan("scan_token_many", "scan_token", 1, 256, 2048, 16, 1, "bf16", True, False, "proj"),
        # the convolution before the scan of scan_train_text
        _conv("conv_train_text", "conv_train", 2048, 8, 2048, 4, "bf16", True, False, "proj"),
        # the convolution over prompts of unequal length, odd channels
        _conv("conv_prompt_ragged", "conv_prompt", 1023, 16, 1025, 4, "fp16", True, True, "batch"),
        # the convolution for one token of each of many texts
        _conv("conv_token_many", "conv_token", 1, 256, 2048, 4, "bf16", True, False, "proj"),
        # dropout of the recurrence's states, one mask for the whole FlyGPT window
        _drop("dropout_states_held", 64, 32, 5000, "fp32", 0.2, True, False),
        # dropout of the scan's output in front of the residual sum
        _drop("dropout_text", 2048, 8, 2048, "bf16", 0.1, False, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_train", "scan_train", "scan_prompt", "scan_prompt", "scan_token",
                     "conv_train", "conv_prompt", "conv_token", "dropout_train"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    layout = rng.choice(["time", "batch", "proj"])
    flag, ragged = rng.random() < 0.5, rng.random() < 0.4
    D = _log_int(rng, 64, 2048)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    if op.endswith("token"):
        T, B, ragged = 1, _log_int(rng, 1, 256), False
    else:
        T = _log_int(rng, 33, 16384 if op == "scan_prompt" else 2048)
        # the listed cases' largest sizes bound a draw's positions
        B = _log_int(rng, 1, max(1, min(64, 2048 * 8 * 2048 // (T * D))))
    if op.startswith("scan"):
        G = rng.choice([g for g in (1, 1, 1, 2, 4, 7) if D % g == 0])
        N = rng.choice([16, 16, 16, rng.randint(1, 16), rng.randint(4, 16)])
        return _scan("", op, T, B, D, N, G, dtype, flag, ragged, layout)
    if op.startswith("conv"):
        return _conv("", op, T, B, D, rng.choice([2, 3, 4, 4]), dtype, flag, ragged, layout)
    return _drop("", T, B, D, dtype, round(rng.uniform(0.02, 0.6), 3), rng.random() < 0.5, flag)


def _lengths(case):
    """Ragged batches hold texts of evenly spread lengths, from none to all of T."""
    T, B = case["T"], case["B"]
    if not case.get("ragged"):
        return [T] * B
    return [T * b // (B - 1) for b in range(B)] if B > 1 else [T // 2]


def work(case):
    T, B, D, op = case["T"], case["B"], case["D"], case["op"]
    e = 4 if case["dtype"] == "fp32" else 2
    rows = sum(_lengths(case)) if op != "dropout_train" else T * B
    x = rows * D * e                       # one [T, B, D] tensor, as far as it holds text
    out = T * B * D * e                    # outputs are written over the whole window
    if op.startswith("scan"):
        N, G, z = case["N"], case["G"], int(case["gated"])
        bc, bc_out = rows * G * N * e, T * B * G * N * e
        state, par = B * D * N * 4, D * (N + 2) * 4
        bytes_ = (2 + z) * x + 2 * bc + out + 2 * state + par
        flops = rows * D * (7 * N + 8 + 6 * z)
        if op == "scan_train":             # the forward, then the backward with its upstream gradient
            bytes_ += (3 + z) * x + 2 * bc + (2 + z) * out + 2 * bc_out + 2 * state + 2 * par
            flops += rows * D * (20 * N + 20 + 10 * z)
        return {"bytes": bytes_, "flops": flops}
    if op.startswith("conv"):
        W, s = case["W"], int(case["silu"])
        state, par = (case["W"] - 1) * B * D * e, D * (case["W"] + 1) * 4
        bytes_ = x + out + 2 * state + par
        flops = rows * D * (2 * W + 4 * s)
        if op == "conv_train":
            bytes_ += 2 * x + out + 2 * state + 2 * par
            flops += rows * D * (6 * W + 12 * s)
        return {"bytes": bytes_, "flops": flops}
    draws = (B if case["held"] else T * B) * D
    return {"bytes": (4 + int(case["residual"])) * x, "flops": rows * D * 3 + draws * 10}


# --------------------------------------------------------------- the inputs

def _seq(g, case, dtype, halves=1, scale=1.0):
    """`halves` tensors [T, B, D] in the case's storage: time or batch outermost,
    or slices of one projection's output."""
    T, B, D = case["T"], case["B"], case["D"]

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    layout = case.get("layout", "time")
    if layout == "proj":
        full = rand(T, B, 2 * D)
        return [full[:, :, i * D:(i + 1) * D] for i in range(halves)]
    if layout == "batch":
        return [rand(B, T, D).transpose(0, 1) for _ in range(halves)]
    return [rand(T, B, D) for _ in range(halves)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, B, D, op = case["T"], case["B"], case["D"], case["op"]
    dtype = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case, "lengths": None}
    if case.get("ragged"):
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if op.startswith("scan"):
        N, G = case["N"], case["G"]
        st["u"], st["z"] = _seq(g, case, dtype, halves=2)
        if not case["gated"]:
            st["z"] = None
        st["delta"] = _seq(g, {**case, "layout": "time" if case["layout"] == "proj" else
                               case["layout"]}, dtype, scale=0.5)[0]
        bc = randn(T, B, 2 * G * N).to(dtype)      # the B and C slices of one projection
        st["Bm"] = bc[:, :, :G * N].unflatten(2, (G, N))
        st["Cm"] = bc[:, :, G * N:].unflatten(2, (G, N))
        # decay rates 1..N and time steps between 1e-3 and 0.1, as such layers start
        st["A"] = -torch.arange(1, N + 1, device="cuda").float() * \
            (1 + 0.1 * randn(D, N)).clamp(0.5, 1.5)
        dt = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        st["delta_bias"] = dt + torch.log(-torch.expm1(-dt))
        st["Dskip"] = 1 + 0.1 * randn(D)
        st["state0"] = 0.5 * randn(B, D, N)
        if op == "scan_train":
            st["grad_out"] = randn(T, B, D).to(dtype)
            st["grad_state"] = 0.1 * randn(B, D, N)
        if op == "scan_token":
            st["new_state"] = torch.empty_like(st["state0"])
    elif op.startswith("conv"):
        W = case["W"]
        st["x"] = _seq(g, case, dtype)[0]
        st["weight"] = randn(D, W) / math.sqrt(W)
        st["bias"] = 0.1 * randn(D)
        st["state0"] = randn(W - 1, B, D).to(dtype)
        if op == "conv_train":
            st["grad_out"] = randn(T, B, D).to(dtype)
            st["grad_state"] = (0.1 * randn(W - 1, B, D)).to(dtype)
        if op == "conv_token":
            st["new_state"] = torch.empty_like(st["state0"])
    else:
        st["x"] = randn(T, B, D).to(dtype)
        st["residual"] = randn(T, B, D).to(dtype) if case["residual"] else None
        st["grad_out"] = randn(T, B, D).to(dtype)
        words = torch.randint(0, 2**31 - 1, (4,), generator=g, device="cuda").tolist()
        st["seed"], st["offset"] = words[0] << 32 | words[1], words[2] << 20 | words[3]
    return st


# ----------------------------------------------------------- the plain forms

def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _valid(st, T, B):
    """[T, B, 1]: true where the text of row b still runs at step t."""
    if st["lengths"] is None:
        return None
    t = torch.arange(T, device="cuda")
    return (t[:, None] < st["lengths"][None, :]).unsqueeze(-1)


def _masked(x, valid):
    return x if valid is None else torch.where(valid, x, torch.zeros_like(x))


def _by_group(x, D):
    """[T, B, G, N] -> [T, B, D, N]: channel d reads group d * G // D."""
    T, B, G, N = x.shape
    return x.unsqueeze(3).expand(T, B, G, D // G, N).reshape(T, B, D, N)


def _plain_scan(st, train):
    case = st["case"]
    T, B, D, N, G = case["T"], case["B"], case["D"], case["N"], case["G"]
    dtype = st["u"].dtype
    valid = _valid(st, T, B)
    u = _masked(st["u"].float(), valid)
    raw = _masked(st["delta"].float(), valid) + st["delta_bias"]
    delta = _masked(_softplus(raw), valid)
    Bm = st["Bm"].float() if valid is None else _masked(st["Bm"].float(), valid.unsqueeze(-1))
    Cm = st["Cm"].float() if valid is None else _masked(st["Cm"].float(), valid.unsqueeze(-1))
    bx, cx = _by_group(Bm, D), _by_group(Cm, D)
    a = torch.exp(delta.unsqueeze(-1) * st["A"])
    hs = (delta * u).unsqueeze(-1) * bx
    h = st["state0"]
    for t in range(T):
        hs[t] += a[t] * h
        h = hs[t]
    state = h.clone()
    y = (hs * cx).sum(-1) + st["Dskip"] * u
    if st["z"] is not None:
        z = _masked(st["z"].float(), valid)
        sig = 1 / (1 + torch.exp(-z))
        out = y * z * sig
    else:
        out = y
    out = _masked(out, valid).to(dtype)
    if not train:
        return [out, state]
    go = _masked(st["grad_out"].float(), valid)
    gy = go if st["z"] is None else go * z * sig
    gh = cx * gy.unsqueeze(-1)             # becomes dL/dh_t
    gh[T - 1] += st["grad_state"]
    for t in range(T - 2, -1, -1):
        gh[t] += a[t + 1] * gh[t + 1]
    g_state0 = a[0] * gh[0]
    g_b = (gh * (delta * u).unsqueeze(-1)).view(T, B, G, D // G, N).sum(3)
    g_c = (hs * gy.unsqueeze(-1)).view(T, B, G, D // G, N).sum(3)
    g_du = (gh * bx).sum(-1)
    prev = torch.cat([st["state0"].unsqueeze(0), hs[:-1]])
    gp = gh * a * prev                     # dL/d(delta A)
    g_a = (gp * delta.unsqueeze(-1)).sum((0, 1))
    g_delta = (gp * st["A"]).sum(-1) + u * g_du
    g_u = delta * g_du + st["Dskip"] * gy
    g_raw = _masked(g_delta * (1 / (1 + torch.exp(-raw))), valid)
    grads = [_masked(g_u, valid).to(dtype), g_raw.to(dtype), g_a, g_b.to(dtype), g_c.to(dtype),
             (gy * u).sum((0, 1)), g_raw.sum((0, 1)), g_state0]
    if st["z"] is not None:
        grads.append(_masked(go * y * sig * (1 + z * (1 - sig)), valid).to(dtype))
    return [out, state] + grads


def _plain_conv(st, train):
    case = st["case"]
    T, B, D, W = case["T"], case["B"], case["D"], case["W"]
    dtype = st["x"].dtype
    valid = _valid(st, T, B)
    xe = torch.cat([st["state0"].float(), _masked(st["x"].float(), valid)])   # [W - 1 + T, B, D]
    w = st["weight"]
    pre = st["bias"].expand(T, B, D)
    for k in range(W):
        pre = pre + w[:, k] * xe[k:k + T]
    sig = 1 / (1 + torch.exp(-pre)) if case["silu"] else None
    y = _masked(pre * sig if case["silu"] else pre, valid).to(dtype)
    # the last W - 1 inputs of each row: positions len .. len + W - 2 of xe
    if st["lengths"] is None:
        state = xe[T:T + W - 1]
    else:
        at = (torch.arange(W - 1, device="cuda")[:, None] + st["lengths"][None, :]).long()
        at = at.unsqueeze(-1).expand(W - 1, B, D)
        state = torch.gather(xe, 0, at)
    state = state.to(dtype)
    if not train:
        return [y, state]
    gp = _masked(st["grad_out"].float(), valid)
    if case["silu"]:
        gp = gp * sig * (1 + pre * (1 - sig))
    gx = torch.zeros_like(xe)
    gw = torch.empty_like(w)
    for k in range(W):
        gx[k:k + T] += w[:, k] * gp
        gw[:, k] = (gp * xe[k:k + T]).sum((0, 1))
    if st["lengths"] is None:
        gx[T:T + W - 1] += st["grad_state"].float()
    else:
        gx.scatter_add_(0, at, st["grad_state"].float())
    return [y, state, _masked(gx[W - 1:], valid).to(dtype), gw, gp.sum((0, 1)),
            gx[:W - 1].to(dtype)]


def _plain_keep(case, seed, offset):
    """Keep mask [rows, D] (rows of one step if held) from the Philox4x32-10
    generator (Salmon et al., SC 2011): counter (channel / 8, row, offset),
    key seed, 16 bits a value, low half first; kept where the value is not
    below round(65536 p)."""
    rows, D = (1 if case["held"] else case["T"]) * case["B"], case["D"]
    cols = (D + 7) // 8
    m32 = 0xFFFFFFFF
    c0 = torch.arange(cols, device="cuda").expand(rows, cols)
    c1 = torch.arange(rows, device="cuda").unsqueeze(1).expand(rows, cols)
    c2 = torch.full((rows, cols), offset & m32, device="cuda")
    c3 = torch.full((rows, cols), offset >> 32 & m32, device="cuda")
    k0, k1 = seed & m32, seed >> 32 & m32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # the low 64 bits wrap, which is wanted
        c0, c1, c2, c3 = ((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32, ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    r = torch.stack([w >> s & 0xFFFF for w in (c0, c1, c2, c3) for s in (0, 16)], dim=-1)
    return r.reshape(rows, cols * 8)[:, :D] >= int(case["p"] * 65536 + 0.5)


def _plain_dropout(st):
    case, x = st["case"], st["x"]
    T, B, D = case["T"], case["B"], case["D"]
    keep = _plain_keep(case, st["seed"], st["offset"]).view(-1, B, D)
    scale = 65536.0 / (65536 - int(case["p"] * 65536 + 0.5))
    zero = torch.zeros((), device="cuda")
    out = torch.where(keep, x.float() * scale, zero)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return [out.to(x.dtype), torch.where(keep, st["grad_out"].float() * scale, zero).to(x.dtype)]


def _own(st):
    import sparse_graph_recurrent_amd as sgr

    case = st["case"]
    op = case["op"]
    if op.startswith("scan"):
        kw = dict(D=st["Dskip"], z=st["z"], delta_bias=st["delta_bias"], delta_softplus=True)
        args = (st["u"], st["delta"], st["A"], st["Bm"], st["Cm"])
        if op == "scan_token":
            u, delta, A, Bm, Cm = args
            kw["z"] = None if st["z"] is None else st["z"][0]
            out, state = sgr.selective_scan_step(st["state0"], u[0], delta[0], A, Bm[0], Cm[0],
                                                 new_state=st["new_state"], **kw)
            return [out.unsqueeze(0), state]
        kw["lengths"] = st["lengths"]
        train = op == "scan_train"
        out, state, saved, ws = sgr.selective_scan_forward(*args, state0=st["state0"], save=train,
                                                           **kw)
        if not train:
            return [out, state]
        g = sgr.selective_scan_backward(*args, saved, st["grad_out"], grad_state=st["grad_state"],
                                        **kw)
        grads = [g[k] for k in ("g_u", "g_delta", "g_A", "g_B", "g_C", "g_D", "g_delta_bias",
                                "g_state0")]
        return [out, state] + grads + ([g["g_z"]] if st["z"] is not None else [])
    if op.startswith("conv"):
        act = "silu" if case["silu"] else None
        if op == "conv_token":
            y, state = sgr.short_conv_step(st["state0"], st["x"][0], st["weight"], st["bias"],
                                           activation=act, new_state=st["new_state"])
            return [y.unsqueeze(0), state]
        kw = dict(bias=st["bias"], state0=st["state0"], lengths=st["lengths"], activation=act)
        y, state = sgr.short_conv_forward(st["x"], st["weight"], **kw)
        if op == "conv_prompt":
            return [y, state]
        g = sgr.short_conv_backward(st["x"], st["weight"], st["grad_out"],
                                    grad_state=st["grad_state"], **kw)
        return [y, state] + [g[k] for k in ("g_x", "g_weight", "g_bias", "g_state0")]
    kw = dict(p=case["p"], seed=st["seed"], offset=st["offset"], held=case["held"])
    return [sgr.dropout_forward(st["x"], residual=st["residual"], **kw),
            sgr.dropout_backward(st["grad_out"], **kw)]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op.startswith("scan"):
        return _plain_scan(state, op == "scan_train")
    if op.startswith("conv"):
        return _plain_conv(state, op == "conv_train")
    return _plain_dropout(state)


# ------------------------------------------------------- the exact definition

def _exact_scan(st, train):
    """One step after the other on [B, G, D / G, N] states; gradients by
    differentiating that program."""
    case = st["case"]
    T, B, D, N, G = case["T"], case["B"], case["D"], case["N"], case["G"]
    leaf = {k: st[k].double().contiguous().requires_grad_(train)
            for k in ("u", "delta", "A", "Bm", "Cm", "Dskip", "delta_bias", "state0")}
    if st["z"] is not None:
        leaf["z"] = st["z"].double().contiguous().requires_grad_(train)
    lens = _lengths(case)
    length = torch.tensor(lens, device="cuda").view(B, 1, 1, 1)
    A = leaf["A"].view(G, D // G, N)
    h = leaf["state0"].view(B, G, D // G, N)
    # only the steps that some row's text reaches change anything
    steps = max(lens) if lens else 0
    dt_all = torch.logaddexp(leaf["delta"] + leaf["delta_bias"],
                             torch.zeros((), dtype=torch.float64, device="cuda"))
    outs = []
    for t in range(steps):
        dt = dt_all[t].view(B, G, D // G, 1)
        u = leaf["u"][t].view(B, G, D // G)
        nxt = torch.exp(dt * A) * h + dt * u.unsqueeze(-1) * leaf["Bm"][t].unsqueeze(2)
        runs = t < length
        h = torch.where(runs, nxt, h) if case["ragged"] else nxt
        y = (h * leaf["Cm"][t].unsqueeze(2)).sum(-1) + u * leaf["Dskip"].view(G, D // G)
        outs.append(torch.where(runs.squeeze(-1), y, torch.zeros_like(y)).view(B, D))
    out = torch.stack(outs) if outs else torch.zeros(0, B, D, dtype=torch.float64, device="cuda")
    if steps < T:
        out = torch.cat([out, torch.zeros(T - steps, B, D, dtype=torch.float64, device="cuda")])
    if st["z"] is not None:
        out = out * leaf["z"] * torch.sigmoid(leaf["z"])
    state = h.view(B, D, N)
    if not train:
        return [out, state]
    order = ["u", "delta", "A", "Bm", "Cm", "Dskip", "delta_bias", "state0"]
    order += ["z"] if st["z"] is not None else []
    grads = torch.autograd.grad([out, state], [leaf[k] for k in order],
                                [st["grad_out"].double(), st["grad_state"].double()],
                                allow_unused=True)
    return [out.detach(), state.detach()] + [
        torch.zeros_like(leaf[k]) if g is None else g for k, g in zip(order, grads)]


def _exact_conv(st, train):
    """Row by row, each cut to its own length; gradients by differentiating."""
    case = st["case"]
    T, B, D, W = case["T"], case["B"], case["D"], case["W"]
    leaf = {k: st[k].double().contiguous().requires_grad_(train)
            for k in ("x", "weight", "bias", "state0")}
    ys, states = [], []
    for b, n in enumerate(_lengths(case)):
        seen = torch.cat([leaf["state0"][:, b], leaf["x"][:n, b]])
        win = torch.stack([seen[k:k + n] for k in range(W)], -1)     # [n, D, W]
        y = (win * leaf["weight"]).sum(-1) + leaf["bias"]
        if case["silu"]:
            y = y * torch.sigmoid(y)
        ys.append(torch.cat([y, torch.zeros(T - n, D, dtype=torch.float64, device="cuda")]))
        states.append(seen[n:])
    y, state = torch.stack(ys, 1), torch.stack(states, 1)
    if not train:
        return [y, state]
    grads = torch.autograd.grad([y, state], [leaf[k] for k in ("x", "weight", "bias", "state0")],
                                [st["grad_out"].double(), st["grad_state"].double()])
    return [y.detach(), state.detach()] + list(grads)


def _exact_dropout(st):
    """The mask again, in unsigned host words."""
    case = st["case"]
    T, B, D = case["T"], case["B"], case["D"]
    rows, cols = (1 if case["held"] else T) * B, -(-D // 8)
    u64 = np.uint64
    mask32, sh = u64(0xFFFFFFFF), u64(32)
    col, row = np.meshgrid(np.arange(cols, dtype=u64), np.arange(rows, dtype=u64))
    ctr = [col, row, np.full_like(col, st["offset"] & 0xFFFFFFFF), np.full_like(col, st["offset"] >> 32)]
    key = [st["seed"] & 0xFFFFFFFF, st["seed"] >> 32]
    for r in range(10):
        a, b = ctr[0] * u64(0xD2511F53), ctr[2] * u64(0xCD9E8D57)
        ctr = [(b >> sh) ^ ctr[1] ^ u64((key[0] + r * 0x9E3779B9) % 2**32), b & mask32,
               (a >> sh) ^ ctr[3] ^ u64((key[1] + r * 0xBB67AE85) % 2**32), a & mask32]
    words = np.stack(ctr, -1).astype("<u4").view("<u2").reshape(rows, cols * 8)[:, :D]
    below = int(case["p"] * 65536 + 0.5)
    keep = torch.from_numpy((words >= below).reshape(-1, B, D)).cuda()
    factor = keep.double() * 65536 / (65536 - below)
    out = st["x"].double() * factor
    if st["residual"] is not None:
        out = out + st["residual"].double()
    return [out, st["grad_out"].double() * factor]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("scan"):
        return _exact_scan(st, case["op"] == "scan_train")
    if case["op"].startswith("conv"):
        return _exact_conv(st, case["op"] == "conv_train")
    return _exact_dropout(st)
