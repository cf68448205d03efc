"""Plain fp64 NumPy definitions of the sequence operators, their gradients as
formulas, and the error bounds of the GPU tests.

The scan's formulas are split into the part that is linear in each of its
factors (``scan_core``) and the elementwise functions around it.  Called with
absolute values, ``scan_core`` gives for every output the sum of its terms'
magnitudes, to which rounding errors of a 32-bit evaluation are proportional.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # half a step of fp32 relative to the value


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(x, 0.0)


def valid(T, B, lengths):
    if lengths is None:
        return np.ones((T, B), bool)
    return np.arange(T)[:, None] < np.clip(lengths, 0, T)[None, :]


def cut(x, ok):
    """x with every entry of steps past its row's length replaced by 0."""
    return np.where(ok.reshape(ok.shape + (1,) * (x.ndim - 2)), x, 0.0)


def spread(x, D):
    """[T, B, G, N] -> [T, B, D, N]."""
    return np.repeat(x, D // x.shape[2], axis=2)


def scan_core(a, dt, u, Bm, Cm, D, gate, dgate, A, state0, go=None, gstate=None):
    """The scan for given decays a [T, B, D, N] and steps dt [T, B, D]; with go,
    also the gradients.  gate, dgate: silu(z) and its derivative, or None."""
    T, B, Dn = u.shape
    G = Bm.shape[2]
    bx, cx = spread(Bm, Dn), spread(Cm, Dn)
    h = state0.copy()
    hs = np.zeros((T + 1,) + h.shape)
    hs[0] = h
    for t in range(T):
        h = a[t] * h + (dt[t] * u[t])[..., None] * bx[t]
        hs[t + 1] = h
    y = (hs[1:] * cx).sum(-1) + D * u
    out = y if gate is None else y * gate
    res = {"out": out, "state": hs[T]}
    if go is None:
        return res
    gy = go if gate is None else go * gate
    g = gstate.copy()  # a_{t+1} dL/dh_{t+1}
    gu, gdt = np.zeros_like(u), np.zeros_like(u)
    gA = np.zeros_like(A)
    gB, gC = np.zeros_like(Bm), np.zeros_like(Cm)
    for t in range(T - 1, -1, -1):
        gh = cx[t] * gy[t][..., None] + g
        gC[t] = (hs[t + 1] * gy[t][..., None]).reshape(B, G, Dn // G, -1).sum(2)
        gB[t] = (gh * (dt[t] * u[t])[..., None]).reshape(B, G, Dn // G, -1).sum(2)
        gx = (gh * bx[t]).sum(-1)
        w = gh * a[t] * hs[t]
        gA += (w * dt[t][..., None]).sum(0)
        gdt[t] = (w * A).sum(-1) + u[t] * gx
        gu[t] = dt[t] * gx + D * gy[t]
        g = a[t] * gh
    res.update(g_u=gu, g_dt=gdt, g_A=gA, g_B=gB, g_C=gC, g_D=(gy * u).sum((0, 1)), g_state0=g)
    if gate is not None:
        res["g_z"] = go * y * dgate
    return res


def scan(p, magnitude=False):
    """Outputs and gradients of a scan problem (a dict of fp64 arrays: u,
    delta, A, B, C and optionally D, z, delta_bias, state0, lengths, go,
    gstate; "softplus").  magnitude=True: the sums of the terms' magnitudes."""
    T, B, Dn = p["u"].shape
    N = p["A"].shape[1]
    ok = valid(T, B, p.get("lengths"))
    none = np.zeros(Dn)
    u, Bm, Cm = (cut(p[k], ok) for k in ("u", "B", "C"))
    raw = cut(p["delta"], ok) + (p["delta_bias"] if p.get("delta_bias") is not None else none)
    dt = cut(softplus(raw) if p["softplus"] else raw, ok)
    a = np.exp(dt[..., None] * p["A"])
    A = p["A"]
    D = p["D"] if p.get("D") is not None else none
    state0 = p["state0"] if p.get("state0") is not None else np.zeros((B, Dn, N))
    gate = dgate = go = gstate = None
    if p.get("z") is not None:
        z = cut(p["z"], ok)
        s = sigmoid(z)
        # the derivative's two terms cancel near z = -1.3
        gate, dgate = cut(z * s, ok), s * (1 + (np.abs(z) if magnitude else z) * (1 - s))
    if p.get("go") is not None:
        go = cut(p["go"], ok)
        gstate = p["gstate"] if p.get("gstate") is not None else np.zeros((B, Dn, N))
    if magnitude:
        m = [None if x is None else np.abs(x)
             for x in (dt, u, Bm, Cm, D, gate, dgate, A, state0, go, gstate)]
        r = scan_core(a, *m)
    else:
        r = scan_core(a, dt, u, Bm, Cm, D, gate, dgate, A, state0, go, gstate)
    r["out"] = cut(r["out"], ok)
    if go is not None:
        gr = r.pop("g_dt") * (sigmoid(raw) if p["softplus"] else 1.0)
        r["g_delta"] = cut(gr, ok)
        r["g_delta_bias"] = r["g_delta"].sum((0, 1))
        for k in ("g_u", "g_z", "g_B", "g_C"):
            if k in r:
                r[k] = cut(r[k], ok)
    return r


def conv(p, magnitude=False):
    """Outputs and gradients of a convolution problem: x [T, B, D], weight
    [D, W], optionally bias, state0 [W - 1, B, D], lengths, gy, gstate; "silu"."""
    x, w = p["x"], p["weight"]
    T, B, D = x.shape
    W = w.shape[1]
    ok = valid(T, B, p.get("lengths"))
    lens = ok.sum(0)
    bias = p["bias"] if p.get("bias") is not None else np.zeros(D)
    s0 = p["state0"] if p.get("state0") is not None else np.zeros((W - 1, B, D))
    xe = np.concatenate([s0, cut(x, ok)])
    pre = sum((w[:, k] * xe[k:k + T] for k in range(W)), bias + np.zeros_like(x))
    dact = np.ones_like(pre)
    y = pre
    if p["silu"]:
        s = sigmoid(pre)
        y, dact = pre * s, s * (1 + pre * (1 - s))
    mag = sum((np.abs(w[:, k] * xe[k:k + T]) for k in range(W)), np.abs(bias) + np.zeros_like(x))
    state = np.stack([xe[lens + k, np.arange(B)] for k in range(W - 1)]) if W > 1 else s0
    r = {"y": cut(np.maximum(mag, np.abs(y)) if magnitude else y, ok),
         "state": np.abs(state) if magnitude else state}
    if p.get("gy") is None:
        return r
    gy = cut(p["gy"], ok)
    gs = p["gstate"] if p.get("gstate") is not None else np.zeros((W - 1, B, D))
    if magnitude:
        # |silu'| changes by at most half of the pre-activation's change
        gy, w, xe, gs = np.abs(gy), np.abs(w), np.abs(xe), np.abs(gs)
        gp = gy * (s * (1 + np.abs(pre) * (1 - s)) + 0.5 * mag if p["silu"] else 1.0)
    else:
        gp = gy * dact
    gxe = np.zeros_like(xe)
    gw = np.zeros_like(w)
    for k in range(W):
        gxe[k:k + T] += w[:, k] * gp
        gw[:, k] = (gp * xe[k:k + T]).sum((0, 1))
    for k in range(W - 1):
        gxe[lens + k, np.arange(B)] += gs[k]
    r.update(g_x=cut(gxe[W - 1:], ok), g_state0=gxe[:W - 1], g_weight=gw, g_bias=gp.sum((0, 1)))
    return r


def philox(counter, key):
    """Philox4x32-10 (Salmon et al., SC 2011) of counters [..., 4], one key."""
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, -1)


def keep(T, B, D, p, seed, offset, held):
    """(mask [T, B, D], scale) of the dropout."""
    cols, rows = -(-D // 8), B if held else T * B
    ctr = np.zeros((rows, cols, 4), np.uint64)
    ctr[..., 0] = np.arange(cols)
    ctr[..., 1] = np.arange(rows)[:, None]
    ctr[..., 2], ctr[..., 3] = offset & 0xFFFFFFFF, offset >> 32 & 0xFFFFFFFF
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    r = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, cols * 8)[:, :D]
    q = int(np.floor(65536.0 * p + 0.5))
    m = np.broadcast_to((r >= q).reshape(1 if held else T, B, D), (T, B, D))
    return m, 65536.0 / (65536 - q) if q < 65536 else 0.0
