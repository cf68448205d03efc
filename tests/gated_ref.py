"""Plain fp64 NumPy definition of the gated scan and its gradients, with a running
bound on the error of a 32-bit evaluation.

The bound follows each value through the formulas (U = 2^-24, half a step of
fp32).  v is a gate's argument; its sum with the bias is rounded (|v| U), its
exponent twice (1.3 |v| U), exponential, sum, reciprocal and product 4 U more:

    the logistic function of -|v|   (5 + 2.4 |v|) U of its value, and 2^-126 (the
                                    hardware's exponential goes no lower)
    that of |v|                     6 U of its value

A step's decay multiplies what was there by the smaller of a and q = 1 - a, with
that error, and rounds twice; magnitudes are sums of absolute terms, so that they
also cover states that are folded from parts.  Folding passes a term through the
products of the decays instead of the decays, and rounds twice a tile of eight
steps: less than as much again, so every bound is doubled.
"""
from __future__ import annotations

import numpy as np

from sequence_ref import U32, sigmoid, valid


def _gate(v):
    """(s(v), s(-v), error of s(v), error of the smaller of the two)."""
    s, o = sigmoid(v), sigmoid(-v)
    small = np.minimum(s, o)
    e_small = small * (5 + 2.4 * np.abs(v)) * U32 + 2.0 ** -126
    return s, o, np.where(v < 0, e_small, 6 * U32 * s), e_small


def gated(p):
    """{name: (value, error bound)}; p: x, f, i, z (or None) [T, B, D], f_bias, i_bias,
    state0 (or None), lengths, and for the gradients go, gstate."""
    x, f = p["x"], p["f"]
    T, B, D = x.shape
    ok = valid(T, B, p.get("lengths"))[..., None]
    cut = lambda a: np.where(ok, a, 0.0)
    x, f = cut(x), cut(f)
    bias = lambda b: 0.0 if b is None else b
    a, q, _, e_decay = _gate(f + bias(p.get("f_bias")))
    e_q = np.where(f + bias(p.get("f_bias")) > 0, e_decay, 6 * U32 * q)
    a, q, e_decay, e_q = np.where(ok, a, 1.0), cut(q), cut(e_decay), cut(e_q)
    own = p.get("i") is not None
    if own:
        g, g_o, e_g, e_gi = _gate(cut(p["i"]) + bias(p.get("i_bias")))
        g, g_o, e_g, e_gi = cut(g), cut(g_o), cut(e_g), cut(e_gi)
    else:
        g, e_g = q, e_q
    u, e_u = g * x, np.abs(x) * (e_g + U32 * g)
    h = np.zeros((B, D)) if p.get("state0") is None else p["state0"]
    mag, err = np.abs(h), np.zeros((B, D))
    hs, mags, errs = [h], [mag], [err]
    for t in range(T):
        h = a[t] * h + u[t]
        err = a[t] * err + mag * e_decay[t] + e_u[t]
        mag = a[t] * mag + np.abs(u[t])
        err = err + 3 * U32 * np.where(ok[t], mag, 0.0)
        hs.append(h), mags.append(mag), errs.append(err)
    hs, mags, errs = np.array(hs), np.array(mags), np.array(errs)
    if p.get("z") is not None:
        z = cut(p["z"])
        s = sigmoid(z)
        e_s = s * (4 + 1.3 * np.abs(z)) * U32
        gate, e_gate = z * s, np.abs(z) * (e_s + U32 * s)
        slope = s * (1 + z * (1 - s))
        e_slope = (1 + np.abs(z)) * (2 * e_s + 4 * U32 * s)
    else:
        gate, e_gate = np.ones_like(x), np.zeros_like(x)
    res = {"out": (cut(hs[1:] * gate),
                   cut(errs[1:] * np.abs(gate) + mags[1:] * (e_gate + U32 * np.abs(gate)))),
           "state": (hs[T], errs[T])}
    if "go" in p:
        go = cut(p["go"])
        y = go * gate
        e_y = np.abs(go) * (e_gate + U32 * np.abs(gate))
        c, e_c = p["gstate"], np.zeros((B, D))
        m_c = np.abs(c)
        gx, gf, gi = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
        ex, ef, ei = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
        for t in range(T - 1, -1, -1):
            gh, m = y[t] + c, np.abs(y[t]) + m_c
            e = e_y[t] + e_c + U32 * m
            before, m_b, e_b = hs[t], mags[t], errs[t]
            if not own:
                before, m_b = before - x[t], m_b + np.abs(x[t])
            gx[t], ex[t] = g[t] * gh, g[t] * e + m * (e_g[t] + U32 * g[t])
            aq = a[t] * q[t]
            e_aq = e_decay[t] + 9 * U32 * aq
            gf[t] = gh * before * aq
            ef[t] = aq * (e * m_b + m * (e_b + 3 * U32 * m_b)) + m * m_b * e_aq
            if own:
                gg = g[t] * g_o[t]
                e_gg = e_gi[t] + 9 * U32 * gg
                gi[t] = gh * x[t] * gg
                ei[t] = np.abs(x[t]) * (e * gg + m * (e_gg + 3 * U32 * gg))
            c, e_c = a[t] * gh, a[t] * e + m * e_decay[t] + np.where(ok[t], 3 * U32 * a[t] * m, 0.0)
            m_c = a[t] * m
        gx, gf, gi, ex, ef, ei = (cut(v) for v in (gx, gf, gi, ex, ef, ei))
        res.update(g_x=(gx, ex), g_f=(gf, ef), g_state0=(c, e_c))
        # added up along the steps, then over slots, chunks and rows
        adds = (T + 64 + 33 * B) * U32
        total = lambda v, e: (v.sum((0, 1)), e.sum((0, 1)) + adds * np.abs(v).sum((0, 1)))
        res["g_f_bias"] = total(gf, ef)
        if own:
            res.update(g_i=(gi, ei), g_i_bias=total(gi, ei))
        if p.get("z") is not None:
            res["g_z"] = (go * hs[1:] * slope,
                          np.abs(go) * (np.abs(slope) * errs[1:] +
                                        mags[1:] * (e_slope + 3 * U32 * np.abs(slope))))
    return {k: (v, 2 * e) for k, (v, e) in res.items()}
