"""Linear attention with a decay for each head, its backward pass, the head
norms with the rotation by position, and 8-bit state entries, in plain float64
numpy, row by row.

TEST INFRASTRUCTURE ONLY.  Written from the formulas of include/gdn_linear.h;
shares no code with the HIP path.  Sequences are given as (first row, end row)
over packed rows, None for a skipped one, whose rows are left at the fill value.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, g, spans, s0, scale, fill=np.nan):
    """q, k [rows][h_k][d_k], v [rows][h_v][d_v], g [rows][h_v], s0
    [n][h_v][d_k][d_v].  Returns (o, final states)."""
    q, k, v, g, s0 = (np.asarray(t, np.float64) for t in (q, k, v, g, s0))
    per = v.shape[1] // q.shape[1]
    o, last = np.full(v.shape, fill), s0.copy()
    for s, span in enumerate(spans):
        if span is None:
            continue
        S = s0[s].copy()
        for r in range(*span):
            qr, kr = np.repeat(q[r], per, 0), np.repeat(k[r], per, 0)
            S = np.exp(g[r])[:, None, None] * S + kr[:, :, None] * v[r][:, None, :]
            o[r] = scale * np.einsum("hk,hkv->hv", qr, S)
        last[s] = S
    return o, last


def attend_backward(q, k, v, g, spans, s0, scale, d_o, d_state, init=None, fill=np.nan):
    """A dict of dq, dk, dv, dg ([rows][h_v]) and d_state0; init[s] false: that
    sequence's d_state0 is zero."""
    q, k, v, g, s0, d_o, d_state = (np.asarray(t, np.float64) for t in (q, k, v, g, s0, d_o, d_state))
    per = v.shape[1] // q.shape[1]
    out = {"dq": np.full(q.shape, fill), "dk": np.full(k.shape, fill), "dv": np.full(v.shape, fill),
           "dg": np.full(g.shape, fill), "d_state0": np.zeros(d_state.shape)}
    group = lambda t: t.reshape(q.shape[1], per, -1).sum(1)  # noqa: E731
    for s, span in enumerate(spans):
        if span is None:
            continue
        states, S = [], s0[s].copy()
        for r in range(*span):
            states.append(S)
            kr = np.repeat(k[r], per, 0)
            S = np.exp(g[r])[:, None, None] * S + kr[:, :, None] * v[r][:, None, :]
        after, E = S, d_state[s].copy()
        for r in range(span[1] - 1, span[0] - 1, -1):
            before = states[r - span[0]]
            qr, kr = np.repeat(q[r], per, 0), np.repeat(k[r], per, 0)
            out["dq"][r] = group(scale * np.einsum("hkv,hv->hk", after, d_o[r]))
            E = E + scale * qr[:, :, None] * d_o[r][:, None, :]
            out["dk"][r] = group(np.einsum("hkv,hv->hk", E, v[r]))
            out["dv"][r] = np.einsum("hkv,hk->hv", E, kr)
            e = np.exp(g[r])
            out["dg"][r] = e * (before * E).sum((1, 2))
            E = e[:, None, None] * E
            after = before
        out["d_state0"][s] = E if init is None or init[s] or span[0] == span[1] else 0.0
    return out


def _pairs(rot, pairs):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if pairs == "neighbours" else (i, i + rot // 2)


def _turn(x, angle, rot, pairs, back=False):
    a, b = _pairs(rot, pairs)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1 if back else 1)
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def _size(x, norm, eps):
    ss = (x * x).sum(-1, keepdims=True)
    return np.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)


def rotate(x, w, pos, inv_freq, rot, norm, pairs, eps):
    """x [rows][heads][d], w [d]."""
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    return _turn(x / _size(x, norm, eps) * w, angle, rot, pairs)


def rotate_backward(x, w, pos, inv_freq, rot, norm, pairs, eps, dy):
    """(dx, dw)"""
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    dn, size = _turn(dy, angle, rot, pairs, back=True), _size(x, norm, eps)
    unit, over = x / size, x.shape[-1] if norm == "rms" else 1
    along = (dn * w * unit).sum(-1, keepdims=True) / over
    return (dn * w - unit * along) / size, (dn * unit).sum((0, 1))


def cached(v, cols=64):
    """The values that an 8-bit entry holds of states [..., d_v] (fp32 or
    narrower), as (integers, scales, values)."""
    v = np.asarray(v, np.float64)
    per = -(-v.shape[-1] // cols)
    ints, scales = np.zeros(v.shape), np.zeros(v.shape[:-1] + (per,), np.float32)
    values = np.zeros(v.shape)
    for b in range(per):
        w = v[..., b * cols:(b + 1) * cols]
        m = np.abs(w).max(-1, keepdims=True)
        fine = np.isfinite(w).all(-1, keepdims=True)
        live = fine & (m >= 2.0 ** -100)
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            up = np.where(live, np.float32(127.0) / m.astype(np.float32), np.float32(0)).astype(np.float32)
            sc = np.where(live, m.astype(np.float32) / np.float32(127.0), np.float32(0)).astype(np.float32)
            sc = np.where(np.isfinite(sc * np.float32(127)), sc, np.nextafter(sc, np.float32(0)))
            sc = np.where(fine, sc, np.float32("nan"))
            n = np.where(live, np.rint(np.where(fine, w, 0.0) * up.astype(np.float64)), 0.0)
        ints[..., b * cols:(b + 1) * cols] = n
        scales[..., b] = sc[..., 0]
        values[..., b * cols:(b + 1) * cols] = n * sc.astype(np.float64)
    return ints, scales, values
