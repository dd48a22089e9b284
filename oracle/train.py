"""The vector-state gated recurrence, its backward pass, its 8-bit form and
the conv's backward pass in plain float64 numpy, row by row.

TEST INFRASTRUCTURE ONLY.  Written from the formulas of include/gdn_train.h;
shares no code with the HIP path.  Sequences are given as lists of lengths
over packed rows; a page of None is a padding sequence, whose rows are left
at the fill value.
"""
from __future__ import annotations

import numpy as np


def softplus(z):
    with np.errstate(invalid="ignore"):  # rows of no sequence may hold anything
        return np.logaddexp(z, 0.0)


def sigmoid(z):
    return np.exp(-softplus(-z))


def _gates(a, b, a_log, dt_bias):
    z = a + dt_bias
    return z, -np.exp(a_log) * softplus(z), sigmoid(b)


def scan(x, a, b, a_log, dt_bias, spans, h0, fill=np.nan):
    """spans: (first row, end row) of each sequence, None for a skipped one;
    h0 [n][C].  Returns (h, final states, the state before each row)."""
    x, a, b, a_log, dt_bias, h0 = (np.asarray(v, np.float64) for v in (x, a, b, a_log, dt_bias, h0))
    h, before, last = np.full(x.shape, fill), np.full(x.shape, fill), h0.copy()
    z, g, beta = _gates(a, b, a_log, dt_bias)
    for s, span in enumerate(spans):
        if span is None:
            continue
        cur = h0[s].copy()
        for r in range(*span):
            before[r] = cur
            cur = np.exp(g[r]) * cur + beta[r] * x[r]
            h[r] = cur
        last[s] = cur
    return h, last, before


def scan_backward(x, a, b, a_log, dt_bias, spans, before, dh, d_state, init=None, fill=np.nan):
    """Gradients given the state before each row.  Returns a dict; init[s]
    false: that sequence's d_state0 is zero."""
    x, a, b, a_log, dt_bias, before, dh, d_state = (
        np.asarray(v, np.float64) for v in (x, a, b, a_log, dt_bias, before, dh, d_state))
    z, g, beta = _gates(a, b, a_log, dt_bias)
    out = {k: np.full(x.shape, fill) for k in ("dx", "da", "db")}
    d0, dA, dB = np.zeros(d_state.shape), np.zeros(a_log.shape), np.zeros(a_log.shape)
    for s, span in enumerate(spans):
        if span is None:
            continue
        mu = d_state[s].copy()
        for r in range(span[1] - 1, span[0] - 1, -1):
            lam = dh[r] + mu
            mu = np.exp(g[r]) * lam
            dg = mu * before[r]
            da = -np.exp(a_log) * dg * sigmoid(z[r])
            out["dx"][r] = beta[r] * lam
            out["da"][r] = da
            out["db"][r] = lam * x[r] * beta[r] * sigmoid(-b[r])
            dA += dg * g[r]
            dB += da
        empty = span[0] == span[1]
        d0[s] = mu if empty or init is None or init[s] else 0.0
    return out | {"d_a_log": dA, "d_dt_bias": dB, "d_state0": d0}


def quantise(v, owned, rows=16, channels=4):
    """The integers and scales of the 8-bit form of fp32-representable v
    [rows][C]; owned[r]: row r belongs to a sequence (others count as 0 and
    are stored as 0)."""
    v = np.where(np.asarray(owned)[:, None], np.asarray(v, np.float64), 0.0)
    R, C = v.shape
    nb, nc = -(-R // rows), -(-C // channels)
    w = np.zeros((nb * rows, nc * channels))
    w[:R, :C] = v
    w = w.reshape(nb, rows, nc, channels)
    top = np.abs(w).max(axis=(1, 3))  # a NaN stays one
    q, scale = np.zeros(w.shape, np.int64), np.zeros((nb, nc))
    for i in range(nb):
        for j in range(nc):
            m = top[i, j]
            if not np.isfinite(m):
                scale[i, j] = np.nan
            elif m >= 2.0 ** -100:
                up = np.float64(np.float32(127.0) / np.float32(m))
                scale[i, j] = np.float32(m) / np.float32(127.0)
                q[i, :, j] = np.rint(w[i, :, j] * up)
    return q, scale


def stored(v, owned, rows=16, channels=4):
    """The values the 8-bit form of v stands for."""
    q, scale = quantise(v, owned, rows, channels)
    w = q * scale[:, None, :, None]
    R, C = np.asarray(v).shape
    return w.reshape(w.shape[0] * rows, -1)[:R, :C]


def rebuilt(x, a, b, a_log, dt_bias, spans, before, block=256):
    """The state before each row as the backward pass rebuilds it from stored
    x, a, b: `before` itself at a first row and at every multiple of block."""
    x, a, b, a_log, dt_bias, before = (np.asarray(v, np.float64) for v in (x, a, b, a_log, dt_bias, before))
    z, g, beta = _gates(a, b, a_log, dt_bias)
    out = before.copy()
    for span in spans:
        if span is None:
            continue
        for r in range(*span):
            if r > span[0] and r % block:
                out[r] = np.exp(g[r - 1]) * out[r - 1] + beta[r - 1] * x[r - 1]
    return out


def conv_backward(w, x, dy, spans, window, d_window, activation=True, init=None, fill=np.nan):
    """w [C][4], window and d_window [n][3][C]."""
    w, x, dy, window, d_window = (np.asarray(v, np.float64) for v in (w, x, dy, window, d_window))
    dx, dw, d0 = np.full(x.shape, fill), np.zeros(w.shape), np.zeros(window.shape)
    for s, span in enumerate(spans):
        if span is None:
            continue
        T = span[1] - span[0]
        have = init is None or bool(init[s])
        X = np.concatenate([window[s] if have else np.zeros_like(window[s]), x[span[0]:span[1]]])
        grad = np.zeros_like(X)
        grad[T:] += d_window[s]
        for t in range(T):
            z = sum(w[:, j] * X[t + j] for j in range(4))
            sg = sigmoid(z)
            dz = dy[span[0] + t] * (sg * (1.0 + z * (1.0 - sg)) if activation else 1.0)
            for j in range(4):
                grad[t + j] += w[:, j] * dz
                dw[:, j] += dz * X[t + j]
        dx[span[0]:span[1]] = grad[3:]
        d0[s] = grad[:3] if have or T == 0 else 0.0
    return {"dx": dx, "d_conv_w": dw, "d_window0": d0}


def conv_forward(w, x, spans, window, activation=True):
    """y and the rolled windows, for checks of the gradients by differences."""
    w, x, window = (np.asarray(v, np.float64) for v in (w, x, window))
    y, roll = np.zeros(x.shape), window.copy()
    for s, span in enumerate(spans):
        if span is None:
            continue
        X = np.concatenate([window[s], x[span[0]:span[1]]])
        T = span[1] - span[0]
        for t in range(T):
            z = sum(w[:, j] * X[t + j] for j in range(4))
            y[span[0] + t] = z * sigmoid(z) if activation else z
        roll[s] = X[T:]
    return y, roll
