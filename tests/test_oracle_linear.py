"""Pins of oracle/linear.py (CPU): closed forms, and its gradients against
differences of its forward passes."""
import numpy as np
import pytest

from oracle import linear as ol


def test_without_decay_a_state_is_a_sum_and_with_full_decay_the_last_row():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 1, 3)), rng.standard_normal((5, 1, 3)), rng.standard_normal((5, 2, 4))
    zero = np.zeros((1, 2, 3, 4))
    o, S = ol.attend(q, k, v, np.zeros((5, 2)), [(0, 5)], zero, 0.5)
    for h in range(2):
        np.testing.assert_allclose(S[0, h], k[:, 0].T @ v[:, h], rtol=1e-13)
        np.testing.assert_allclose(o[:, h], 0.5 * np.tril(q[:, 0] @ k[:, 0].T) @ v[:, h], rtol=1e-12)
    o, S = ol.attend(q, k, v, np.full((5, 2), -np.inf), [(0, 5)], zero + 3.0, 1.0)
    np.testing.assert_allclose(S[0, 1], np.outer(k[4, 0], v[4, 1]), rtol=1e-13)
    np.testing.assert_allclose(o[2, 0], (q[2, 0] @ k[2, 0]) * v[2, 0], rtol=1e-12)


def test_decays_multiply_and_sequences_do_not_meet():
    g = np.log([[0.5], [0.25], [0.125]])
    one = np.ones((3, 1, 1))
    o, S = ol.attend(one, one, one, g, [(0, 2), None, (2, 3)], np.full((3, 1, 1, 1), 8.0), 1.0)
    np.testing.assert_allclose(o[:, 0, 0], [8 * 0.5 + 1, (8 * 0.5 + 1) * 0.25 + 1, 8 * 0.125 + 1])
    assert S[1, 0, 0, 0] == 8.0
    o, _ = ol.attend(one, one, one, g, [(0, 2), None], np.zeros((2, 1, 1, 1)), 1.0)
    assert np.isnan(o[2]).all()


def _differences(f, x, at, step=1e-5):
    out = []
    for i in at:
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out.append((f(hi) - f(lo)) / (2 * step))
    return np.array(out)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "s0"])
def test_gradients_are_differences(name):
    rng = np.random.default_rng(1)
    rows, hk, hv, dk, dv, spans = 9, 2, 4, 3, 5, [(0, 4), (4, 4), (4, 9)]
    t = {"q": rng.standard_normal((rows, hk, dk)), "k": rng.standard_normal((rows, hk, dk)),
         "v": rng.standard_normal((rows, hv, dv)), "g": -rng.random((rows, hv)), "s0": rng.standard_normal((3, hv, dk, dv))}
    d_o, d_state = rng.standard_normal((rows, hv, dv)), rng.standard_normal((3, hv, dk, dv))

    def loss(x):
        a = {**t, name: x}
        o, S = ol.attend(a["q"], a["k"], a["v"], a["g"], spans, a["s0"], 0.7)
        return (o * d_o).sum() + (S * d_state).sum()

    got = ol.attend_backward(t["q"], t["k"], t["v"], t["g"], spans, t["s0"], 0.7, d_o, d_state)
    grad = got["d_state0" if name == "s0" else "d" + name]
    at = [tuple(rng.integers(0, n) for n in grad.shape) for _ in range(12)]
    np.testing.assert_allclose([grad[i] for i in at], _differences(loss, t[name], at), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_rotation(norm, pairs):
    rng = np.random.default_rng(2)
    x, w, pos, f = rng.standard_normal((4, 3, 10)), 1 + rng.random(10), np.array([0, 1, 7, -3]), np.array([1.0, 0.3, 0.01])
    args = (pos, f, 6, norm, pairs, 1e-3)
    y = ol.rotate(x, w, *args)
    size = np.sqrt((x * x).sum(-1, keepdims=True) / (10 if norm == "rms" else 1) + 1e-3)
    np.testing.assert_allclose(y[0], (x / size * w)[0])  # position 0
    np.testing.assert_allclose((y * y).sum(-1), ((x / size * w) ** 2).sum(-1))  # a rotation
    a, b = (0, 3) if pairs == "halves" else (0, 1)
    n = (x / size * w)[1]
    np.testing.assert_allclose(y[1][:, a], n[:, a] * np.cos(1.0) - n[:, b] * np.sin(1.0))
    dy = rng.standard_normal(x.shape)
    dx, dw = ol.rotate_backward(x, w, *args, dy)
    at = [(0, 0, 1), (1, 2, 9), (2, 1, 0), (3, 0, 5)]
    np.testing.assert_allclose([dx[i] for i in at], _differences(lambda v: (ol.rotate(v, w, *args) * dy).sum(), x, at),
                               rtol=1e-6, atol=1e-8)
    at = [(0,), (4,), (9,)]
    np.testing.assert_allclose([dw[i] for i in at], _differences(lambda v: (ol.rotate(x, v, *args) * dy).sum(), w, at),
                               rtol=1e-6, atol=1e-8)


def test_8_bit_entries():
    v = np.array([[127.0, -63.5, 0.49, 0.5, 1.5, 0.0] + [0.0] * 58 + [2.0 ** -101, 3.0], [0.0] * 64 + [np.inf, 1.0]], np.float32)
    n, s, x = ol.cached(v)
    assert s[0, 0] == 1.0 and list(n[0, :6]) == [127, -64, 0, 0, 2, 0]  # ties to even
    assert s[0, 1] == np.float32(3.0) / np.float32(127.0) and n[0, 65] == 127 and n[0, 64] == 0
    assert s[1, 0] == 0.0 and np.isnan(s[1, 1]) and np.isnan(x[1, 64:]).all() and (x[1, :64] == 0).all()
    top = np.finfo(np.float32).max
    n, s, x = ol.cached(np.array([[top, -top]], np.float32))
    assert np.isfinite(s * np.float32(127)).all() and np.isfinite(x).all()
    assert (ol.cached(np.full((1, 3), 2.0 ** -101))[1] == 0).all()
