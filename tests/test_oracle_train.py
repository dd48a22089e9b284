"""CPU pins of oracle/train.py: its gradients against central differences of
its own forward functions, the 8-bit form's error and its edge cases."""
import numpy as np

import oracle.train as ora

SPANS = [(2, 9), None, (12, 12), (12, 13), (13, 30)]
N, C = 33, 5


def _inputs(seed=0):
    r = np.random.default_rng(seed)
    f = lambda *s: r.standard_normal(s)
    return dict(x=f(N, C), a=f(N, C), b=f(N, C), a_log=np.log(r.uniform(1, 16, C)), dt_bias=f(C) - 2.0,
                h0=f(len(SPANS), C)), f(N, C), f(len(SPANS), C), r


def test_scan_gradients_are_those_of_differences():
    inp, dh, ds, r = _inputs()

    def value(**v):
        h, last, _ = ora.scan(v["x"], v["a"], v["b"], v["a_log"], v["dt_bias"], SPANS, v["h0"])
        live = [s for s, sp in enumerate(SPANS) if sp]
        return np.nansum(h * dh) + (last[live] * ds[live]).sum()

    before = ora.scan(inp["x"], inp["a"], inp["b"], inp["a_log"], inp["dt_bias"], SPANS, inp["h0"])[2]
    g = ora.scan_backward(inp["x"], inp["a"], inp["b"], inp["a_log"], inp["dt_bias"], SPANS, before, dh, ds)
    for k, name in (("x", "dx"), ("a", "da"), ("b", "db"), ("a_log", "d_a_log"), ("dt_bias", "d_dt_bias"),
                    ("h0", "d_state0")):
        step = r.standard_normal(inp[k].shape)
        e = 1e-6
        num = (value(**{**inp, k: inp[k] + e * step}) - value(**{**inp, k: inp[k] - e * step})) / (2 * e)
        assert abs(np.nansum(g[name] * step) - num) <= 1e-7 * (1 + abs(num)), name


def test_conv_gradients_are_those_of_differences():
    r = np.random.default_rng(1)
    w, x, dy = r.standard_normal((C, 4)), r.standard_normal((N, C)), r.standard_normal((N, C))
    win, dwin = r.standard_normal((len(SPANS), 3, C)), r.standard_normal((len(SPANS), 3, C))
    live = [s for s, sp in enumerate(SPANS) if sp]
    for act in (True, False):
        def value(w, x, win):
            y, roll = ora.conv_forward(w, x, SPANS, win, act)
            return (y * dy).sum() + (roll[live] * dwin[live]).sum()

        g = ora.conv_backward(w, x, dy, SPANS, win, dwin, act)
        for k, (v, name) in enumerate(((w, "d_conv_w"), (x, "dx"), (win, "d_window0"))):
            step, e = r.standard_normal(v.shape), 1e-6
            at = [w, x, win]
            up, down = ([u + s * e * step if i == k else u for i, u in enumerate(at)] for s in (1, -1))
            num = (value(*up) - value(*down)) / (2 * e)
            assert abs(np.nansum(g[name] * step) - num) <= 1e-7 * (1 + abs(num)), (act, name)


def test_the_8_bit_form():
    r = np.random.default_rng(2)
    v = r.standard_normal((37, 7)).astype(np.float32)
    owned = np.ones(37, bool)
    owned[20:25] = False
    s = ora.stored(v, owned)
    _, scale = ora.quantise(v, owned)
    assert (s[~owned] == 0).all()
    err = np.abs(s - v)[owned]
    assert err.max() <= 0.5 * scale.max() * (1 + 1e-6)  # half a step of the largest block
    v[:16, :4] = 1e-37
    v[16, 4] = np.inf
    s = ora.stored(v, np.ones(37, bool))
    assert (s[:16, :4] == 0).all() and np.isnan(s[16:32, 4:]).all() and np.isfinite(s[32:]).all()


def test_states_rebuilt_from_exact_values_are_the_states():
    inp, _, _, _ = _inputs(3)
    a = (inp["x"], inp["a"], inp["b"], inp["a_log"], inp["dt_bias"], SPANS)
    before = ora.scan(*a, inp["h0"])[2]
    np.testing.assert_allclose(ora.rebuilt(*a, before, block=8), before, rtol=1e-13)
