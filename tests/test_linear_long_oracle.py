"""linear_long.py against the row-by-row oracle, and what its bounds refuse (CPU)."""
import numpy as np
import pytest
import torch

import linear_long as ll
from oracle import linear as ol


def data(rows, heads, dk, dv, fast, seed=0):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    t = (n((rows, heads, dk)), n((rows, heads, dk)), n((rows, heads, dv)), -fast * rng.random((rows, heads)) ** 3,
         n((heads, dk, dv)), 0.5, n((rows, heads, dv)), n((heads, dk, dv)))
    return tuple(torch.from_numpy(x) if isinstance(x, np.ndarray) else x for x in t)


@pytest.mark.parametrize("rows", [1, 2, 64, 65, 200])
def test_it_is_the_recurrence(rows):
    q, k, v, g, S0, scale, d_o, d_state = a = data(rows, 3, 5, 7, 1.0)
    o, S = ll.attend(q, k, v, g, S0, scale)
    ref, last = ol.attend(q, k, v, g, [(0, rows)], S0[None], scale)
    np.testing.assert_allclose(o, ref, rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(S, last[0], rtol=1e-11, atol=1e-11)
    want = ol.attend_backward(q, k, v, g, [(0, rows)], S0[None], scale, d_o, d_state[None])
    for name, t in zip(("dq", "dk", "dv", "dg", "d_state0"), ll.gradients(*a)):
        np.testing.assert_allclose(t, want[name][0] if name == "d_state0" else want[name], rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("rows", [150, 3000])
def test_a_wrong_gradient_of_the_decays_is_beyond_the_bound(rows, whole):
    """Three times the error to expect is below what zeros, the other sign, a row
    left out of the sums, or a part of the end's share would make."""
    q, k, v, g, S0, scale, d_o, d_state = a = data(rows, 4, 8, 8, 0.1)
    dq, dk, dv, dg, _ = ll.gradients(*a)
    _, _, dq2, dk2, _, _ = ll.squares(*a)
    err = ll.dg_error(q, k, dq2, dk2, ll.slack(8, 8, rows), whole)
    bound = 3 * (err if whole else (err ** 2).sum(0).sqrt())
    at, size = rows // 2, (lambda t: t.sum(0).abs()) if whole else (lambda t: (t ** 2).sum(0).sqrt())
    missing = torch.where(torch.arange(rows)[:, None] <= at, ((q * dq).sum(-1) - (k * dk).sum(-1))[at], 0.0)
    assert (size(dg) > bound).all() and (size(2 * dg) > bound).all() and (size(missing) > bound).all()
    assert (size(torch.ones_like(dg) * 0.02 * dg[-1].abs()) > bound).all()
