"""Linear attention and the rotation at their edges: what is not finite in a
backward pass, heads near the ends of the number range, batches with bad bounds
cut into segments, strides that repeat a row."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
from linear_util import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("hk,hv", [(1, 2), (2, 2)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [150, 700])
def test_what_is_not_finite_shows_in_the_gradients(rows, act, hk, hv, with_dg):
    """An input that is not finite leaves its column of the gradients that it
    enters as a row not finite from its row on (dq), or up to it (dk, dv), asked
    for the decays' gradient or not, one value head to a key head or two."""
    at = 100
    for name, out, rest in (("k", "dq", slice(at, rows)), ("q", "dk", slice(0, at + 1)), ("d_o", "dv", slice(0, at + 1))):
        c = Case([rows, 20], hk=hk, hv=hv, act=act)
        clean = c.backward(with_dg=with_dg)
        c.t[name][at, 5] = float("nan")
        got = c.backward(with_dg=with_dg)
        assert not torch.isfinite(getattr(got, out)[rest, 5]).any(), (name, out)
        for a, b in zip(got[:3], clean[:3]):
            assert torch.equal(a[rows:], b[rows:])
