"""Linear attention and the rotation at their edges: what is not finite in a
backward pass, heads near the ends of the number range, batches with bad bounds
cut into segments, strides that repeat a row."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
import test_gpu_rotate
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


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("shape", [dict(act="f32"), dict(), dict(act="f32", d=80, rot=36, pad=1), dict(d=250, rot=64, norm="l2"), dict(d=256, rot=256, norm="l2", act="f32")],
                         ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()) or "plain")
def test_heads_whose_squares_are_out_of_range(shape, eps):
    """The norm of a head is a number wherever the head's values are: rows times
    2^-100 to 2^120, gradients too, within the bounds of rows near 1."""
    g = gdn()
    c = test_gpu_rotate.Case(9, eps=eps, **shape)
    times = torch.tensor([2.0 ** e for e in (120, 100, 64, 60, 0, -45, -52, -70, -100)], device=DEV)[:, None]
    for t in ("q", "k"):
        c.x[t].copy_((c.x[t].float() * times).to(c.x[t].dtype))
    c.check(*g.gdnl_rotate_forward(*c.args()))
    c.check_backward(g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"]))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_heads_of_the_largest_and_the_smallest_numbers(act):
    """A head of 64 values m and -m has the root mean square m: 1 and -1 come out."""
    g = gdn()
    dt = torch.float32 if act == "f32" else torch.bfloat16
    dims = g.RotateDims(2, 0, 64, 0, act_dtype=act, eps=0.0)
    sign = torch.where(torch.arange(128, device=DEV) % 3 == 0, -1.0, 1.0)
    m = torch.tensor([torch.finfo(dt).max, torch.finfo(dt).tiny, 2.0 ** -133, 2.0 ** 61], device=DEV)[:, None]
    q = (sign * m).to(dt)
    y, _ = g.gdnl_rotate_forward(dims, q, q[:, :0], None, None, None, None)
    # the squares' sum, the root and two products: within 32 half steps of fp32
    assert (y.float() - sign).abs().max() <= (32 * 2.0 ** -24 if act == "f32" else 2.0 ** -8)
    none = torch.zeros(1, 128, dtype=dt, device=DEV)
    y, _ = g.gdnl_rotate_forward(g.RotateDims(2, 0, 64, 0, act_dtype=act, eps=1e-42), none, none[:, :0], None, None, None, None)
    assert (y == 0).all()


@pytest.mark.parametrize("d_state", [True, False])
@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("with_d_state0", [True, False])
def test_workspace_of_exactly_what_a_call_asks_for(d_state, with_dg, with_d_state0):
    """Each combination within its own size, filled with NaN, gives the bits of a
    call with room for any; half of what 128 rows need is refused."""
    g = gdn()
    c = Case([700, 0, 300, 70], hk=1, hv=2, dk=16, dv=24, act="bf16", fast=0.1)
    size = g.gdnl_attend_workspace_bytes(c.dims, c.n, c.rows, True, (with_dg, d_state, with_d_state0))
    most = g.gdnl_attend_workspace_bytes(c.dims, c.n, c.rows, True)
    assert size <= most

    def run(n_bytes):
        ws = torch.full((n_bytes + 256,), 255, dtype=torch.uint8, device=DEV)
        out = g.LinearGrads(*(torch.zeros_like(c.t[t]) for t in "qkv"), torch.zeros(c.rows, c.hv, device=DEV) if with_dg else None,
                            torch.zeros(c.n, c.hv, c.dk, c.dv, device=DEV) if with_d_state0 else None)
        g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"],
                               d_state=torch.from_numpy(c.d_state).to(DEV) if d_state else None, out=out, workspace=ws[:n_bytes])
        torch.cuda.synchronize()
        assert (ws[n_bytes:] == 255).all()
        return out

    for a, b in zip(run(size), run(most)):
        assert (a is None and b is None) or torch.equal(a, b)
    small = g.gdnl_attend_workspace_bytes(c.dims, c.n, 128, True, (with_dg, d_state, with_d_state0))
    with pytest.raises(g.GdnError):
        run(small // 2)


def test_decays_of_one_row_expanded_over_all():
    """A g [rows][heads] whose rows are one and the same memory has a gradient for every row."""
    g = gdn()
    c = Case([70, 3], decay="head", act="bf16", fast=0.1)
    one, rows = c.g, c.g.expand(c.rows, c.hv)
    want = {}
    for gates in (rows.contiguous(), rows):
        o = g.gdnl_attend_forward(c.dims, c.t["q"], c.t["k"], c.t["v"], gates, c.batch, g.StatePool(c.s0.to(DEV)))
        d = g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], gates, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"])
        assert d.dg.shape == (c.rows, c.hv)
        for n, t in {"o": o, **d._asdict()}.items():
            assert torch.equal(want.setdefault(n, t), t), n
    summed = g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], one, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"]).dg
    # the sum of rows rounded one by one: half a step each
    assert ((want["dg"].double().sum(0) - summed.double()).abs() <= 2.0 ** -24 * (want["dg"].double().abs().sum(0) + summed.double().abs())).all()
