"""Calls of include/gdn_linear.h whose history autograd would lose are refused
(host only: the refusal comes before the device's)."""
import pytest
import torch
from torch.autograd import forward_ad

from test_linear_abi import L, _host_calls  # noqa: F401

GRAD = "records nothing for autograd"


def calls():
    g, t, attend, rot, cache = _host_calls()
    back = {**attend, "d_o": t(4, 32), "d_state": t(1, 2, 8, 16)}
    turn = {**rot, "d_yq": t(4, 16), "d_yk": t(4, 8)}
    return [(g.gdnl_attend_forward, attend, ("q", "k", "v", "g", "state_in")),
            (g.gdnl_attend_backward, back, ("q", "k", "v", "g", "state_in", "d_o", "d_state")),
            (g.gdnl_rotate_forward, rot, ("q", "k", "wq", "wk")),
            (g.gdnl_rotate_backward, turn, ("q", "k", "wq", "wk", "d_yq", "d_yk")),
            (g.gdnl_cache_store, cache, ("state",)), (g.gdnl_cache_load, cache, ("state",))]


def with_(kw, name, change):
    """The call's arguments with one tensor changed, a pool's buffer where it is a pool."""
    t = kw[name]
    if t is None:  # a weight of ones
        t = torch.ones(8)
    if isinstance(t, torch.Tensor):
        return {**kw, name: change(t)}
    return {**kw, name: type(t)(change(t.buf))}


def test_inputs_that_require_a_gradient(L):  # noqa: F811
    for f, kw, names in calls():
        for n in names:
            asking = with_(kw, n, lambda t: t.clone().requires_grad_())
            with pytest.raises(ValueError, match=GRAD):
                f(**asking)
            with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):
                f(**asking)


def test_inputs_with_a_tangent(L):  # noqa: F811
    for f, kw, names in calls():
        for n in names:
            with forward_ad.dual_level(), torch.no_grad():
                with pytest.raises(ValueError, match=GRAD):
                    f(**with_(kw, n, lambda t: forward_ad.make_dual(t, torch.ones_like(t))))
                with pytest.raises(ValueError, match="on a GPU"):
                    f(**kw)
