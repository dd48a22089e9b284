"""The operators of include/gdn_linear.h as they are used together: serving
(rotate, prompts, states kept in 8 bits and restored, single rows) and a
trainable layer."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
from oracle import linear as ol

pytestmark = pytest.mark.gpu

HK, HV, D = 2, 4, 64


def _layer(rows, seed=0, act="f32"):
    g = gdn()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = torch.float32 if act == "f32" else torch.bfloat16
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    return {"rot": g.RotateDims(HK, HK, D, 32, act_dtype=act), "dims": g.LinearDims(HK, HV, D, D, act_dtype=act, scale=D ** -0.5),
            "q": n(rows, HK * D).to(dt), "k": n(rows, HK * D).to(dt), "v": n(rows, HV * D).to(dt), "g": -0.1 * n(rows, HV).abs(),
            "wq": 1 + 0.1 * n(D), "wk": 1 + 0.1 * n(D), "inv": 10000.0 ** (-torch.arange(16, device=DEV) / 16.0)}


def test_serving():
    """Two requests share a prefix: it is prefilled once, kept in 8 bits and restored for the second."""
    g = gdn()
    prefix, more = 100, 4
    t = _layer(prefix + 2 * more)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    pos = torch.cat([torch.arange(prefix), torch.arange(more).repeat(2) + prefix]).to(torch.int32).to(DEV)
    q, k = g.gdnl_rotate_forward(t["rot"], t["q"], t["k"], t["wq"], t["wk"], pos, t["inv"])
    pool, cache = g.StatePool(torch.zeros(3, HV, D, D, device=DEV)), g.StateCache.alloc(t["dims"], 2, DEV)
    o = torch.zeros_like(t["v"])
    rows = prefix + 2 * more
    g.gdnl_attend_forward(t["dims"], q, k, t["v"], t["g"], g.Batch(i32(0, prefix), i32(2), torch.zeros(1, dtype=torch.uint8, device=DEV), 0, rows), pool, o=o)
    g.gdnl_cache_store(t["dims"], i32(2), i32(1), pool, cache)
    g.gdnl_cache_load(t["dims"], i32(1), i32(0), cache, pool)
    for j in range(more):
        first, second = prefix + j, prefix + more + j
        cu = i32(first, first + 1)
        g.gdnl_attend_forward(t["dims"], q, k, t["v"], t["g"], g.Batch(cu, i32(2), None, 1, rows), pool, o=o)
        g.gdnl_attend_forward(t["dims"], q, k, t["v"], t["g"], g.Batch(i32(second, second + 1), i32(0), None, 1, rows), pool, o=o)
    heads = lambda x, h: host(x).reshape(rows, h, D)  # noqa: E731
    args = (host(pos), host(t["inv"]), 32, "rms", "halves", 1e-6)
    rq, rk = ol.rotate(heads(t["q"], HK), host(t["wq"]), *args), ol.rotate(heads(t["k"], HK), host(t["wk"]), *args)
    rv, rg = heads(t["v"], HV), host(t["g"])
    ref, last = ol.attend(rq, rk, rv, rg, [(0, prefix)], np.zeros((1, HV, D, D)), D ** -0.5)
    one, _ = ol.attend(rq, rk, rv, rg, [(prefix, prefix + more)], last, D ** -0.5)
    got = heads(o, HV)
    scale = np.abs(ref[:prefix]).max()
    # sums of some hundred fp32 products of values below `scale`
    assert np.abs(got[:prefix] - ref[:prefix]).max() <= 500 * 2.0 ** -24 * scale * 8
    assert np.abs(got[prefix:prefix + more] - one[prefix:prefix + more]).max() <= 500 * 2.0 ** -24 * scale * 8
    kept = ol.cached(last.astype(np.float32))[2]
    two, _ = ol.attend(rq, rk, rv, rg, [(prefix + more, rows)], kept, D ** -0.5)
    # an integer that falls the other way moves its value by a scale, 1/127 of a block's largest
    step = np.abs(last).max() / 127 * np.abs(rq).max() * D ** -0.5
    assert np.abs(got[prefix + more:] - two[prefix + more:]).max() <= 500 * 2.0 ** -24 * scale * 8 + 4 * step


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_trainable_layer(act):
    """torch.autograd.Functions over the calls: gradients arrive at the leaves and are the formulas'."""
    g = gdn()
    rows, lens = 150, [100, 0, 50]
    t = _layer(rows, seed=3, act=act)
    cu = torch.tensor([0, 100, 100, 150], dtype=torch.int32, device=DEV)
    batch = g.Batch(cu, torch.arange(3, dtype=torch.int32, device=DEV), None, 0, rows)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(DEV)
    zero = g.StatePool(torch.zeros(3, HV, D, D, device=DEV))

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk):
            ctx.save_for_backward(q, k, wq, wk)
            return g.gdnl_rotate_forward(t["rot"], q, k, wq, wk, pos, t["inv"])

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq, dk):
            q, k, wq, wk = ctx.saved_tensors
            return tuple(g.gdnl_rotate_backward(t["rot"], q, k, wq, wk, pos, t["inv"], dq.contiguous(), dk.contiguous()))

    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, gates):
            ctx.save_for_backward(q, k, v, gates)
            return g.gdnl_attend_forward(t["dims"], q, k, v, gates, batch, zero, g.StatePool(torch.empty_like(zero.buf)))

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_o):
            out = g.gdnl_attend_backward(t["dims"], *ctx.saved_tensors, batch, zero, d_o.contiguous())
            return out.dq, out.dk, out.dv, out.dg

    leaves = {n: t[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk", "v", "g")}
    d_o = torch.randn(rows, HV * D, device=DEV).to(t["v"].dtype)
    Attend.apply(*Rotate.apply(leaves["q"], leaves["k"], leaves["wq"], leaves["wk"]), leaves["v"], leaves["g"]).backward(d_o)

    heads = lambda x, h: host(x).reshape(rows, h, -1)  # noqa: E731
    args = (host(pos), host(t["inv"]), 32, "rms", "halves", 1e-6)
    x = {n: heads(t[n], HK) for n in ("q", "k")}
    y = {n: ol.rotate(x[n], host(t["w" + n]), *args) for n in ("q", "k")}
    ref = ol.attend_backward(y["q"], y["k"], heads(t["v"], HV), host(t["g"]), [(0, 100), (100, 100), (100, 150)],
                             np.zeros((3, HV, D, D)), D ** -0.5, heads(d_o, HV), np.zeros((3, HV, D, D)))
    want = {"v": ref["dv"], "g": ref["dg"]}
    for n in ("q", "k"):
        want[n], want["w" + n] = ol.rotate_backward(x[n], host(t["w" + n]), *args, ref["d" + n])
    # three roundings to the act dtype on the way (y, its gradient, the result), each half a step of a value that
    # random signs spread over the norm; fp32: some hundred of them
    tol = 4 * torch.finfo(t["v"].dtype).eps / 2 * (1 if act == "bf16" else 100)
    for n, w in want.items():
        got = host(leaves[n].grad).reshape(w.shape)
        assert np.linalg.norm(got - w) <= tol * np.linalg.norm(w), n
