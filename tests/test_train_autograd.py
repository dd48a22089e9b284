"""The training binding and autograd: history that would be lost in silence is
refused (CPU), and a torch.autograd.Function over the calls trains (GPU)."""
import numpy as np
import pytest
import torch


def host_call():
    """Arguments that are right but for being on the host, the last thing refused."""
    import linear_attention_ssm_gdn_amd as g
    t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    batch = g.Batch(torch.tensor([0, 4], dtype=torch.int32), t(1, dt=torch.int32), None, 0, 4)
    return g, dict(dims=g.ScanDims(8, act_dtype="f32"), params=g.ScanParams(t(8), t(8)), x=t(4, 8), a=t(4, 8),
                   b=t(4, 8), batch=batch, state_in=g.StatePool(t(1, 8)))


@pytest.mark.parametrize("name", ["x", "a", "b", "a_log", "dt_bias", "state"])
def test_a_forward_call_that_would_lose_history_is_refused(name):
    g, kw = host_call()
    t = {"state": kw["state_in"].buf}.get(name, getattr(kw["params"], name, kw.get(name)))
    t.requires_grad_()
    with pytest.raises(ValueError, match="autograd"):
        g.gdnt_scan_forward(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):  # all else is in order
        g.gdnt_scan_forward(**kw)


def test_backward_calls_that_would_lose_history_are_refused():
    g, kw = host_call()
    saved = g.ScanSaved(torch.zeros(1, 8))
    scan = lambda dh, **more: g.gdnt_scan_backward(kw["dims"], kw["params"], kw["batch"], kw["state_in"], saved, dh,
                                                   x=kw["x"], a=kw["a"], b=kw["b"], **more)
    wants = lambda *s: torch.zeros(*s, requires_grad=True)
    with pytest.raises(ValueError, match="autograd"):
        scan(wants(4, 8))
    with pytest.raises(ValueError, match="autograd"):
        scan(torch.zeros(4, 8), d_state=wants(1, 8))
    kw["x"].requires_grad_()  # its gradient is what the call returns
    with pytest.raises(ValueError, match="on a GPU"):
        scan(torch.zeros(4, 8))
    cd = g.Dims(1, 1, 32, 32, act_dtype="f32")
    with pytest.raises(ValueError, match="autograd"):
        g.gdnt_conv_backward(cd, torch.zeros(96, 4), torch.zeros(4, 96), wants(4, 96), kw["batch"])


@pytest.mark.gpu
def test_a_function_over_the_calls():
    """As the module's docstring has it: gradients arrive at the leaves, and are those of the calls by hand."""
    from gpu_util import DEV, gdn
    from train_util import Case
    g = gdn()
    c = Case([40, 0, 300, 7], 72, "f32", "f32", seed=71)

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, a, b, a_log, dt_bias):
            ctx.params, ctx.saved = g.ScanParams(a_log, dt_bias), g.ScanSaved.alloc(c.dims, c.rows, DEV)
            ctx.pool = g.StatePool(c.h0.to(DEV))
            ctx.save_for_backward(x, a, b)
            return g.gdnt_scan_forward(c.dims, ctx.params, x, a, b, c.batch, ctx.pool, g.StatePool(c.h0.to(DEV)),
                                       saved=ctx.saved)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dh):
            x, a, b = ctx.saved_tensors
            out = g.gdnt_scan_backward(c.dims, ctx.params, c.batch, ctx.pool, ctx.saved, dh.contiguous(), x=x, a=a, b=b)
            return out.dx, out.da, out.db, out.d_a_log, out.d_dt_bias

    leaves = [t.clone().requires_grad_() for t in (c.t["x"], c.t["a"], c.t["b"], c.params.a_log, c.params.dt_bias)]
    Scan.apply(*leaves).backward(c.t["dh"])
    saved = c.saved()
    c.forward(saved)
    want = c.backward(saved, d_state=False)
    for t, w in zip(leaves, want):
        assert np.array_equal(t.grad.cpu().numpy(), w.cpu().numpy())
