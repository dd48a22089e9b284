"""Linear attention over segments of hundreds and thousands of rows: whole
numbers without decays, where every result is the exact one, and normal numbers
with decays, in the norm of a sequence and head, against float64."""
import numpy as np
import pytest
import torch

import linear_long as ll
from gpu_util import DEV, gdn
from train_util import DT, rounded

pytestmark = pytest.mark.gpu

# Rows of a segment follow from rows times heads: named by what they are forward, and backward where it differs.
CASES = {
    "uncut": dict(lens=[656, 257, 320, 1000], hk=32, hv=64),
    "uncut, 256 and 257 rows": dict(lens=[256, 257], hk=128, hv=128),
    "cut at 257 rows": dict(lens=[256, 257], hk=1, hv=2),
    "256": dict(lens=[3000, 0, 257], hk=32, hv=32),
    "512": dict(lens=[6500, 3], hk=16, hv=32),
    "1024": dict(lens=[5000, 700], hk=64, hv=64),
    "4096, 2048 backward": dict(lens=[10000, 333], hk=64, hv=128),
    "256 of 128 x 128": dict(lens=[2500, 70], hk=8, hv=16, d=128),
    "uncut, 128 x 64": dict(lens=[700, 300], hk=64, hv=128, d=128, dv=64),
}


class Case:
    def __init__(self, lens, hk, hv, d=8, dv=None, act="f32", decay="row", whole=False, fast=0.05, seed=1):
        rng = np.random.default_rng(seed)
        g = gdn()
        self.lens, self.hk, self.hv, self.dk, self.dv, self.act, self.decay = lens, hk, hv, d, dv or d, act, decay
        self.cu, self.n = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), len(lens)
        self.rows, self.scale = int(self.cu[-1]), 1.0 if whole else 0.5
        width = {"q": hk * d, "k": hk * d, "v": hv * self.dv, "d_o": hv * self.dv}
        state = self.n, hv, d, self.dv
        if whole:  # few of a wide head's places: sums below 2^24
            few = lambda n, w, k: rng.integers(-1, 2, (n, w)) * (rng.random((n, w)) < 8 / k)  # noqa: E731
            self.t = {n: rounded(few(self.rows, w, w // (hk if n in "qk" else hv)), act).to(DEV) for n, w in width.items()}
            self.s0, self.d_state = (rng.integers(-3, 4, state).astype(np.float32) for _ in range(2))
            self.g = torch.zeros((self.rows, hv) if decay == "row" else hv, device=DEV)
        else:
            self.t = {n: rounded(rng.standard_normal((self.rows, w)), act).to(DEV) for n, w in width.items()}
            self.s0, self.d_state = (rng.standard_normal(state).astype(np.float32) for _ in range(2))
            gates = -fast * rng.random((self.rows, hv) if decay == "row" else hv).astype(np.float32) ** 3
            self.g = torch.from_numpy(gates).to(DEV)
        self.dims = g.LinearDims(hk, hv, d, self.dv, act_dtype=act, scale=self.scale)
        self.batch = g.Batch(torch.from_numpy(self.cu).to(DEV), torch.arange(self.n, dtype=torch.int32, device=DEV), None, 0, self.rows)

    def run(self):
        """(o, states, gradients), the forward call in place."""
        g = gdn()
        start = torch.from_numpy(self.s0).to(DEV)
        pool = g.StatePool(start.clone())
        args = self.dims, self.t["q"], self.t["k"], self.t["v"], self.g, self.batch
        o = g.gdnl_attend_forward(*args, pool)
        d = g.gdnl_attend_backward(*args, g.StatePool(start), self.t["d_o"], d_state=torch.from_numpy(self.d_state).to(DEV))
        torch.cuda.synchronize()
        return o, pool.buf, d

    def inputs(self, s):
        """Those of one sequence by value head, as linear_long takes them."""
        r, per = slice(self.cu[s], self.cu[s + 1]), self.hv // self.hk
        q, k = (self.t[n][r].double().reshape(-1, self.hk, self.dk).repeat_interleave(per, 1) for n in "qk")
        v, d_o = (self.t[n][r].double().reshape(-1, self.hv, self.dv) for n in ("v", "d_o"))
        g = self.g[r].double() if self.decay == "row" else self.g.double().expand(len(q), self.hv)
        s0, d_state = (torch.from_numpy(t[s]).to(DEV).double() for t in (self.s0, self.d_state))
        return q, k, v, g, s0, self.scale, d_o, d_state

    def grouped(self, t):
        return t.reshape(len(t), self.hk, -1, t.shape[-1]).sum(2)


@pytest.mark.parametrize("decay", ["row", "head"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_whole_numbers(name, act, decay):
    c = Case(**CASES[name], act=act, decay=decay, whole=True)
    o, states, d = c.run()

    def same(what, got, want, dt):
        want = want.to(DT[dt]).reshape(got.shape)
        assert torch.equal(got, want), f"{what}: {int((got != want).sum())} of {got.numel()}"

    dg_sum = torch.zeros(c.hv, dtype=torch.float64, device=DEV)
    for s in range(c.n):
        r, a = slice(c.cu[s], c.cu[s + 1]), c.inputs(s)
        if r.start == r.stop:
            continue
        ref, last = ll.attend(*a[:6])
        dq, dk, dv, dg, d0 = ll.gradients(*a)
        assert max(float(t.abs().max()) for t in (ref, last, dq, dk, dv, d0)) < 2.0 ** 23
        same("o", o[r], ref, act)
        same("state", states[s], last, "f32")
        same("dq", d.dq[r], c.grouped(dq), act)
        same("dk", d.dk[r], c.grouped(dk), act)
        same("dv", d.dv[r], dv, act)
        same("d_state0", d.d_state0[s], d0, "f32")
        if decay == "row":
            same("dg", d.dg[r], dg, "f32")
        dg_sum += dg.sum(0)
    if decay == "head":
        same("dg", d.dg, dg_sum, "f32")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("decay,fast", [("row", 0.05), ("head", 0.05), ("row", 3.0)])
@pytest.mark.parametrize("name", CASES)
def test_errors_are_those_of_fp32_sums(name, fast, act, decay):
    """The norm of what a result is off by, beyond the half step of a bf16
    rounding, against its terms' root sums of squares."""
    c = Case(**CASES[name], act=act, decay=decay, fast=fast)
    o, states, d = c.run()

    def within(what, got, want, square, bound, dt, axes):
        off = (got.double().reshape(want.shape) - want).abs()
        if dt == "bf16":
            off = (off - 2.0 ** (want.abs().log2().floor() - 8)).clamp(min=0.0)
        ratio = float(((off ** 2).sum(axes) / square.sum(axes)).sqrt().max())
        assert ratio <= bound, f"{what}: {ratio:.3g} > {bound:.3g}"

    dg_ref, dg_err2 = (torch.zeros(c.hv, dtype=torch.float64, device=DEV) for _ in range(2))
    for s in range(c.n):
        r, a = slice(c.cu[s], c.cu[s + 1]), c.inputs(s)
        rows = r.stop - r.start
        if rows == 0:
            continue
        ref, last = ll.attend(*a[:6])
        dq, dk, dv, dg, d0 = ll.gradients(*a)
        o2, S2, dq2, dk2, dv2, d02 = ll.squares(*a)
        slack, q, k = ll.slack(c.dk, c.dv, rows), a[0], a[1]
        within("o", o[r], ref, o2, slack, act, (0, 2))
        within("state", states[s], last, S2, ll.state_slack(rows), "f32", (1, 2))
        within("dq", d.dq[r], c.grouped(dq), c.grouped(dq2), slack, act, (0, 2))
        within("dk", d.dk[r], c.grouped(dk), c.grouped(dk2), slack, act, (0, 2))
        within("dv", d.dv[r], dv, dv2, slack, act, (0, 2))
        within("d_state0", d.d_state0[s], d0, d02, ll.state_slack(rows), "f32", (1, 2))
        if decay == "row":
            bound2 = 9 * (ll.dg_error(q, k, dq2, dk2, slack) ** 2).sum(0)
            ratio = float((((d.dg[r].double() - dg) ** 2).sum(0) / bound2).sqrt().max())
            assert ratio <= 1.0, f"dg: {ratio:.3g} of its bound"
        dg_ref += dg.sum(0)
        dg_err2 += ll.dg_error(q, k, dq2, dk2, slack, whole=True) ** 2
    if decay == "head":
        ratio = float(((d.dg.double() - dg_ref).abs() / (9 * dg_err2).sqrt()).max())
        assert ratio <= 1.0, f"dg: {ratio:.3g} of its bound"
