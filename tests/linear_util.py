"""Inputs, runs and tolerances of the GPU tests of include/gdn_linear.h."""
from __future__ import annotations

import numpy as np
import torch

from gpu_util import DEV, gdn, host
from oracle import linear as ol
from train_util import DT, close, rounded

HALF32 = 2.0 ** -24  # half a step of fp32


class Case:
    """A packed ragged batch on the host and the GPU.

    lens: sequence lengths; decay: "row" or "head"; skip: sequences given a
    negative page; gap: rows before the first sequence; tail: rows behind the
    last one; pad: extra elements between rows; offset: elements before the
    first; fast: the largest -g."""

    def __init__(self, lens, hk=2, hv=4, dk=32, dv=32, act="f32", state="f32", decay="row", skip=(), gap=0, tail=0,
                 pad=0, offset=0, has_init=None, scale=0.5, fast=1.0, seed=0, max_len=0):
        rng = np.random.default_rng(seed)
        g = gdn()
        self.lens, self.hk, self.hv, self.dk, self.dv, self.act, self.state = list(lens), hk, hv, dk, dv, act, state
        self.pad, self.offset, self.decay, self.scale = pad, offset, decay, scale
        n = len(lens)
        cu = gap + np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.n, self.rows = n, int(cu[-1]) + tail
        self.spans = [None if s in skip else (int(cu[s]), int(cu[s + 1])) for s in range(n)]
        self.owned = np.zeros(self.rows, bool)
        for sp in self.spans:
            if sp:
                self.owned[sp[0]:sp[1]] = True
        self.init = np.ones(n, bool) if has_init is None else np.asarray(has_init, bool)
        self.pages = rng.permutation(n + 2)[:n].astype(np.int32)
        self.pages[list(skip)] = -1
        self.dims = g.LinearDims(hk, hv, dk, dv, act_dtype=act, state_dtype=state, scale=scale)
        self.width = {"q": hk * dk, "k": hk * dk, "v": hv * dv, "d_o": hv * dv}
        self.t = {}
        for name, w in self.width.items():
            v = rounded(rng.standard_normal((self.rows, w)), act)
            v[torch.from_numpy(~self.owned)] = float("nan")  # rows nobody may read
            self.t[name] = self.strided(v)
        gates = -fast * rng.random((self.rows, hv) if decay == "row" else hv).astype(np.float32) ** 3
        if decay == "row":
            gates[~self.owned] = np.nan
        self.g = torch.from_numpy(gates).to(DEV)
        self.s0 = rounded(rng.standard_normal((n + 2, hv, dk, dv)), state)
        self.d_state = rng.standard_normal((n, hv, dk, dv)).astype(np.float32)
        self.batch = g.Batch(torch.from_numpy(cu.astype(np.int32)).to(DEV), torch.from_numpy(self.pages).to(DEV),
                             None if has_init is None else torch.tensor(has_init, dtype=torch.uint8, device=DEV),
                             max_len, self.rows)

    def strided(self, v):
        rows, w = v.shape
        buf = torch.full((rows * (w + self.pad) + self.offset + 1,), float("nan"), dtype=v.dtype, device=DEV)
        out = buf[self.offset:self.offset + rows * (w + self.pad)].view(rows, w + self.pad)[:, :w]
        out.copy_(v.to(DEV))
        return out

    def blank(self, name):
        return self.strided(torch.full((self.rows, self.width[name]), float("nan"), dtype=DT[self.act]))

    def f64(self, name):
        heads = self.hk if name in ("q", "k") else self.hv
        return host(self.t[name]).reshape(self.rows, heads, -1)

    def gates(self):
        g = host(self.g)
        return g if self.decay == "row" else np.broadcast_to(g, (self.rows, self.hv))

    def seq_s0(self):
        s0 = self.s0.double().numpy()[np.maximum(self.pages, 0)]
        return np.where(self.init[:, None, None, None], s0, 0.0)

    def forward(self, in_place=False, batch=None, err=None, workspace=None):
        """(o, state_out) of one call; untouched places stay NaN."""
        g = gdn()
        si = g.StatePool(self.s0.to(DEV).clone())
        so = si if in_place else g.StatePool(torch.full_like(si.buf, float("nan")))
        o = g.gdnl_attend_forward(self.dims, self.t["q"], self.t["k"], self.t["v"], self.g, batch or self.batch, si, so,
                                  o=self.blank("v"), err=err, workspace=workspace)
        torch.cuda.synchronize()
        return o, so

    def backward(self, d_state=True, with_dg=True, batch=None, err=None, workspace=None):
        g = gdn()
        nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
        dg = (nan(self.rows, self.hv) if self.decay == "row" else nan(self.hv)) if with_dg else None
        out = g.LinearGrads(self.blank("q"), self.blank("k"), self.blank("v"), dg, nan(self.n, self.hv, self.dk, self.dv))
        out = g.gdnl_attend_backward(self.dims, self.t["q"], self.t["k"], self.t["v"], self.g, batch or self.batch,
                                     g.StatePool(self.s0.to(DEV)), self.t["d_o"],
                                     d_state=torch.from_numpy(self.d_state).to(DEV) if d_state else None, out=out,
                                     err=err, workspace=workspace)
        torch.cuda.synchronize()
        return out

    # ---------------------------------------------------------------- bounds
    # Errors are bounded by `tol` times the same sums over absolute values.  A
    # sum of n products in fp32 is off by at most n half steps; on a value's way
    # there are products over d_k and d_v, over the 64 rows of a chunk, and four
    # operations on the state for each chunk of its sequence.  A decay 2^d has an
    # exponent off by 3 half steps of d, so a weight is off by 3 |d| ln 2 half
    # steps of itself; as x e^{-x} <= (2/e) e^{-x/2}, that is under 3 half steps
    # of the weight with half the decay: absolute sums are taken with g / 2.
    # With bf16 rows P and S stand as two terms each: the first leaves 2^-7 of
    # the value (cut off), the second 2^-8 of that: 2^-15 each.
    def tol(self, split=False):
        chunks = -(-max(self.lens, default=0) // 64)
        adds = 2 * max(self.dk, self.dv) + 160 + 4 * chunks
        return adds * HALF32 + (2.0 ** -14 if split and self.act == "bf16" else 0.0)

    def inputs(self):
        return self.f64("q"), self.f64("k"), self.f64("v"), self.gates()

    def check_forward(self, o, so):
        q, k, v, g = self.inputs()
        with np.errstate(invalid="ignore"):
            ref, last = ol.attend(q, k, v, g, self.spans, self.seq_s0(), self.scale)
            mag, last_mag = ol.attend(*map(np.abs, (q, k, v)), g / 2, self.spans, np.abs(self.seq_s0()), abs(self.scale))
        close("o", host(o).reshape(ref.shape), ref, mag, self.tol(split=True), self.act)
        if so is not None:
            pages, pmag = np.full(tuple(so.buf.shape), np.nan), np.zeros(tuple(so.buf.shape))
            for s, sp in enumerate(self.spans):
                if sp and sp[1] > sp[0]:
                    pages[self.pages[s]], pmag[self.pages[s]] = last[s], last_mag[s]
            close("state", host(so.buf), pages, pmag, self.tol(), self.state)

    def check_backward(self, got, d_state=True, dead=None):
        q, k, v, g = self.inputs()
        d_o, ds = self.f64("d_o"), self.d_state if d_state else np.zeros_like(self.d_state)
        per = self.hv // self.hk
        with np.errstate(invalid="ignore"):
            ref = ol.attend_backward(q, k, v, g, self.spans, self.seq_s0(), self.scale, d_o, ds, self.init)
            mag = ol.attend_backward(*map(np.abs, (np.repeat(q, per, 1), np.repeat(k, per, 1), v)), g / 2, self.spans,
                                     np.abs(self.seq_s0()), abs(self.scale), np.abs(d_o), np.abs(ds), self.init)
        group = lambda t: t.reshape(self.rows, self.hk, per, -1).sum(2)  # noqa: E731
        for name, m in (("dq", group(mag["dq"])), ("dk", group(mag["dk"])), ("dv", mag["dv"])):
            close(name, host(getattr(got, name)).reshape(m.shape), ref[name], m, self.tol(split=True) + per * HALF32, self.act)
        close("d_state0", host(got.d_state0), ref["d_state0"], np.abs(mag["d_state0"]), self.tol(), "f32")
        if got.dg is None:
            return ref
        # dg is a sum over the rows behind: every term of it is a product with dq or dk
        m = np.full(g.shape, np.nan)
        for sp in self.spans:
            if sp and sp[1] > sp[0]:
                r = slice(*sp)
                terms = (np.repeat(np.abs(q[r]), per, 1) * mag["dq"][r]).sum(-1) + 2 * (np.repeat(np.abs(k[r]), per, 1) * mag["dk"][r]).sum(-1)
                m[r] = terms[::-1].cumsum(0)[::-1] + mag["dg"][r][-1]
        dg = ref["dg"] if dead is None else np.where(dead, 0.0, ref["dg"])
        tol = 2 * self.tol() + 8 * HALF32
        if self.decay == "row":
            close("dg", host(got.dg), dg, m, tol, "f32")
        else:
            close("dg", host(got.dg), np.nansum(dg, 0), np.nansum(m, 0), tol, "f32")
        return ref
