"""Inputs, runs and tolerances of the GPU tests of include/gdn_train.h."""
from __future__ import annotations

import numpy as np
import torch

from gpu_util import DEV, gdn, host

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
#: a rounding is off by at most half a step of the value
HALF = {"bf16": torch.finfo(torch.bfloat16).eps / 2, "f32": torch.finfo(torch.float32).eps / 2}
ULP = 2.0 ** -23


def rounded(v, dt):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(DT[dt])


class Case:
    """A packed ragged batch on the host and the GPU.

    lens: sequence lengths; skip: sequences given a negative page; gap: rows
    before the first sequence; tail: rows behind the last one; pad: extra
    elements between rows; dt_lo, dt_hi: range of the softplus step."""

    def __init__(self, lens, C, act="bf16", state="f32", skip=(), gap=0, tail=0, pad=0, has_init=None, seed=0,
                 dt_lo=0.02, dt_hi=0.5, offset=0):
        rng = np.random.default_rng(seed)
        g = gdn()
        self.lens, self.C, self.act, self.state, self.pad, self.offset = list(lens), C, act, state, pad, offset
        n = len(lens)
        cu = gap + np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.n, self.rows = n, int(cu[-1]) + tail
        self.spans = [None if s in skip else (int(cu[s]), int(cu[s + 1])) for s in range(n)]
        self.owned = np.zeros(self.rows, bool)
        for sp in self.spans:
            if sp:
                self.owned[sp[0]:sp[1]] = True
        self.has_init = has_init
        self.init = np.ones(n, bool) if has_init is None else np.asarray(has_init, bool)
        pages = rng.permutation(n + 2)[:n].astype(np.int32)
        pages[list(skip)] = -1
        self.pages = pages
        self.dims = g.ScanDims(C, act_dtype=act, state_dtype=state)
        step = np.exp(rng.uniform(np.log(dt_lo), np.log(dt_hi), C))
        self.a_log = np.log(rng.uniform(1, 16, C)).astype(np.float32)
        self.dt_bias = np.log(np.expm1(step)).astype(np.float32)
        self.params = g.ScanParams(torch.from_numpy(self.a_log).to(DEV), torch.from_numpy(self.dt_bias).to(DEV))
        self.t = {}
        for k in ("x", "a", "b", "dh"):
            v = rounded(rng.standard_normal((self.rows, C)), act)
            v[torch.from_numpy(~self.owned)] = float("nan")  # rows nobody may read
            self.t[k] = self.strided(v)
        self.h0 = rounded(rng.standard_normal((n + 2, C)), state)
        self.d_state = rng.standard_normal((n, C)).astype(np.float32)
        self.batch = g.Batch(torch.from_numpy(cu.astype(np.int32)).to(DEV), torch.from_numpy(pages).to(DEV),
                             None if has_init is None else torch.tensor(has_init, dtype=torch.uint8, device=DEV),
                             0, self.rows)

    def strided(self, v):
        """v on the GPU with `pad` elements between rows, `offset` elements into its buffer."""
        buf = torch.full((v.shape[0] * (v.shape[1] + self.pad) + self.offset + 1,), float("nan"), dtype=v.dtype,
                         device=DEV)
        out = buf[self.offset:self.offset + v.shape[0] * (v.shape[1] + self.pad)].view(v.shape[0], v.shape[1] + self.pad)[:, :v.shape[1]]
        out.copy_(v.to(DEV))
        return out

    def f64(self, k):
        return host(self.t[k])

    def seq_h0(self):
        h0 = self.h0.double().numpy()[np.maximum(self.pages, 0)]
        return np.where(self.init[:, None], h0, 0.0)

    def empty_rows(self):
        return self.strided(torch.full((self.rows, self.C), float("nan"), dtype=DT[self.act]))

    def forward(self, saved=None, in_place=False, batch=None, err=None, state_in=None):
        """(h, state_in, state_out) of one call; untouched places stay NaN."""
        g = gdn()
        si = g.StatePool(self.h0.to(DEV).clone()) if state_in is None else state_in
        so = si if in_place else g.StatePool(torch.full_like(si.buf, float("nan")))
        h = self.empty_rows()
        g.gdnt_scan_forward(self.dims, self.params, self.t["x"], self.t["a"], self.t["b"], batch or self.batch, si, so,
                            h=h, saved=saved, err=err)
        torch.cuda.synchronize()
        return h, si, so

    def saved(self, ckpt=False):
        s = gdn().ScanSaved.alloc(self.dims, self.rows, DEV, ckpt=ckpt)
        s.states.fill_(float("nan"))
        return s

    def grads_out(self):
        g = gdn()
        f = lambda *s: torch.full(s, float("nan"), device=DEV)
        return g.ScanGrads(self.empty_rows(), self.empty_rows(), self.empty_rows(), f(self.C), f(self.C),
                           f(self.n, self.C))

    def backward(self, saved, from_ckpt=False, d_state=True, batch=None, err=None):
        g = gdn()
        xab = {} if from_ckpt else {k: self.t[k] for k in "xab"}
        out = g.gdnt_scan_backward(self.dims, self.params, batch or self.batch, g.StatePool(self.h0.to(DEV)), saved,
                                   self.t["dh"], d_state=torch.from_numpy(self.d_state).to(DEV) if d_state else None,
                                   out=self.grads_out(), err=err, **xab)
        torch.cuda.synchronize()
        return out

    # ---------------------------------------------------------------- bounds
    # alpha = 2^y by the hardware's exponential, off by one ulp, from a y off by
    # 8 half ulps of itself: a product of n decays is off by n ulps and, as
    # n |g| e^{-n |g|} <= 1/e, by less than 4 half ulps more.  u and each fma add
    # a few half ulps.  With every term of a sum counted by its magnitude (the
    # same recurrence over absolute values), the error of a state is below
    # (32 + 1.5 n) ulps of that, n the longest sequence; gradients multiply two
    # such quantities and a few factors good to some ulps: twice that and 32.
    def tol(self):
        return (32 + 1.5 * max(self.lens, default=0)) * ULP


def close(name, got, ref, mag, tol, dt):
    """|got - ref| <= half a step of the type + tol * mag where ref is a number; got untouched (NaN) where ref is NaN."""
    got, ref, mag = (np.asarray(v, np.float64) for v in (got, ref, mag))
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    wrote = ~np.isnan(ref)
    assert np.isnan(got[~wrote]).all(), f"{name}: a row that nobody owns was written"
    assert not np.isnan(got[wrote]).any(), f"{name}: a value is missing"
    off = np.abs(got - ref)[wrote] - (HALF[dt] * np.abs(ref) + (1 + HALF[dt]) * tol * mag)[wrote]
    assert off.size == 0 or off.max() <= 1e-37, f"{name}: {off.max():.3e} beyond its bound at {int(off.argmax())}"


def check_forward(c, h, so, ora):
    args = (c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans)
    with np.errstate(invalid="ignore"):
        ref, last, before = ora.scan(c.f64("x"), *args, c.seq_h0())
        mag, last_mag, _ = ora.scan(np.abs(c.f64("x")), *args, np.abs(c.seq_h0()))
    close("h", host(h), ref, mag, c.tol(), c.act)
    if so is not None:
        pages = np.full(tuple(so.buf.shape), np.nan)
        pmag = np.zeros_like(pages)
        for s, sp in enumerate(c.spans):
            if sp and sp[1] > sp[0]:
                pages[c.pages[s]], pmag[c.pages[s]] = last[s], last_mag[s]
        close("state", host(so.buf), pages, pmag, c.tol(), c.state)
    return ref, before


def check_grads(c, g, ora, x=None, a=None, b=None, before=None, d_state=True):
    """g against the oracle at x, a, b (default: the inputs) with the state before each row."""
    x, a, b = (c.f64(k) if v is None else v for k, v in (("x", x), ("a", a), ("b", b)))
    ds = c.d_state if d_state else np.zeros_like(c.d_state)
    args = (a, b, c.a_log, c.dt_bias, c.spans)
    with np.errstate(invalid="ignore"):
        hb = ora.scan(x, *args, c.seq_h0())[2] if before is None else before
        hm = ora.scan(np.abs(x), *args, np.abs(c.seq_h0()))[2]
        if before is not None:
            hm = np.maximum(hm, np.abs(before))
        ref = ora.scan_backward(x, *args, hb, c.f64("dh"), ds, c.init)
        mag = ora.scan_backward(np.abs(x), *args, hm, np.abs(c.f64("dh")), np.abs(ds), c.init)
    tol = 2 * c.tol() + 32 * ULP
    # 1 - beta is off by an ulp of 1, whatever is left of it
    beta = ora.sigmoid(b)
    mag["db"] = np.abs(mag["db"]) + np.abs(mag["dx"] * x) * 2 * ULP / tol
    del beta
    # fp32 sums within 256 rows: at most 8 + 2 + 8 additions deep on a value's way, inside tol
    for k in ("dx", "da", "db"):
        close(k, host(getattr(g, k)), ref[k], np.abs(mag[k]), tol, c.act)
    # the bounds of a sum are those of its terms: every term of d_a_log, d_dt_bias has one sign in `mag`
    for k in ("d_a_log", "d_dt_bias"):
        close(k, host(getattr(g, k)), ref[k], np.abs(mag[k]), tol, "f32")
    close("d_state0", host(g.d_state0), ref["d_state0"], np.abs(mag["d_state0"]), tol, "f32")  # zeros where skipped
    return ref
