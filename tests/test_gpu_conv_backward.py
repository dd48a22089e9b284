"""GPU tests of the conv's backward pass against the float64 oracle
(oracle/train.py), and of conv, recurrence and both backward passes run
together as a trainable block."""
import numpy as np
import pytest
import torch

import oracle.train as ora
from gpu_util import DEV, gdn, host
from train_util import DT, HALF, ULP, close, rounded

pytestmark = pytest.mark.gpu


class Conv:
    def __init__(self, lens, heads=(1, 1, 32, 32), act="bf16", ydt="f32", skip=(), gap=0, tail=0, pad=0, offset=0,
                 has_init=None, seed=0):
        rng = np.random.default_rng(seed)
        g = gdn()
        self.dims = g.Dims(*heads, act_dtype=act)
        self.C, self.act, self.ydt, self.n, self.pad, self.offset = self.dims.c_conv, act, ydt, len(lens), pad, offset
        cu = gap + np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.rows = int(cu[-1]) + tail
        self.spans = [None if s in skip else (int(cu[s]), int(cu[s + 1])) for s in range(self.n)]
        self.pages = rng.permutation(self.n + 2)[:self.n].astype(np.int32)
        self.pages[list(skip)] = -1
        owned = np.zeros(self.rows, bool)
        for sp in self.spans:
            if sp:
                owned[sp[0]:sp[1]] = True
        self.owned = owned
        self.init = np.ones(self.n, bool) if has_init is None else np.asarray(has_init, bool)
        self.w = rounded(rng.standard_normal((self.C, 4)) * 0.25, act).to(DEV)
        self.win = rounded(rng.standard_normal((self.n + 2, 4, self.C)), act).to(DEV)  # a pool with a spare row
        self.x, self.dy = (self.strided(self.hide(rounded(rng.standard_normal((self.rows, self.C)), dt)))
                           for dt in (act, ydt))
        self.d_window = rng.standard_normal((self.n, 3, self.C)).astype(np.float32)
        self.batch = g.Batch(torch.from_numpy(cu.astype(np.int32)).to(DEV), torch.from_numpy(self.pages).to(DEV),
                             None if has_init is None else torch.tensor(has_init, dtype=torch.uint8, device=DEV), 0,
                             self.rows)

    def hide(self, v):
        v[torch.from_numpy(~self.owned)] = float("nan")
        return v

    def strided(self, v):
        n = v.shape[0] * (v.shape[1] + self.pad)
        buf = torch.full((n + self.offset + 1,), float("nan"), dtype=v.dtype, device=DEV)
        out = buf[self.offset:self.offset + n].view(v.shape[0], v.shape[1] + self.pad)[:, :v.shape[1]]
        out.copy_(v.to(DEV))
        return out

    def run(self, activation=True, d_window=True, conv=True, err=None, batch=None):
        g = gdn()
        f = lambda *s: torch.full(s, float("nan"), device=DEV)
        out = g.ConvGrads(self.strided(torch.full((self.rows, self.C), float("nan"), dtype=DT[self.act])),
                          f(self.C, 4), f(self.n, 3, self.C))
        pool = g.ConvPool(self.win, None) if conv else None
        g.gdnt_conv_backward(self.dims, self.w, self.x, self.dy, batch or self.batch, pool, activation=activation,
                             d_window=torch.from_numpy(self.d_window).to(DEV) if d_window else None, out=out, err=err)
        torch.cuda.synchronize()
        return out

    def check(self, out, activation=True, d_window=True, conv=True):
        init = self.init if conv else np.zeros(self.n, bool)
        win = host(self.win)[np.maximum(self.pages, 0), :3]
        dwin = self.d_window if d_window else np.zeros_like(self.d_window)
        args = (host(self.x), host(self.dy), self.spans, win, dwin)
        with np.errstate(invalid="ignore"):
            ref = ora.conv_backward(host(self.w), *args, activation, init)
            # z is off by 5 half ulps of the sum of its terms' magnitudes, and |silu''| <= 0.5 turns that into an error
            # of silu'; the hardware's sigmoid is off by some ulps of 1 and silu' <= 1.1 by a few of its factors; |z|
            # below comes from inputs of a few units: 40 ulps of |dy| (1 + |z|), here with 1 + |z| <= 16
            mag = ora.conv_backward(np.abs(host(self.w)), np.abs(host(self.x)), np.abs(host(self.dy)), self.spans,
                                    np.abs(win), np.abs(dwin), False, init)
        tol = 16 * 40 * ULP
        close("dx", host(out.dx), ref["dx"], mag["dx"], tol, self.act)
        # a sum of at most 16 + 4 + 2 fp32 additions deep, then fp64: inside tol
        close("d_conv_w", host(out.d_conv_w), ref["d_conv_w"], mag["d_conv_w"], tol, "f32")
        close("d_window0", host(out.d_window0), ref["d_window0"], mag["d_window0"], tol, "f32")  # zeros where skipped


LENS = {"one": [1], "two": [2], "three": [3], "four": [4], "edge": [15, 16, 17], "tile": [256], "tile+2": [258, 1],
        "ragged": [0, 1, 5, 300, 0, 2, 3, 16, 0], "ones": [1] * 35, "shorts": [3, 2, 1, 2, 3, 4, 1, 1, 1, 5, 16, 2, 250]}


@pytest.mark.parametrize("act,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
def test_conv_backward(lens, act, ydt):
    c = Conv(LENS[lens], act=act, ydt=ydt, seed=len(lens))
    c.check(c.run())


@pytest.mark.parametrize("pad,offset,heads", [(0, 0, (2, 2, 32, 64)), (3, 1, (1, 1, 32, 32)), (4, 4, (1, 3, 64, 32))])
def test_conv_backward_padding_gaps_and_strides(pad, offset, heads):
    c = Conv([60, 5, 0, 300, 2, 33], heads, skip=(1, 3), gap=9, tail=270, pad=pad, offset=offset,
             has_init=[1, 1, 0, 1, 0, 1], seed=3)
    for kw in (dict(), dict(activation=False), dict(d_window=False), dict(conv=False)):
        c.check(c.run(**kw), **kw)


def test_long_strips_equal_short_ones():
    """A batch large enough for strips of 57 and of 25 rows gives every row of dx and d_window0 the bits that the same
    sequence alone gives in shorter strips: a row's sums do not depend on where it lies."""
    g = gdn()
    lens = [1, 700, 0, 58, 57, 2, 3000, 115, 26, 900]
    for heads, ask in (((16, 32, 128, 128), 57), ((8, 16, 128, 128), 25)):
        c = Conv(lens, heads, act="bf16", ydt="bf16", seed=21)
        waves = lambda own: -(-c.rows // own) * -(-c.C // 256)
        assert (57 if waves(57) >= 2048 else 25 if waves(25) >= 2048 else 13) == ask
        out = c.run()
        for s, (r0, r1) in enumerate(c.spans):
            if r0 == r1:
                continue
            one = g.Batch(torch.tensor([0, r1 - r0], dtype=torch.int32, device=DEV), c.batch.page_idx[s:s + 1], None, 0,
                          r1 - r0)
            got = g.gdnt_conv_backward(c.dims, c.w, c.x[r0:r1], c.dy[r0:r1], one, g.ConvPool(c.win, None),
                                       d_window=torch.from_numpy(c.d_window[s:s + 1]).to(DEV))
            assert torch.equal(got.dx, out.dx[r0:r1]), s
            assert torch.equal(got.d_window0[0], out.d_window0[s]), s


def test_conv_backward_bad_batches():
    g = gdn()
    c = Conv([20, 20, 20], act="f32", seed=4)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = g.Batch(torch.tensor([0, 20, 40, 99], dtype=torch.int32, device=DEV), c.batch.page_idx, None, 0, c.rows)
    out = c.run(err=err, batch=b)
    assert int(err.item()) == g.GDN_DEVERR_BATCH
    c.spans[2] = None
    c.check(out)
    err.zero_()
    pages = c.batch.page_idx.clone()
    pages[1] = 5  # 5 pages: 0..4
    out = c.run(err=err, batch=g.Batch(c.batch.cu_seqlens, pages, None, 0, c.rows))
    assert int(err.item()) == g.GDN_DEVERR_PAGE
    c.spans = [(0, 20), None, (40, 60)]
    c.check(out)
    err.zero_()
    out = c.run(err=err, batch=g.Batch(c.batch.cu_seqlens, c.batch.page_idx, None, 19, c.rows))
    assert int(err.item()) == g.GDN_DEVERR_BATCH and float(out.d_conv_w.abs().sum()) == 0


def test_conv_backward_of_nothing():
    g = gdn()
    c = Conv([0, 0], act="f32", seed=5)
    out = c.run()
    assert float(out.d_conv_w.abs().sum()) == 0
    assert np.array_equal(host(out.d_window0), c.d_window.astype(np.float64))


@pytest.mark.parametrize("bits", [False, True])
def test_a_trainable_block(bits):
    """conv -> recurrence forward, then both backward passes, as a training step runs them, in fp32 against the
    oracle's formulas chained the same way."""
    g = gdn()
    c = Conv([45, 300, 1, 83], act="f32", ydt="f32", seed=9)
    C = c.C
    rng = np.random.default_rng(2)
    dims = g.ScanDims(C, act_dtype="f32", state_dtype="f32")
    a_log = np.log(rng.uniform(1, 16, C)).astype(np.float32)
    dt = np.log(np.expm1(np.exp(rng.uniform(np.log(0.02), np.log(0.5), C)))).astype(np.float32)
    params = g.ScanParams(torch.from_numpy(a_log).to(DEV), torch.from_numpy(dt).to(DEV))
    a, b, dh = (torch.from_numpy(rng.standard_normal((c.rows, C)).astype(np.float32)).to(DEV) for _ in range(3))
    conv = g.ConvPool.alloc(c.dims, c.n + 2, 4, DEV)
    conv.buf.copy_(c.win)
    y = g.gdn_conv_update(c.dims, c.w, c.x, c.batch, conv, y_dtype="f32")  # rolls conv.buf; c.win stays
    state0 = g.StatePool(torch.from_numpy(rng.standard_normal((c.n + 2, C)).astype(np.float32)).to(DEV))
    state = g.StatePool(state0.buf.clone())
    saved = g.ScanSaved.alloc(dims, c.rows, DEV, ckpt=bits)
    h = g.gdnt_scan_forward(dims, params, y, a, b, c.batch, state, saved=saved)
    xab = {} if bits else dict(x=y, a=a, b=b)
    gs = g.gdnt_scan_backward(dims, params, c.batch, state0, saved, dh, **xab)
    gc = g.gdnt_conv_backward(c.dims, c.w, c.x, gs.dx, c.batch, g.ConvPool(c.win, None))
    torch.cuda.synchronize()

    win = host(c.win)[c.pages, :3]
    h0 = host(state0.buf)[c.pages]
    yr, _ = ora.conv_forward(host(c.w), host(c.x), c.spans, win)
    hr, last, before = ora.scan(yr, host(a), host(b), a_log, dt, c.spans, h0)
    v = [yr, host(a), host(b)]
    if bits:
        # the integers are those of the fp32 y, which may round the other way than the oracle's: take the kernel's y
        v = [ora.stored(t, c.owned) for t in (host(y), host(a), host(b))]
        before = ora.rebuilt(*v, a_log, dt, c.spans, before)
    sr = ora.scan_backward(*v, a_log, dt, c.spans, before, host(dh), np.zeros((c.n, C)))
    cr = ora.conv_backward(host(c.w), host(c.x), sr["dx"], c.spans, win, np.zeros((c.n, 3, C)))
    # fp32 throughout: some hundred ulps, against the largest of each result
    for name, got, want in (("h", h, hr), ("da", gs.da, sr["da"]), ("d_a_log", gs.d_a_log, sr["d_a_log"]),
                            ("dx", gc.dx, cr["dx"]), ("d_conv_w", gc.d_conv_w, cr["d_conv_w"]),
                            ("d_state0", gs.d_state0, sr["d_state0"]), ("d_window0", gc.d_window0, cr["d_window0"]),
                            ("state", state.buf[torch.from_numpy(c.pages).long().to(DEV)], last)):
        assert np.abs(host(got) - want).max() <= 1000 * ULP * np.abs(want).max(), name


def test_conv_backward_replayed_from_a_graph():
    g = gdn()
    c = Conv([45, 0, 300, 3], act="bf16", ydt="bf16", seed=11)
    ws = torch.empty(g.gdnt_conv_workspace_bytes(c.dims, c.n, c.rows), dtype=torch.uint8, device=DEV)
    dwin = torch.from_numpy(c.d_window).to(DEV)
    pool = g.ConvPool(c.win, None)
    out = g.ConvGrads(torch.empty_like(c.x), torch.empty(c.C, 4, device=DEV), torch.empty(c.n, 3, c.C, device=DEV))
    step = lambda: g.gdnt_conv_backward(c.dims, c.w, c.x, c.dy, c.batch, pool, d_window=dwin, out=out, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        c.x.copy_(torch.randn(c.rows, c.C).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in out]
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w, t) for w, t in zip(want, out)), k
