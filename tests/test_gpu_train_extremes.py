"""GPU tests of include/gdn_train.h at the ends of the number range: the
lowest and the largest finite numbers, infinities and NaNs, in every input,
against the float64 oracle (oracle/train.py) and against the same call
without them."""
import numpy as np
import pytest
import torch

import oracle.train as ora
from gpu_util import DEV, gdn, host
from test_gpu_conv_backward import Conv
from test_gpu_scan import decode
from train_util import DT, Case, check_forward, check_grads

pytestmark = pytest.mark.gpu


def largest(act, sign):
    return sign * torch.finfo(DT[act]).max


def check_step(c, ckpt=False):
    """Forward and backward against the oracle, from the activations or at the values the 8 bits stand for."""
    saved = c.saved(ckpt=ckpt)
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    out = c.backward(saved, from_ckpt=ckpt)
    if not ckpt:
        check_grads(c, out, ora)
        return
    v, _, _ = decode(c, saved)
    assert np.isfinite(v[:, c.owned]).all()
    with np.errstate(invalid="ignore", over="ignore"):
        before = ora.scan(c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans, c.seq_h0())[2]
        rb = ora.rebuilt(v[0], v[1], v[2], c.a_log, c.dt_bias, c.spans, before)
    check_grads(c, out, ora, x=v[0], a=v[1], b=v[2], before=rb)


@pytest.mark.parametrize("C", [64, 66])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_products_with_the_largest_x(act, C):
    """lambda x beta (1 - beta) is in range where lambda x beta is not."""
    c = Case([300, 290], C, act, "f32", seed=62)
    for r, ch, end in ((5, 2, 300), (303, C - 1, 590)):
        c.t["x"][r, ch] = largest(act, 1)
        c.t["b"][r, ch] = 0.875
        c.t["dh"][r, ch] = 2.0
        # nothing behind the row, so that only db meets the large state
        c.t["dh"][r + 1:end, ch] = 0.0
        c.d_state[int(r > 299), ch] = 0.0
    check_step(c)


@pytest.mark.parametrize("C", [64, 66])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name,sign", [("x", -1), ("x", 1), ("a", -1), ("b", -1), ("b", 1)])
def test_checkpoint_of_the_largest_numbers(name, sign, act, C):
    """The lowest and the largest number of the type in 8 bits: its block's other values are stored as zeros, all of
    them finite, and the gradients are those at the stored values (64 channels: whole tiles loaded ahead in bf16)."""
    c = Case([300, 290], C, act, "f32", seed=61)
    for r, ch in ((5, 2), (200, 33), (303, C - 1)):
        c.t[name][r, ch] = largest(act, sign)
        if name == "x":
            c.t["b"][r, ch] = -60.0  # an update of 3e12, so that h and what follows from it stay in range
    check_step(c, True)


def nan_of(dt, sign):
    """A quiet NaN of the type with its sign bit as asked."""
    if dt == torch.bfloat16:
        return torch.tensor([0x7FC0 - (1 << 15 if sign < 0 else 0)], dtype=torch.int16).view(dt)[0]
    return torch.tensor([0x7FC00000 - (1 << 31 if sign < 0 else 0)], dtype=torch.int32).view(dt)[0]


def put(c, name, rows, channels, value):
    """`value` at the given places of one input of c; parameters and states have a channel alone to place it in."""
    for ch in channels:
        if name == "state":
            c.h0[int(c.pages[1]), ch] = value
        elif name in ("a_log", "dt_bias"):
            getattr(c.params, name)[ch] = value
            getattr(c, name)[ch] = float(value)
        elif name == "d_state":
            c.d_state[1, ch] = float(value)
        else:
            for r in rows:
                c.t[name][r, ch] = value


def same(p, q):
    """Bit for bit, NaNs for NaNs."""
    p, q = p.detach().cpu(), q.detach().cpu()
    return bool(((p == q) | (torch.isnan(p) & torch.isnan(q))).all())


def results(c, ckpt):
    saved = c.saved(ckpt=ckpt)
    h, _, so = c.forward(saved)
    return h, so.buf, saved.states, *c.backward(saved, from_ckpt=ckpt)


# The tiles of the forward pass are 128 rows, a wave's 16: the second sequence begins at row 200, inside a tile that
# goes on from the first one and in the same 16 rows as row 203, and goes on into the next tiles; 300 and 410 lie in
# tiles without a first row.
NAN_LENS, NAN_ROWS = [200, 400, 90], (203, 300, 410)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "a", "b", "a_log", "dt_bias", "state", "dh", "d_state"])
def test_a_nan_stays_in_its_sequence_and_channel(name, act, sign):
    """Everything else keeps its bits; in the channel itself NaNs stand where the formulas have them, both ways."""
    C, channels = 72, (6, 33, 70)
    where = (203,) if sign > 0 else (300,)
    for rows in (where, NAN_ROWS):
        c, clean = (Case(NAN_LENS, C, act, "f32", seed=63) for _ in range(2))
        put(c, name, rows, channels, nan_of(DT[act] if name in ("x", "a", "b", "dh") else torch.float32, sign))
        rest = [k for k in range(C) if k not in channels]
        for got, want in zip(results(c, False), results(clean, False)):
            assert same(got[..., rest], want[..., rest])
        saved = c.saved()
        h, _, so = c.forward(saved)
        check_forward(c, h, so, ora)
        check_grads(c, c.backward(saved), ora)


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("C", [64, 66])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_the_largest_decay_gates(act, C, ckpt):
    """a at the largest number forgets the state: every gradient is a number, d_a_log (0 times a g beyond fp32) too."""
    c = Case([300, 290], C, act, "f32", seed=64)
    for r, ch in ((5, 2), (200, 33), (303, C - 1)):
        c.t["a"][r, ch] = largest(act, 1)
    check_step(c, ckpt)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_infinite_gates_are_their_limits(act):
    """An infinite a or b gives what a gate far out gives, bit for bit, in h, the states and every gradient."""
    far, inf = (Case([300, 290], 72, act, "f32", seed=65) for _ in range(2))
    for name, r, ch, sign in (("a", 5, 2, 1), ("a", 203, 33, -1), ("b", 300, 8, 1), ("b", 400, 71, -1)):
        far.t[name][r, ch] = 1e6 * sign
        inf.t[name][r, ch] = float("inf") * sign
    for p, q in zip(results(far, False), results(inf, False)):
        assert same(p, q)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "a", "b", "dh"])
def test_a_nan_in_8_bits_stays_in_its_blocks(name, act):
    """16 rows by 4 channels of NaNs (dh is not stored: itself alone); all other channels keep their bits, and in these
    NaNs stand where the formulas at the stored values have them."""
    C = 72
    c, clean = (Case(NAN_LENS, C, act, "f32", seed=66) for _ in range(2))
    put(c, name, NAN_ROWS, (6, 33), nan_of(DT[act], 1))
    touched = [6, 33] if name == "dh" else [4, 5, 6, 7, 32, 33, 34, 35]
    rest = [k for k in range(C) if k not in touched]
    for got, want in zip(results(c, True), results(clean, True)):
        assert same(got[..., rest], want[..., rest])
    saved = c.saved(ckpt=True)
    c.forward(saved)
    v, _, _ = decode(c, saved)
    out = c.backward(saved, from_ckpt=True)
    with np.errstate(invalid="ignore"):
        before = ora.scan(c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans, c.seq_h0())[2]
        rb = ora.rebuilt(v[0], v[1], v[2], c.a_log, c.dt_bias, c.spans, before)
        ref = ora.scan_backward(v[0], v[1], v[2], c.a_log, c.dt_bias, c.spans, rb, c.f64("dh"), c.d_state, c.init)
    for k, r in ref.items():
        assert np.array_equal(np.isnan(host(getattr(out, k))), np.isnan(r)), k


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "a", "b", "a_log", "dt_bias", "state", "dh", "d_state"])
def test_an_infinity_stays_in_its_sequence_and_channel(name, act):
    """Every other channel, and every other sequence of the channel, keeps its bits, forward and backward."""
    C, channels = 72, (6, 33, 70)
    for value in (float("inf"), float("-inf")):
        c, clean = (Case(NAN_LENS, C, act, "f32", seed=67) for _ in range(2))
        put(c, name, NAN_ROWS, channels, value)
        rest = [k for k in range(C) if k not in channels]
        got, want = results(c, False), results(clean, False)
        for p, q in zip(got, want):
            assert same(p[..., rest], q[..., rest])
        if name in ("a_log", "dt_bias"):
            continue
        other = [r for r in range(c.rows) if not 200 <= r < 600]
        for k in (0, 3, 4, 5):  # h, dx, da, db
            assert same(got[k][other], want[k][other])
        page = int(c.pages[0]), int(c.pages[2])
        assert same(got[1][list(page)], want[1][list(page)]) and same(got[-1][[0, 2]], want[-1][[0, 2]])


def test_an_infinite_gradient_is_the_formulas():
    """dh infinite at one row: what it reaches is infinite with the formulas' signs, or NaN where they have Inf - Inf
    and 0 Inf."""
    c = Case([300, 20], 64, "f32", "f32", seed=68)
    c.t["dh"][150, 7], c.t["dh"][310, 8] = float("inf"), float("-inf")
    saved = c.saved()
    c.forward(saved)
    out = c.backward(saved)
    with np.errstate(invalid="ignore", over="ignore"):
        args = (c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans)
        ref = ora.scan_backward(*args, ora.scan(*args, c.seq_h0())[2], c.f64("dh"), c.d_state, c.init)
    for k, r in ref.items():
        got = host(getattr(out, k))
        assert np.array_equal(np.isnan(got), np.isnan(r)) and np.array_equal(got[np.isinf(r)], r[np.isinf(r)]), k
        assert np.isfinite(got[np.isfinite(r)]).all(), k


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "a", "b", "a_log", "dt_bias", "state"])
def test_a_nan_in_the_one_launch_form(name, act):
    """At most 8 rows a sequence, one launch: rows, sequences and channels as above."""
    g = gdn()
    c, clean = (Case([1, 8, 0, 3, 7], 72, act, "f32", seed=69) for _ in range(2))
    put(c, name, (4,), (6, 33, 71), nan_of(DT[act] if name in ("x", "a", "b") else torch.float32, -1))
    rest = [k for k in range(72) if k not in (6, 33, 71)]
    few = lambda c: c.forward(batch=g.Batch(c.batch.cu_seqlens, c.batch.page_idx, None, 8, c.rows))
    (h, _, so), (h2, _, so2) = few(c), few(clean)
    assert same(h[:, rest], h2[:, rest]) and same(so.buf[:, rest], so2.buf[:, rest])
    check_forward(c, h, so, ora)


# ------------------------------------------------------------------------ conv


CONV_LENS = [70, 1, 200, 2, 60]  # the third from row 71 to 270


@pytest.mark.parametrize("act,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("name", ["x", "dy", "w", "window", "d_window"])
def test_conv_nan_stays_in_its_sequence_and_channel(name, act, ydt):
    """NaN at a sequence's first, middle and last rows: NaNs where the formulas have them, all else in its bounds, the
    other channels bit for bit; infinities change no other channel and no other sequence."""
    C = 96
    for value in (float("nan"), float("inf"), float("-inf")):
        c, clean = (Conv(CONV_LENS, act=act, ydt=ydt, seed=70) for _ in range(2))
        channels = (6, 33, 95)
        for ch, row in zip(channels, (71, 130, 270)):
            if name == "w":
                c.w[ch, 1] = value
            elif name == "window":
                c.win[int(c.pages[2]), 1, ch] = value
            elif name == "d_window":
                c.d_window[2, 1, ch] = value
            else:
                getattr(c, name)[row, ch] = value
        out, ref = c.run(), clean.run()
        rest = [k for k in range(C) if k not in channels]
        assert same(out.dx[:, rest], ref.dx[:, rest]) and same(out.d_conv_w[rest], ref.d_conv_w[rest])
        assert same(out.d_window0[..., rest], ref.d_window0[..., rest])
        if name != "w":
            other = [r for r in range(c.rows) if not 71 <= r <= 270]
            assert same(out.dx[other], ref.dx[other])
            assert same(out.d_window0[[0, 1, 3, 4]], ref.d_window0[[0, 1, 3, 4]])
        if value != value:
            c.check(out)


def test_conv_backward_far_out():
    """z at the ends of the range: silu' is 0 or 1 there, and nothing becomes NaN."""
    c = Conv([40, 300], act="f32", ydt="f32", seed=72)
    c.x[10:14, :8] = 1e30
    c.x[60:64, 8:16] = -1e30
    c.x[200, 16:24] = 90.0
    c.x[210, 24:32] = -90.0
    out = c.run()
    assert all(bool(torch.isfinite(t).all()) for t in out)
