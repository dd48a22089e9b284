"""GPU tests of include/gdn_train.h at the ends of the number range: the
lowest and the largest finite numbers, infinities and NaNs, in every input,
against the float64 oracle (oracle/train.py) and against the same call
without them."""
import numpy as np
import pytest
import torch

import oracle.train as ora
from gpu_util import DEV, gdn, host
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
