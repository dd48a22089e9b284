"""Linear attention on whole numbers, where every product and sum is a number
of 24 bits and only the last rounding is left: outputs are equal to the exact
ones, bit for bit, and what is held in fewer bits on the way shows.  And, with
decays, how far bf16 outputs are off beyond the half step of their rounding."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, host
from linear_util import Case
from oracle import linear as ol
from train_util import DT

pytestmark = pytest.mark.gpu


def pairs(rng, rows, heads, d, lens, near):
    """Two tensors whose rows 2j and 2j + 1 of a sequence are: 1 and -1 at every
    place, or (near) 65 to 109 at the same 16 places of both tensors' heads and
    all but the same in both rows, 1 more or less at each."""
    shape = rows, heads, 2, d
    v = rng.choice([-1, 1], shape) if not near else rng.integers(65, 110, shape)
    r0 = 0
    for n in lens:
        a, b = v[r0:r0 + n - n % 2:2], v[r0 + 1:r0 + n:2]
        b[:] = a + rng.integers(-1, 2, a.shape) if near else -a
        r0 += n
    if near:
        v[..., rng.permutation(d)[16:]] = 0
    return v[:, :, 0], v[:, :, 1]


def fill(c, q, k, v, d_o, s0=None, d_state=None):
    for name, t in (("q", q), ("k", k), ("v", v), ("d_o", d_o)):
        c.t[name].copy_(torch.from_numpy(t.reshape(c.rows, -1).astype(np.float32)).to(DT[c.act]))
    c.g.zero_()
    c.s0 = torch.zeros(c.n + 2, c.hv, c.dk, c.dv) if s0 is None else torch.from_numpy(s0.astype(np.float32))
    c.d_state = np.zeros((c.n, c.hv, c.dk, c.dv), np.float32) if d_state is None else d_state.astype(np.float32)
    return c


def check_equal(c, with_dg=True, dg=False):
    """All outputs against the oracle's, whose whole numbers of up to 2^53 are exact."""
    q, k, v, g = c.inputs()
    ref, last = ol.attend(q, k, v, g, c.spans, c.seq_s0(), c.scale)
    grads = ol.attend_backward(q, k, v, g, c.spans, c.seq_s0(), c.scale, c.f64("d_o"), c.d_state, c.init)
    o, so = c.forward()
    got = c.backward(with_dg=with_dg)

    def same(name, t, want, dt):
        want = torch.from_numpy(np.ascontiguousarray(want.reshape(t.shape))).to(DT[dt]).to(DEV)
        assert torch.equal(t, want), f"{name}: {int((t != want).sum())} of {t.numel()}"

    same("o", o, ref, c.act)
    for s in range(c.n):
        if c.lens[s]:
            same("state", so.buf[c.pages[s]], last[s], "f32")
    for name in ("dq", "dk", "dv"):
        same(name, getattr(got, name), grads[name], c.act)
    same("d_state0", got.d_state0, grads["d_state0"], "f32")
    if dg and with_dg:
        same("dg", got.dg, grads["dg"], "f32")


WIDTHS = [(128, 128), (64, 64), (64, 128), (128, 64), (48, 104)]


@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_weights_of_18_bits(dk, dv, act, with_dg):
    """q.k, or v.d_o, is a number of up to 16 * 110^2 < 2^18 and much the same for
    two rows, which it weighs by 1 and -1; 64 of them are below 2^24, as is what
    the rows before leave."""
    lens = [63, 150, 1, 64]
    for big in ("qk", "v_do"):
        c = Case(lens, hk=1, hv=2, dk=dk, dv=dv, act=act, scale=1.0, pad=8)
        rng = np.random.default_rng(dk + dv)
        q, k = pairs(rng, c.rows, 1, dk, lens, big == "qk")
        v, d_o = pairs(rng, c.rows, 2, dv, lens, big == "v_do")
        check_equal(fill(c, q, k, v, d_o), with_dg)


@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_states_of_17_bits(dk, dv, act, with_dg):
    """States, and their gradients, of numbers up to 100000 in fours that all but
    cancel, read by rows whose values are 0 or 1 and alike in pairs: sums of 128
    of them stay below 2^24, and dg, a sum in 64 bits, is the rounded exact one."""
    rng = np.random.default_rng(dk * dv)
    lens = [5, 130, 64]
    c = Case(lens, hk=1, hv=2, dk=dk, dv=dv, act=act, scale=1.0)

    def fours(n):
        x = rng.integers(65536, 100000, (n, 2, dk // 2, dv // 2))
        less = lambda: rng.integers(0, 3, x.shape)  # noqa: E731
        m = np.empty((n, 2, dk, dv), np.int64)
        m[..., ::2, ::2], m[..., 1::2, ::2], m[..., ::2, 1::2], m[..., 1::2, 1::2] = x, -x + less(), -x + less(), x + less()
        return m

    def alike(h, d):
        few = rng.random((c.rows, h, d // 2)) < 0.3
        return np.repeat(few, 2, -1).astype(int)

    check_equal(fill(c, alike(1, dk), alike(1, dk), alike(2, dv), alike(2, dv), fours(c.n + 2), fours(c.n)), with_dg, dg=True)


@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_bf16_outputs_are_fp32_sums_rounded_once(dk, dv, with_dg):
    """Beyond the half step of its last rounding an output is off by no more
    than fp32 sums are.  A sum of n terms of random signs rounds n partial sums,
    of up to 3 root sums of squares r of its terms each, by up to a half step of
    2^-24: n^(1/2) 2^-24 * 3 r at random; n is at most 2 * 128 products of heads,
    64 rows, and 16 for decays and chunks: 3.3e-6 r, below 2^-18 r = 3.8e-6 r.
    A weight or a state held in 16 bits would be off by 2^-17 of every term."""
    lens = [400, 70, 1, 64]
    c = Case(lens, hk=1, hv=2, dk=dk, dv=dv, act="bf16", fast=0.05, seed=dk + dv)
    q, k, v, g = c.inputs()
    ref, _ = ol.attend(q, k, v, g, c.spans, c.seq_s0(), c.scale)
    r2, _ = ol.attend(q * q, k * k, v * v, 2 * g, c.spans, c.seq_s0() ** 2, c.scale ** 2)
    grads = ol.attend_backward(q, k, v, g, c.spans, c.seq_s0(), c.scale, c.f64("d_o"), c.d_state, c.init)
    grads2 = ol.attend_backward(q * q, k * k, v * v, 2 * g, c.spans, c.seq_s0() ** 2, c.scale ** 2, c.f64("d_o") ** 2,
                                c.d_state.astype(np.float64) ** 2, c.init)
    o, _ = c.forward()
    got = c.backward(with_dg=with_dg)
    for name, t, want, square in (("o", o, ref, r2), *((n, getattr(got, n), grads[n], grads2[n]) for n in ("dq", "dk", "dv"))):
        half = 2.0 ** (np.floor(np.log2(np.abs(want))) - 8)  # half a step of eight bits
        over = (np.abs(host(t).reshape(want.shape) - want) - half) / np.sqrt(square)
        assert over.max() <= 2.0 ** -18, (name, over.max())
