"""Head norms with the rotation by position on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
from oracle import linear as ol
from train_util import close, rounded

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, rows, hq=3, hk=2, d=64, rot=64, act="bf16", norm="rms", pairs="halves", pad=0, offset=0, far=100000,
                 weights=True, eps=1e-6, seed=0):
        rng = np.random.default_rng(seed)
        self.rows, self.hq, self.hk, self.d, self.rot, self.act = rows, hq, hk, d, rot, act
        self.norm, self.pairs, self.eps, self.pad, self.offset = norm, pairs, eps, pad, offset
        self.dims = gdn().RotateDims(hq, hk, d, rot, act_dtype=act, norm=norm, pairs=pairs, eps=eps)
        self.x = {t: self.strided(rounded(rng.standard_normal((rows, h * d)), act)) for t, h in (("q", hq), ("k", hk))}
        self.dy = {t: self.strided(rounded(rng.standard_normal((rows, h * d)), act)) for t, h in (("q", hq), ("k", hk))}
        w = lambda: torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(DEV)  # noqa: E731
        self.w = {"q": w(), "k": w()} if weights else {"q": None, "k": None}
        self.pos = torch.from_numpy(rng.integers(-far, far + 1, rows).astype(np.int32)).to(DEV)
        self.inv = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))).astype(np.float32)).to(DEV)

    def strided(self, v):
        rows, w = v.shape
        buf = torch.full((rows * (w + self.pad) + self.offset + 1,), float("nan"), dtype=v.dtype, device=DEV)
        out = buf[self.offset:self.offset + rows * (w + self.pad)].view(rows, w + self.pad)[:, :w]
        out.copy_(v.to(DEV))
        return out

    def args(self):
        return self.dims, self.x["q"], self.x["k"], self.w["q"], self.w["k"], self.pos, self.inv

    def heads(self, t):
        return host(t).reshape(self.rows, -1, self.d)

    # n = x root w is off by a few half steps: the sum of d squares by at most d
    # (in 16 partial sums d/16 + 4), the root and two products by six; the sine
    # and cosine by two ulps of 1 and the angle's fraction of a turn, in fp32, by
    # 2 pi 2^-25; |a| and |b| of a pair meet in both of its values.
    def tol(self):
        return (self.d / 16 + 32) * 2.0 ** -24

    def check(self, yq, yk):
        for t, y in (("q", yq), ("k", yk)):
            x = self.heads(self.x[t])
            w = np.ones(self.d) if self.w[t] is None else host(self.w[t])
            args = (host(self.pos), host(self.inv), self.rot, self.norm, self.pairs, self.eps)
            ref = ol.rotate(x, w, *args)
            size = np.abs(x / ol._size(x, self.norm, self.eps) * w)
            a, b = ol._pairs(self.rot, self.pairs)
            size[..., a] = size[..., b] = size[..., a] + size[..., b]
            close("y" + t, self.heads(y), ref, size, self.tol(), self.act)

    def check_backward(self, g):
        for t, dx, dw in (("q", g.dq, g.dwq), ("k", g.dk, g.dwk)):
            x, dy = self.heads(self.x[t]), self.heads(self.dy[t])
            w = np.ones(self.d) if self.w[t] is None else host(self.w[t])
            args = (host(self.pos), host(self.inv), self.rot, self.norm, self.pairs, self.eps)
            ref, ref_w = ol.rotate_backward(x, w, *args, dy)
            turned = np.abs(dy).copy()
            a, b = ol._pairs(self.rot, self.pairs)
            turned[..., a] = turned[..., b] = turned[..., a] + turned[..., b]
            root = 1 / ol._size(x, self.norm, self.eps)
            unit = np.abs(x) * root
            dn = turned * np.abs(w)
            along = (dn * unit).sum(-1, keepdims=True) / (self.d if self.norm == "rms" else 1)
            close("d" + t, self.heads(dx), ref, root * (dn + unit * along), 3 * self.tol(), self.act)
            if dw is not None:
                # fp32 within a lane: at most rows * heads / 16 terms of it, and 16 lanes
                terms = self.rows * x.shape[1] / 16 + 16
                close("dw" + t, host(dw), ref_w, (turned * unit).sum((0, 1)), self.tol() + terms * 2.0 ** -24, "f32")


SHAPES = [
    dict(rows=1), dict(rows=70, act="f32"), dict(rows=70, d=128, rot=128), dict(rows=5, d=256, rot=256), dict(rows=9, d=256, rot=64, act="f32"),
    dict(rows=33, d=80, rot=48, pairs="neighbours", norm="l2", act="f32"), dict(rows=33, d=80, rot=48, pairs="neighbours"),
    dict(rows=33, d=80, rot=36), dict(rows=20, d=2, rot=2, act="f32"), dict(rows=20, d=6, rot=4, pairs="neighbours"), dict(rows=7, d=62, rot=30),
    dict(rows=7, d=250, rot=250), dict(rows=7, d=64, rot=0), dict(rows=7, d=64, rot=0, act="f32", pairs="neighbours"),
    dict(rows=40, d=64, rot=32, pad=3, offset=1), dict(rows=40, d=64, rot=32, pad=4, offset=4, norm="l2"), dict(rows=40, d=64, rot=32, pad=1, offset=3, act="f32"),
    dict(rows=12, hq=40, hk=1), dict(rows=12, hq=0, hk=5), dict(rows=12, hq=5, hk=0, act="f32"), dict(rows=12, weights=False),
    dict(rows=12, far=2**31 - 1, act="f32"), dict(rows=5001, hq=2, hk=1, d=32, rot=16), dict(rows=4097, hq=1, hk=1, d=24, rot=24, act="f32"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[",".join(f"{k}={v}" for k, v in s.items()) for s in SHAPES])
def test_forward_and_backward(shape):
    g = gdn()
    c = Case(**shape)
    c.check(*g.gdnl_rotate_forward(*c.args()))
    c.check_backward(g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"]))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_in_place_and_without_weight_gradients(act):
    g = gdn()
    c = Case(50, act=act, pad=8)
    yq, yk = g.gdnl_rotate_forward(*c.args())
    want = g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"])
    out = g.RotateGrads(c.dy["q"], c.dy["k"], None, torch.empty(c.d, device=DEV))
    g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"], out=out)
    assert torch.equal(out.dq, want.dq) and torch.equal(out.dk, want.dk) and torch.equal(out.dwk, want.dwk)
    a, b = g.gdnl_rotate_forward(*c.args(), yq=c.x["q"], yk=c.x["k"])
    assert a is c.x["q"] and torch.equal(a, yq) and torch.equal(b, yk)


def test_heads_of_zeros_and_the_ends_of_the_range():
    g = gdn()
    for norm in ("rms", "l2"):
        c = Case(6, act="f32", norm=norm, eps=1e-6)
        clean = g.gdnl_rotate_forward(*c.args())
        c.x["q"][1, :64] = 0
        c.x["q"][2, 5] = float("nan")
        c.x["q"][3, 5] = float("inf")
        yq, yk = g.gdnl_rotate_forward(*c.args())
        d = g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"])
        assert (yq[1, :64] == 0).all() and torch.isfinite(d.dq[1]).all()
        assert torch.isnan(yq[2, :64]).all() and torch.isnan(yq[3, 5])
        same = torch.ones(6, 3 * 64, dtype=torch.bool)
        same[1:4, :64] = False
        assert torch.equal(yq[same.to(DEV)], clean[0][same.to(DEV)]) and torch.equal(yk, clean[1])
        assert torch.isfinite(d.dq[same.to(DEV)]).all() and torch.isfinite(d.dk).all()


def test_nothing_to_do():
    g = gdn()
    c = Case(0)
    yq, yk = g.gdnl_rotate_forward(*c.args())
    assert yq.shape == (0, 3 * 64) and yk.shape == (0, 2 * 64)
    d = g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"])
    assert (d.dwq == 0).all() and (d.dwk == 0).all()


def test_captured_on_another_stream():
    g = gdn()
    c = Case(300, d=128, rot=128)
    ws = torch.empty(g.gdnl_rotate_workspace_bytes(c.dims, c.rows), dtype=torch.uint8, device=DEV)
    yq, yk = g.gdnl_rotate_forward(*c.args())
    out = g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"], workspace=ws)

    def step():
        g.gdnl_rotate_forward(*c.args(), yq=yq, yk=yk)
        g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"], out=out, workspace=ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        c.x["q"].normal_()
        c.pos += 17
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (yq, yk, *out)]
        for t in (yq, yk, *out):
            t.zero_()
        ws.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((yq, yk, *out), want):
            assert torch.equal(a, b)


def test_rows_beyond_4_gb():
    g = gdn()
    dims = g.RotateDims(1, 1, 64, 64)
    rows, stride = 2300, 1 << 20
    buf = torch.empty(rows * stride, dtype=torch.bfloat16, device=DEV).view(rows, stride)
    q, k = buf[:, :64].normal_(), buf[:, 64:128].normal_()
    pos, inv = torch.arange(rows, dtype=torch.int32, device=DEV), torch.full((32,), 0.1, device=DEV)
    want = g.gdnl_rotate_forward(dims, q.contiguous(), k.contiguous(), None, None, pos, inv)
    got = g.gdnl_rotate_forward(dims, q, k, None, None, pos, inv, yq=q, yk=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
