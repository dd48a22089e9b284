"""Linear attention and the rotation at their edges: what is not finite in a
backward pass, heads near the ends of the number range, batches with bad bounds
cut into segments, strides that repeat a row."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
import test_gpu_rotate
from linear_util import Case
from oracle import linear as ol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("hk,hv", [(1, 2), (2, 2)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [150, 700])
def test_what_is_not_finite_shows_in_the_gradients(rows, act, hk, hv, with_dg):
    """An input that is not finite leaves its column of the gradients that it
    enters as a row not finite from its row on (dq), or up to it (dk, dv), asked
    for the decays' gradient or not, one value head to a key head or two."""
    at = 100
    for name, out, rest in (("k", "dq", slice(at, rows)), ("q", "dk", slice(0, at + 1)), ("d_o", "dv", slice(0, at + 1))):
        c = Case([rows, 20], hk=hk, hv=hv, act=act)
        clean = c.backward(with_dg=with_dg)
        c.t[name][at, 5] = float("nan")
        got = c.backward(with_dg=with_dg)
        assert not torch.isfinite(getattr(got, out)[rest, 5]).any(), (name, out)
        for a, b in zip(got[:3], clean[:3]):
            assert torch.equal(a[rows:], b[rows:])


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("shape", [dict(act="f32"), dict(), dict(act="f32", d=80, rot=36, pad=1), dict(d=250, rot=64, norm="l2"), dict(d=256, rot=256, norm="l2", act="f32")],
                         ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()) or "plain")
def test_heads_whose_squares_are_out_of_range(shape, eps):
    """The norm of a head is a number wherever the head's values are: rows times
    2^-100 to 2^120, gradients too, within the bounds of rows near 1."""
    g = gdn()
    c = test_gpu_rotate.Case(9, eps=eps, **shape)
    times = torch.tensor([2.0 ** e for e in (120, 100, 64, 60, 0, -45, -52, -70, -100)], device=DEV)[:, None]
    for t in ("q", "k"):
        c.x[t].copy_((c.x[t].float() * times).to(c.x[t].dtype))
    c.check(*g.gdnl_rotate_forward(*c.args()))
    c.check_backward(g.gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"]))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_heads_of_the_largest_and_the_smallest_numbers(act):
    """A head of 64 values m and -m has the root mean square m: 1 and -1 come out."""
    g = gdn()
    dt = torch.float32 if act == "f32" else torch.bfloat16
    dims = g.RotateDims(2, 0, 64, 0, act_dtype=act, eps=0.0)
    sign = torch.where(torch.arange(128, device=DEV) % 3 == 0, -1.0, 1.0)
    m = torch.tensor([torch.finfo(dt).max, torch.finfo(dt).tiny, 2.0 ** -133, 2.0 ** 61], device=DEV)[:, None]
    q = (sign * m).to(dt)
    y, _ = g.gdnl_rotate_forward(dims, q, q[:, :0], None, None, None, None)
    # the squares' sum, the root and two products: within 32 half steps of fp32
    assert (y.float() - sign).abs().max() <= (32 * 2.0 ** -24 if act == "f32" else 2.0 ** -8)
    none = torch.zeros(1, 128, dtype=dt, device=DEV)
    y, _ = g.gdnl_rotate_forward(g.RotateDims(2, 0, 64, 0, act_dtype=act, eps=1e-42), none, none[:, :0], None, None, None, None)
    assert (y == 0).all()


@pytest.mark.parametrize("d_state", [True, False])
@pytest.mark.parametrize("with_dg", [True, False])
@pytest.mark.parametrize("with_d_state0", [True, False])
def test_workspace_of_exactly_what_a_call_asks_for(d_state, with_dg, with_d_state0):
    """Each combination within its own size, filled with NaN, gives the bits of a
    call with room for any; half of what 128 rows need is refused."""
    g = gdn()
    c = Case([700, 0, 300, 70], hk=1, hv=2, dk=16, dv=24, act="bf16", fast=0.1)
    size = g.gdnl_attend_workspace_bytes(c.dims, c.n, c.rows, True, (with_dg, d_state, with_d_state0))
    most = g.gdnl_attend_workspace_bytes(c.dims, c.n, c.rows, True)
    assert size <= most

    def run(n_bytes):
        ws = torch.full((n_bytes + 256,), 255, dtype=torch.uint8, device=DEV)
        out = g.LinearGrads(*(torch.zeros_like(c.t[t]) for t in "qkv"), torch.zeros(c.rows, c.hv, device=DEV) if with_dg else None,
                            torch.zeros(c.n, c.hv, c.dk, c.dv, device=DEV) if with_d_state0 else None)
        g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"],
                               d_state=torch.from_numpy(c.d_state).to(DEV) if d_state else None, out=out, workspace=ws[:n_bytes])
        torch.cuda.synchronize()
        assert (ws[n_bytes:] == 255).all()
        return out

    for a, b in zip(run(size), run(most)):
        assert (a is None and b is None) or torch.equal(a, b)
    small = g.gdnl_attend_workspace_bytes(c.dims, c.n, 128, True, (with_dg, d_state, with_d_state0))
    with pytest.raises(g.GdnError):
        run(small // 2)


def test_decays_of_one_row_expanded_over_all():
    """A g [rows][heads] whose rows are one and the same memory has a gradient for every row."""
    g = gdn()
    c = Case([70, 3], decay="head", act="bf16", fast=0.1)
    one, rows = c.g, c.g.expand(c.rows, c.hv)
    want = {}
    for gates in (rows.contiguous(), rows):
        o = g.gdnl_attend_forward(c.dims, c.t["q"], c.t["k"], c.t["v"], gates, c.batch, g.StatePool(c.s0.to(DEV)))
        d = g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], gates, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"])
        assert d.dg.shape == (c.rows, c.hv)
        for n, t in {"o": o, **d._asdict()}.items():
            assert torch.equal(want.setdefault(n, t), t), n
    summed = g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], one, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"]).dg
    # the sum of rows rounded one by one: half a step each
    assert ((want["dg"].double().sum(0) - summed.double()).abs() <= 2.0 ** -24 * (want["dg"].double().abs().sum(0) + summed.double().abs())).all()


def test_angles_near_half_a_turn():
    """Values of 1 turned against 0 are cosine and sine of the angle, off by the
    library's two ulps and two roundings, six half steps of 2^-24 of themselves,
    where a sine is near 0 too: a fraction of a turn rounded to fp32 alone would
    be off by up to 2 pi 2^-26 whatever its size.  2^-45 is for the angle's own
    rounding in 64 bits, of up to 2^19 radians."""
    rows = 5000
    rng = np.random.default_rng(3)
    g = gdn()
    inv = np.array([np.pi, 1.0], np.float32)
    pos = rng.integers(-100000, 100000, rows).astype(np.int32)
    q = torch.zeros(rows, 4, device=DEV)
    q[:, :2] = 1.0  # pairs (0, 2) and (1, 3)
    y, _ = g.gdnl_rotate_forward(g.RotateDims(1, 0, 4, 4, act_dtype="f32", norm="l2", eps=0.0), q, q[:, :0], None, None,
                                 torch.from_numpy(pos).to(DEV), torch.from_numpy(inv).to(DEV))
    y = host(y) / float(np.float32(1.0) / np.sqrt(np.float32(2.0)))
    angle = pos[:, None].astype(np.float64) * inv.astype(np.float64)
    for got, want in ((y[:, :2], np.cos(angle)), (y[:, 2:], np.sin(angle))):
        assert (np.abs(got - want) <= 6 * 2.0 ** -24 * np.abs(want) + 2.0 ** -45).all(), np.abs(got - want).max() * 2 ** 24


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows,shape", [(1 << 20, dict(hq=8, hk=0, d=4)), (20000, dict(hq=3, hk=9, d=80, pairs="neighbours")), (20000, dict(hq=2, hk=2, d=256))])
def test_weights_gradients_over_many_rows(rows, act, shape):
    """The error of a weight's gradient does not grow with the rows beyond its
    terms' root sum of squares r.  A term dy x / |x| is off by four half steps of
    2^-24 at random, 4 / 3^(1/2); a sum of 32 of them in fp32 by a half step of
    each of its partial sums, of i^(1/2) terms: (32 / 2 / 3)^(1/2); together 3.3
    half steps of r in the norm, below 4.  Summed in fp32 throughout, 512 terms to
    a lane are off by (512 / 2 / 3)^(1/2) = 9."""
    c = test_gpu_rotate.Case(rows, act=act, rot=0, **shape)
    got = gdn().gdnl_rotate_backward(*c.args(), c.dy["q"], c.dy["k"])
    for t, dw in (("q", got.dwq), ("k", got.dwk)):
        x, dy = c.heads(c.x[t]), c.heads(c.dy[t])
        if x.shape[1] == 0:
            continue
        terms = dy * x / ol._size(x, c.norm, c.eps)
        off, r2 = host(dw) - terms.sum((0, 1)), (terms ** 2).sum((0, 1))
        assert np.sqrt((off ** 2).sum() / r2.sum()) <= 4 * 2.0 ** -24


def bad_batch(c, cu, pages=None, max_len=0):
    g = gdn()
    return g.Batch(torch.tensor(cu, dtype=torch.int32, device=DEV), c.batch.page_idx if pages is None else pages, None, max_len, c.rows)


def check_skipped(c, batch, bit, live, act_rows):
    """Sequences `live` as in the whole batch, bit for bit, and nothing of others
    written but zeros into d_state0; act_rows: rows that a live sequence owns."""
    good_o, good_s = c.forward()
    good = c.backward()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, so = c.forward(batch=batch, err=err)
    assert int(err.item()) == bit
    err.zero_()
    d = c.backward(batch=batch, err=err)
    assert int(err.item()) == bit
    mine = torch.zeros(c.rows, dtype=torch.bool)
    for r in act_rows:
        mine[r] = True
    mine = mine.to(DEV)
    for a, b in ((o, good_o), (d.dq, good.dq), (d.dk, good.dk), (d.dv, good.dv), (d.dg, good.dg)):
        assert torch.equal(a[mine], b[mine]) and torch.isnan(a[~mine]).all()
    pages = host(batch.page_idx).astype(int)
    for s in range(c.n):
        if s in live:
            assert torch.equal(so.buf[pages[s]].nan_to_num(3.0), good_s.buf[c.pages[s]].nan_to_num(3.0))
            assert torch.equal(d.d_state0[s], good.d_state0[s])
        else:
            assert (d.d_state0[s] == 0).all()
            if pages[s] < len(so.buf) and pages[s] >= 0:
                assert torch.isnan(so.buf[pages[s]]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_bad_bounds_beside_sequences_of_several_segments(act):
    """Sequences of three and more segments stay whole beside one whose bounds
    decrease, one that begins before an earlier one's end, one beyond the rows,
    and one whose page is beyond the pools."""
    g = gdn()
    lens = [400, 300, 500, 350]
    c = Case(lens, hk=1, hv=2, dk=16, dv=8, act=act, fast=0.1)
    rows = [slice(0, 400), slice(400, 700), slice(700, 1200), slice(1200, 1550)]
    for cu, live in (([0, 400, -2, 1200, 1550], (0, 3)),   # 1: negative end; 2: from -2 on
                     ([0, 400, 300, 1200, 1550], (0, 3)),  # 1: decreasing; 2: begins within 0
                     ([0, 400, 700, 1200, 1551], (0, 1, 2))):
        check_skipped(c, bad_batch(c, cu), g.GDN_DEVERR_BATCH, live, [rows[s] for s in live])
    pages = c.batch.page_idx.clone()
    pages[2] = 6  # the pools have 6
    check_skipped(c, bad_batch(c, [0, 400, 700, 1200, 1550], pages), g.GDN_DEVERR_PAGE, (0, 1, 3), [rows[s] for s in (0, 1, 3)])
    # longer than max_seqlen: the cut is that of sequences of up to 400 rows, as in a batch told so
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, _ = c.forward(batch=bad_batch(c, [0, 400, 700, 1200, 1550], max_len=400), err=err)
    assert int(err.item()) == g.GDN_DEVERR_BATCH and torch.isnan(o[rows[2]]).all()
    d = c.backward(batch=bad_batch(c, [0, 400, 700, 1200, 1550], max_len=400), err=err)
    assert torch.isnan(d.dq[rows[2]]).all() and (d.d_state0[2] == 0).all() and torch.isfinite(d.dq[rows[3]]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 300])
def test_bad_bounds_among_more_sequences_than_one_launch_places(act, rows):
    """More than 256 sequences: segments and decays are two launches, a thread finds a slot's segment."""
    g = gdn()
    n = 300
    lens = [2] * n
    lens[40], lens[299] = rows, rows
    c = Case(lens, hk=1, hv=2, dk=8, dv=8, act=act, fast=0.1)
    cu = [int(v) for v in host(c.batch.cu_seqlens)]
    starts = list(cu)
    cu[101] = 0  # 100 decreases, 101 begins before the end of 99
    live = [s for s in range(n) if s not in (100, 101)]
    check_skipped(c, bad_batch(c, cu), g.GDN_DEVERR_BATCH, live, [slice(starts[s], starts[s + 1]) for s in live])


def test_states_in_place_of_cut_sequences():
    """A cut sequence's first segment takes the page as it was, whatever the last one has written by then."""
    c = Case([1300, 70, 900, 257], hk=1, hv=2, dk=32, dv=32, act="bf16", fast=0.01)
    want_o, want_s = c.forward()
    for _ in range(5):
        o, so = c.forward(in_place=True)
        assert torch.equal(o, want_o)
        for s in range(c.n):
            assert torch.equal(so.buf[c.pages[s]], want_s.buf[c.pages[s]])
