"""Linear attention on the GPU against the fp64 oracle: chunks and single rows,
forward and backward, at the sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
from linear_util import HALF32, Case

pytestmark = pytest.mark.gpu

LENS = [0, 1, 63, 64, 65, 0, 130, 17]
SHAPES = [
    dict(),
    dict(act="bf16"),
    dict(dk=128, dv=128, hk=1, hv=2, act="bf16"),
    dict(dk=128, dv=128, hk=1, hv=1),
    dict(dk=40, dv=72, hk=1, hv=3, act="bf16", state="bf16"),
    dict(dk=72, dv=24, hk=3, hv=3, decay="head"),
    dict(dk=64, dv=128, hk=1, hv=2, decay="head", act="bf16"),
    dict(dk=1, dv=1, hk=1, hv=1),
    dict(dk=13, dv=7, hk=1, hv=2, act="bf16"),
    dict(dk=31, dv=33, hk=1, hv=1, pad=3, offset=1),
    dict(dk=48, dv=16, pad=5, offset=3, act="bf16"),
    dict(dk=16, dv=80, pad=8, offset=8, act="bf16", scale=-2.0),
    dict(fast=60.0, act="bf16"),
    dict(fast=60.0),
    dict(fast=0.0),
    dict(skip=(3,), gap=5, tail=9, has_init=[1, 0, 1, 0, 1, 0, 0, 1], act="bf16"),
]
IDS = [",".join(f"{k}={v}" for k, v in s.items()) or "plain" for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    c = Case(LENS, **shape)
    o, so = c.forward()
    c.check_forward(o, so)
    o2, so2 = c.forward(in_place=True)
    assert torch.equal(o.nan_to_num(7.0), o2.nan_to_num(7.0))
    for s, sp in enumerate(c.spans):
        if sp and sp[1] > sp[0]:
            assert torch.equal(so.buf[c.pages[s]], so2.buf[c.pages[s]])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    c = Case(LENS, **shape)
    c.check_backward(c.backward())


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_backward_without_the_optional_parts(act):
    c = Case([70, 3], act=act, decay="head")
    full = c.backward(d_state=False)
    c.check_backward(full, d_state=False)
    less = c.backward(d_state=False, with_dg=False)
    assert less.dg is None
    c.check_backward(less, d_state=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["row", "head"])
def test_several_segments(act, decay):
    """Long sequences are cut into segments whose states are joined."""
    c = Case([1300, 256, 0, 1100, 5], hk=1, hv=2, dk=40, dv=24, act=act, decay=decay, fast=0.1)
    o, so = c.forward()
    c.check_forward(o, so)
    o, so2 = c.forward(in_place=True)
    c.check_forward(o, None)
    c.check_backward(c.backward())
    c.check_backward(c.backward(d_state=False), d_state=False)


def test_several_segments_with_padding_and_fresh_states():
    c = Case([300, 290, 1100], hk=1, hv=1, dk=16, dv=16, skip=(1,), gap=3, tail=4, has_init=[0, 1, 1], act="bf16", fast=0.05)
    o, so = c.forward()
    c.check_forward(o, so)
    c.check_backward(c.backward())


SHORT = [
    dict(dk=128, dv=128, hk=1, hv=2, act="bf16"),
    dict(dk=40, dv=72, hk=1, hv=3, act="bf16", state="bf16"),
    dict(dk=31, dv=33, hk=1, hv=1, pad=3, offset=1),
    dict(dk=48, dv=16, hk=1, hv=2, pad=5, offset=3, act="bf16"),
    dict(dk=72, dv=24, hk=3, hv=3, decay="head"),
    dict(fast=60.0, act="bf16"),
    dict(skip=(2,), gap=5, tail=9, has_init=[1, 0, 1, 0], act="bf16", fast=0.02),
]


@pytest.mark.parametrize("shape", SHORT, ids=[",".join(f"{k}={v}" for k, v in s.items()) for s in SHORT])
def test_short_segments(shape):
    """Few sequences and heads: cut from 513 rows on."""
    c = Case([513, 0, 128, 640], **{"fast": 0.3, **shape})
    o, so = c.forward()
    c.check_forward(o, so)
    c.check_backward(c.backward())


@pytest.mark.parametrize("rows", [1025, 17000])
def test_many_segments(rows):
    """More segments than a wave, and than a workgroup, joins in a round."""
    c = Case([rows, 3], hk=1, hv=1, dk=8, dv=8, fast=0.01)
    o, so = c.forward()
    c.check_forward(o, so)
    c.check_backward(c.backward())


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[70, 300], [700, 1100]])
def test_gate_gradients_end_at_the_initial_state(act, lens):
    """The first decay's gradient is <S_0, d_state0>: its walk is held there.

    Both are sums over d_k d_v products in 64 bits, so what is left is the
    rounding of the result, and 2^-40 of the absolute sums for that of the
    walk.  It is 0 where the sequence begins with zeros, and the same whether
    d_state0 is asked for or not."""
    g = gdn()
    c = Case(lens, act=act, has_init=[1, 0], fast=0.1)
    got = c.backward()
    first = int(host(c.batch.cu_seqlens)[0]), int(host(c.batch.cu_seqlens)[1])
    s0, d0 = c.s0.double().numpy()[c.pages[0]], host(got.d_state0)[0]
    want, size = (s0 * d0).sum((1, 2)), np.abs(s0 * d0).sum((1, 2))
    assert (np.abs(host(got.dg)[first[0]] - want) <= HALF32 * np.abs(want) + 2.0 ** -40 * (size + np.abs(host(got.dg)).max())).all()
    assert (np.abs(host(got.dg)[first[1]]) <= 2.0 ** -40 * np.abs(host(got.dg)).max()).all()
    bare = g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, c.batch, g.StatePool(c.s0.to(DEV)), c.t["d_o"],
                                  d_state=torch.from_numpy(c.d_state).to(DEV),
                                  out=g.LinearGrads(c.blank("q"), c.blank("k"), c.blank("v"), torch.zeros_like(got.dg), None))
    torch.cuda.synchronize()
    assert bare.d_state0 is None and torch.equal(bare.dg, got.dg)


@pytest.mark.parametrize("rows", [1, 3, 8])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_few_rows(shape, rows):
    """max_seqlen up to 8: row by row, in place and from one pool to another."""
    shape = {k: v for k, v in shape.items() if k not in ("skip", "has_init")}
    c = Case([1, rows, 0, rows, 1], max_len=rows, skip=(3,), has_init=[1, 1, 1, 1, 0], **shape)
    o, so = c.forward()
    c.check_forward(o, so)
    o2, so2 = c.forward(in_place=True)
    assert torch.equal(o.nan_to_num(7.0), o2.nan_to_num(7.0))


def test_a_prompt_then_single_rows_is_one_sequence():
    g = gdn()
    c = Case([150], dk=64, dv=64, hk=1, hv=2)
    whole, so = c.forward()
    pool = g.StatePool(c.s0.to(DEV).clone())
    b = lambda r0, r1, n: g.Batch(torch.tensor([r0, r1], dtype=torch.int32, device=DEV), c.batch.page_idx, None, n, 150)  # noqa: E731
    o = torch.zeros_like(whole)
    g.gdnl_attend_forward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, b(0, 100, 0), pool, o=o)
    for r in range(100, 150):
        g.gdnl_attend_forward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, b(r, r + 1, 1), pool, o=o)
    c.check_forward(o, None)
    p = c.pages[0]
    # both are within the bound of the exact state, whose size random signs leave far below its bound
    assert (pool.buf[p] - so.buf[p]).abs().max() <= 2 * c.tol() * 150 * so.buf[p].abs().max()


# ------------------------------------------------------------------ refusals


@pytest.mark.parametrize("max_len", [0, 5])
def test_bad_sequences_are_skipped_and_told(max_len):
    g = gdn()
    c = Case([4, 4, 4, 4], max_len=max_len, act="bf16")
    good, _ = c.forward()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cases = [([0, 4, 8, 12, 17], None, g.GDN_DEVERR_BATCH, [0, 1, 2]),      # beyond n_rows
             ([0, 4, -2, 12, 16], None, g.GDN_DEVERR_BATCH, None),
             ([0, 4, 8, 12, 16], 2, g.GDN_DEVERR_PAGE, [0, 1, 3])]
    for cu, far, bit, live in cases:
        pages = c.batch.page_idx.clone()
        if far is not None:
            pages[far] = 6  # the pools have 6
        err.zero_()
        b = g.Batch(torch.tensor(cu, dtype=torch.int32, device=DEV), pages, None, max_len, 16)
        o, so = c.forward(batch=b, err=err)
        assert int(err.item()) == bit
        c.backward(batch=b, err=err)
        assert int(err.item()) == bit
        if live is not None:
            for s in range(4):
                rows = slice(4 * s, 4 * s + 4)
                assert torch.equal(o[rows], good[rows]) if s in live else torch.isnan(o[rows]).all()
    if max_len:
        err.zero_()
        b = g.Batch(torch.tensor([0, 4, 10, 12, 16], dtype=torch.int32, device=DEV), c.batch.page_idx, None, max_len, 16)
        o, _ = c.forward(batch=b, err=err)
        assert int(err.item()) == g.GDN_DEVERR_BATCH and torch.isnan(o[4:10]).all() and torch.equal(o[:4], good[:4])


def test_gradients_of_skipped_and_empty_sequences():
    c = Case([70, 0, 5, 0], skip=(2, 3), has_init=[1, 0, 1, 1])
    d = c.backward()
    assert torch.equal(d.d_state0[1].cpu(), torch.from_numpy(c.d_state[1]))  # handed through, whatever has_init says
    assert (d.d_state0[2:] == 0).all()
    d = c.backward(d_state=False)
    assert (d.d_state0[1:] == 0).all()


# ------------------------------------------------------------------ extremes


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows,max_len", [(100, 0), (8, 8), (700, 0)])
def test_a_decay_of_zero_begins_anew(act, rows, max_len):
    for low in (-np.inf, -1e30, -200.0):
        c = Case([rows], act=act, max_len=max_len, fast=0.3)
        c.g[3] = low
        c.g[rows - 2, 1] = low
        c.g[0, 2] = low
        o, so = c.forward()
        c.check_forward(o, so)
        if max_len == 0:
            dead = host(c.g) < -128
            c.check_backward(c.backward(), dead=dead)
            assert (c.backward().dg.cpu().numpy()[dead] == 0).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "max"])
@pytest.mark.parametrize("rows,max_len", [(150, 0), (8, 8), (700, 0)])
def test_what_is_not_finite_reaches_its_column_from_its_row_on(act, bad, rows, max_len):
    at = 100 if rows > 100 else 4
    clean = Case([rows, 20 if not max_len else 5], act=act, max_len=max_len)
    o0, so0 = clean.forward()
    value = torch.finfo(clean.t["v"].dtype).max if bad == "max" else bad
    c = Case([rows, 20 if not max_len else 5], act=act, max_len=max_len)
    c.t["v"][at, 2 * c.dv + 5] = value
    o, so = c.forward()
    hurt = torch.zeros_like(o0, dtype=torch.bool)
    hurt[at:rows, 2 * c.dv + 5] = True
    assert torch.equal(o[~hurt], o0[~hurt])
    page = c.pages[0]
    col = so.buf[page, 2, :, 5]
    if bad != "max":  # the largest number may stay one
        assert not torch.isfinite(o[hurt]).any() and not torch.isfinite(col).any()
    keep = torch.ones_like(so.buf, dtype=torch.bool)
    keep[page, 2, :, 5] = False
    assert torch.equal(so.buf[keep].nan_to_num(3.0), so0.buf[keep].nan_to_num(3.0))
    # in k: the row of the state, every column of o from that row on; in q: that row alone
    c = Case([rows, 20 if not max_len else 5], act=act, max_len=max_len)
    c.t["k"][at, 3] = value
    o, _ = c.forward()
    assert torch.equal(o[:at], o0[:at]) and torch.equal(o[rows:], o0[rows:])
    c = Case([rows, 20 if not max_len else 5], act=act, max_len=max_len)
    c.t["q"][at, 3] = value
    o, so = c.forward()
    assert torch.equal(o[:at], o0[:at]) and torch.equal(o[at + 1:], o0[at + 1:])
    assert torch.equal(so.buf.nan_to_num(3.0), so0.buf.nan_to_num(3.0))
    c = Case([rows, 20 if not max_len else 5], act=act, max_len=max_len)
    c.g[at, 1] = float("nan")
    o, so = c.forward()
    assert torch.equal(o[:at], o0[:at]) and torch.equal(o[rows:], o0[rows:])
    h = slice(c.dv, 2 * c.dv)
    assert torch.isnan(o[at:rows, h]).all()
    if not max_len:  # never into another sequence
        d, d0 = c.backward(), clean.backward()
        for a, b in zip(d[:4], d0[:4]):
            assert torch.equal(a[rows:], b[rows:])
        assert torch.equal(d.d_state0[1], d0.d_state0[1])


# ------------------------------------------------- streams, graphs, big offsets


def test_on_another_stream_and_twice_at_once():
    c, d = Case([1300, 70], act="bf16", dk=64, dv=64), Case([5, 1400], act="bf16", dk=64, dv=64, seed=5)
    want = [x.forward()[0] for x in (c, d)], [x.backward() for x in (c, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = gdn()
    got = []
    for x, s in zip((c, d), streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o = x.blank("v")
            pool = g.StatePool(x.s0.to(DEV).clone())
            ds = torch.from_numpy(x.d_state).to(DEV)
            g.gdnl_attend_forward(x.dims, x.t["q"], x.t["k"], x.t["v"], x.g, x.batch, pool,
                                  g.StatePool(torch.empty_like(pool.buf)), o=o)
            got.append((o, g.gdnl_attend_backward(x.dims, x.t["q"], x.t["k"], x.t["v"], x.g, x.batch, pool, x.t["d_o"],
                                                  d_state=ds)))
    torch.cuda.synchronize()
    for (o, grads), o0, grads0 in zip(got, *want):
        assert torch.equal(o, o0)
        for a, b in zip(grads, grads0):
            assert torch.equal(a, b)


@pytest.mark.parametrize("max_len", [0, 2])
def test_captured_and_replayed(max_len):
    """One capture serves other lengths, pages and values; each replay is the eager result."""
    g = gdn()
    c = Case([1, 2, 1] if max_len else [1300, 2, 90], act="bf16", dk=64, dv=64, max_len=max_len)
    pool, so = g.StatePool(c.s0.to(DEV).clone()), g.StatePool(torch.zeros_like(c.s0.to(DEV)))
    o, ds = torch.zeros_like(c.t["v"]), torch.from_numpy(c.d_state).to(DEV)
    ws = torch.empty(g.gdnl_attend_workspace_bytes(c.dims, c.n, c.rows, backward=True), dtype=torch.uint8, device=DEV)
    grads = c.backward(workspace=ws)

    def step():
        g.gdnl_attend_forward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, c.batch, pool, so, o=o, workspace=ws)
        if not max_len:
            g.gdnl_attend_backward(c.dims, c.t["q"], c.t["k"], c.t["v"], c.g, c.batch, pool, c.t["d_o"], d_state=ds,
                                   out=grads, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        c.t["v"].normal_()
        cu = [[0, 1, 3, 4], [0, 2, 3, 4], [0, 0, 1, 3]][k] if max_len else [[0, 1300, 1302, 1392], [0, 10, 1300, 1301], [0, 0, 1390, 1392]][k]
        c.batch.cu_seqlens.copy_(torch.tensor(cu, dtype=torch.int32))
        for t in (o, so.buf, *grads):
            t.zero_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (o, so.buf, *grads)]
        for t in (o, so.buf, *grads):
            t.zero_()
        ws.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o, so.buf, *grads), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("max_len", [0, 1])
def test_rows_beyond_4_gb(max_len):
    """Packed rows whose byte offsets pass 32 bits, at both ends of the tensor."""
    g = gdn()
    dims = g.LinearDims(1, 1, 16, 16, act_dtype="bf16")
    stride, rows = 1 << 20, 2300
    buf = torch.empty(rows * stride, dtype=torch.bfloat16, device=DEV).view(rows, stride)
    q, k, v, o = (buf[:, j * 64:j * 64 + 16] for j in range(4))
    for t in (q, k, v):
        t.normal_()
    n = 1 if max_len else 70
    cu = torch.tensor([0, n, rows - n, rows], dtype=torch.int32, device=DEV)
    gates = torch.full((1,), -0.1, device=DEV)
    pool = g.StatePool(torch.zeros(3, 1, 16, 16, device=DEV))
    pages = torch.tensor([0, -1, 2], dtype=torch.int32, device=DEV)
    g.gdnl_attend_forward(dims, q, k, v, gates, g.Batch(cu, pages, None, max_len, rows), pool, o=o)
    for r0, p in ((0, 0), (rows - n, 2)):
        small = g.StatePool(torch.zeros(1, 1, 16, 16, device=DEV))
        b = g.Batch(torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), None, max_len, n)
        want = g.gdnl_attend_forward(dims, *(t[r0:r0 + n].contiguous() for t in (q, k, v)), gates, b, small)
        assert torch.equal(o[r0:r0 + n], want) and torch.equal(pool.buf[p], small.buf[0])


@pytest.mark.parametrize("hv", [1, 8, 48, 600])
def test_a_larger_batchs_workspace_serves_smaller_ones(hv):
    """Segments are cut by rows and heads: any batch of fewer rows needs no more, and gives the same bits."""
    g = gdn()
    dims = g.LinearDims(1, hv, 8, 8, act_dtype="f32")
    most = 9000 if hv < 600 else 1200
    spaces = [torch.empty(g.gdnl_attend_workspace_bytes(dims, 3, most, backward=b), dtype=torch.uint8, device=DEV) for b in (False, True)]
    for rows in (1, 129, 257, 513, 1025, 2049, 4097, most):
        if rows > most:
            continue
        c = Case([rows, 0, 0], hk=1, hv=hv, dk=8, dv=8, fast=0.1)
        o, so = c.forward(workspace=spaces[0])
        o2, so2 = c.forward()
        assert torch.equal(o, o2) and torch.equal(so.buf.nan_to_num(1), so2.buf.nan_to_num(1))
        for a, b in zip(c.backward(workspace=spaces[1]), c.backward()):
            assert torch.equal(a, b)


def test_many_sequences_and_an_empty_batch():
    g = gdn()
    c = Case([1, 0, 2] * 700, hk=1, hv=2, dk=8, dv=8)
    o, so = c.forward()
    c.check_forward(o, so)
    c.check_backward(c.backward())
    none = g.Batch(torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), None, 0, 0)
    e = lambda w: torch.empty(0, w, device=DEV)  # noqa: E731
    dims = g.LinearDims(1, 2, 8, 8, act_dtype="f32")
    pool = g.StatePool(torch.ones(1, 2, 8, 8, device=DEV))
    assert g.gdnl_attend_forward(dims, e(8), e(8), e(16), e(2), none, pool).shape == (0, 16)
    d = g.gdnl_attend_backward(dims, e(8), e(8), e(16), torch.zeros(2, device=DEV), none, pool, e(16))
    assert (d.dg == 0).all() and (pool.buf == 1).all()


def test_results_do_not_depend_on_timing():
    c = Case([1500, 70], act="bf16", dk=64, dv=64, decay="head")
    o, so = c.forward()
    d = c.backward()
    for _ in range(5):
        o2, so2 = c.forward()
        assert torch.equal(o, o2) and torch.equal(so.buf.nan_to_num(1), so2.buf.nan_to_num(1))
        for a, b in zip(d, c.backward()):
            assert torch.equal(a, b)
