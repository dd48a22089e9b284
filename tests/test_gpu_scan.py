"""GPU tests of the vector-state gated recurrence: forward, backward, 8-bit
checkpoint, each against the float64 oracle (oracle/train.py) at the sizes
and masks where it can go wrong."""
import numpy as np
import pytest
import torch

import oracle.train as ora
from gpu_util import DEV, gdn, host
from train_util import ULP, Case, check_forward, check_grads

pytestmark = pytest.mark.gpu

# lengths around the row group (8), the wave (32), the tile (256); ragged; empty; single
LENS = {
    "one": [1], "eight": [8], "nine": [9], "tile": [256], "tile+1": [257], "ragged": [3, 0, 1, 31, 300, 0, 65, 2],
    "ones": [1] * 40, "long": [1025], "two_tiles_each": [511, 513, 256],
}
TYPES = [("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("act,state", TYPES)
@pytest.mark.parametrize("C", [1, 5, 64, 100])
@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
def test_forward_and_backward(lens, C, act, state):
    c = Case(LENS[lens], C, act, state, seed=C + len(lens))
    saved = c.saved()
    h, si, so = c.forward(saved)
    check_forward(c, h, so, ora)
    check_grads(c, c.backward(saved), ora)


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("C", [8, 72, 200, 328])
def test_backward_of_many_tiles(C, ckpt):
    """bf16 rows on 16 bytes and channels a multiple of 8: tiles whose rows are loaded ahead, between ones that are
    not (a sequence's end inside), in columns that end before their 64 channels."""
    c = Case([700, 1, 0, 513, 255, 90, 2000, 3], C, "bf16", "f32", tail=40, seed=C)
    saved = c.saved(ckpt=ckpt)
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    if not ckpt:
        check_grads(c, c.backward(saved), ora)
        return
    v, _, _ = decode(c, saved)
    with np.errstate(invalid="ignore"):
        before = ora.scan(c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans, c.seq_h0())[2]
        rb = ora.rebuilt(v[0], v[1], v[2], c.a_log, c.dt_bias, c.spans, before)
    check_grads(c, c.backward(saved, from_ckpt=True), ora, x=v[0], a=v[1], b=v[2], before=rb)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("C", [65, 129, 193, 255])
def test_a_last_channel_of_its_own_column(C, act):
    """Odd widths whose last channel begins a tile's column (and one in a column's last lane), rows on odd offsets."""
    c = Case([300, 0, 5, 130], C, act, "f32", tail=20, pad=C % 4 - 1, seed=C)
    saved = c.saved()
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    check_grads(c, c.backward(saved), ora)


@pytest.mark.parametrize("rows", [1, 31, 32, 273])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (1, 1)])
def test_pairs_that_end_with_the_tensor(rows, pad, offset):
    """bf16 rows on odd offsets, the last row's last pair the tensor's end."""
    for C in (66, 128, 67):
        c = Case([rows], C, "bf16", "f32", pad=pad, offset=offset, seed=rows)
        saved = c.saved()
        h, _, so = c.forward(saved)
        check_forward(c, h, so, ora)
        check_grads(c, c.backward(saved), ora)


@pytest.mark.parametrize("act,state", [("bf16", "bf16"), ("f32", "f32")])
def test_other_types_padding_gaps_tails_and_strides(act, state):
    """Padding sequences (their rows NaN: unread), rows before the first and behind the last sequence, padded rows
    at odd offsets (the element-wise loads), has_init of both kinds."""
    for pad, offset, C in ((0, 0, 128), (3, 1, 72), (4, 4, 64)):
        c = Case([70, 5, 0, 400, 1, 33], C, act, state, skip=(1, 3), gap=11, tail=270, pad=pad, offset=offset,
                 has_init=[1, 1, 0, 1, 0, 0], seed=7)
        saved = c.saved()
        h, si, so = c.forward(saved)
        check_forward(c, h, so, ora)
        check_grads(c, c.backward(saved), ora)
        check_grads(c, c.backward(saved, d_state=False), ora, d_state=False)


def test_states_in_place_equal_states_apart():
    """state_out may be state_in: a page is read before the call's end writes it, whether the sequence ends in the
    tile it starts in or later."""
    c = Case([5, 700, 1, 256, 2, 64], 192, "bf16", "f32", seed=3)
    h1, _, so = c.forward()
    h2, _, sip = c.forward(in_place=True)
    assert torch.equal(h1[torch.from_numpy(c.owned)], h2[torch.from_numpy(c.owned)])
    used = torch.from_numpy(c.pages).long()
    assert torch.equal(so.buf[used], sip.buf[used])
    rest = [p for p in range(c.n + 2) if p not in c.pages]
    assert torch.equal(sip.buf[rest].cpu(), c.h0[rest])


@pytest.mark.parametrize("act,state", TYPES)
@pytest.mark.parametrize("C", [3, 64, 1028])
def test_few_rows_a_sequence(C, act, state):
    """max_seqlen up to 8: one launch without a row map; also what it must refuse."""
    g = gdn()
    c = Case([1, 8, 0, 3, 1, 7], C, act, state, skip=(3,), has_init=[1, 0, 1, 1, 1, 1], tail=2, seed=C)
    b = g.Batch(c.batch.cu_seqlens, c.batch.page_idx, c.batch.has_init, 8, c.rows)
    h, _, so = c.forward(batch=b)
    check_forward(c, h, so, ora)
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)  # it needs no workspace
    h2 = c.empty_rows()
    so2 = g.StatePool(torch.full_like(so.buf, float("nan")))
    g.gdnt_scan_forward(c.dims, c.params, c.t["x"], c.t["a"], c.t["b"], b, g.StatePool(c.h0.to(DEV)), so2, h=h2,
                        workspace=ws)
    assert torch.equal(host_t(h2), host_t(h)) and torch.equal(host_t(so2.buf), host_t(so.buf))


def host_t(t):
    return torch.nan_to_num(t.detach().double().cpu(), nan=1e9)


@pytest.mark.parametrize("max_seqlen", [0, 4])
def test_bad_batches_are_skipped_and_flagged(max_seqlen):
    """A page beyond the pool, bounds that decrease, overlap or pass n_rows, and a sequence longer than max_seqlen
    skip that sequence alone (max_seqlen 4: the one-launch form, 0: the tiles)."""
    g = gdn()
    c = Case([4, 4, 4, 4], 64, "f32", "f32", seed=5)
    cu = c.batch.cu_seqlens
    good = c.batch.page_idx

    def run(cu_, pages, n_rows=c.rows, limit=max_seqlen):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        b = g.Batch(torch.tensor(cu_, dtype=torch.int32, device=DEV),
                    torch.tensor(pages, dtype=torch.int32, device=DEV), None, limit, n_rows)
        h, _, so = c.forward(batch=b, err=err)
        return host(h), host(so.buf), int(err.item())

    pages = good.tolist()
    base, st, e = run(cu.tolist(), pages)
    assert e == 0 and not np.isnan(base).any()
    h, so, e = run(cu.tolist(), [pages[0], 6, pages[2], pages[3]])  # 6 pages: 0..5
    assert e == g.GDN_DEVERR_PAGE and np.isnan(h[4:8]).all() and np.array_equal(np.delete(h, range(4, 8), 0),
                                                                               np.delete(base, range(4, 8), 0))
    assert np.isnan(so[pages[1]]).all()
    h, so, e = run([0, 4, 8, 12, 99], pages)
    assert e == g.GDN_DEVERR_BATCH and np.isnan(h[12:]).all() and np.array_equal(h[:12], base[:12])
    h, so, e = run([0, 4, 8, 6, 16], pages)  # the third decreases
    assert e == g.GDN_DEVERR_BATCH and np.array_equal(h[:8], base[:8]) and np.isnan(so[pages[2]]).all()
    h, so, e = run([-3, 4, 8, 12, 16], pages)
    assert e == g.GDN_DEVERR_BATCH and np.isnan(h[:4]).all() and np.array_equal(h[4:], base[4:])
    h, so, e = run([0, 4, 2, 6, 8], pages)  # the second decreases, the third begins inside the first
    assert e == g.GDN_DEVERR_BATCH and np.array_equal(h[:4], base[:4])
    assert np.isnan(h[4:6]).all() and np.isnan(so[pages[1:3]]).all() and not np.isnan(h[6:8]).any()
    h, so, e = run(cu.tolist(), pages, limit=3)
    assert e == g.GDN_DEVERR_BATCH and np.isnan(h).all() and np.isnan(so).all()


def test_many_sequences():
    """More sequences than a workgroup has threads, of every length from 0 to 6, in both forms."""
    g = gdn()
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 7, 1500).tolist()
    c = Case(lens, 20, "f32", "f32", skip=(7, 900), seed=8)
    saved = c.saved()
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    check_grads(c, c.backward(saved), ora)
    b = g.Batch(c.batch.cu_seqlens, c.batch.page_idx, None, 6, c.rows)
    h, _, so = c.forward(batch=b)
    check_forward(c, h, so, ora)


@pytest.mark.parametrize("n", [4096, 4097])
def test_sequences_around_the_last_batch_of_one_launch(n):
    g = gdn()
    c = Case(np.random.default_rng(n).integers(0, 3, n).tolist(), 5, "f32", "f32", seed=n)
    b = g.Batch(c.batch.cu_seqlens, c.batch.page_idx, None, 2, c.rows)
    h, _, so = c.forward(batch=b)
    check_forward(c, h, so, ora)


def test_rows_beyond_four_gigabytes():
    """Row offsets that pass 32 bits: x, dh and dx with 3 MB between rows, against the same rows packed."""
    c = Case([300, 1400], 64, "bf16", "f32", seed=19)
    saved = c.saved(ckpt=True)
    h, _, so = c.forward(saved)
    want = c.backward(saved)
    stride = 3 << 19
    wide = {k: torch.zeros((c.rows, stride), dtype=torch.bfloat16, device=DEV) for k in ("x", "dh", "dx")}
    assert c.rows * stride * 2 > 1 << 32
    for k in ("x", "dh"):
        wide[k][:, :64].copy_(c.t[k])
        c.t[k] = wide[k][:, :64]
    saved2 = c.saved()
    h2, _, so2 = c.forward(saved2)
    assert torch.equal(h2, h) and torch.equal(saved2.states[1:2], saved.states[1:2])
    g = gdn()
    out = c.grads_out()._replace(dx=wide["dx"][:, :64])
    plain = Case([300, 1400], 64, "bf16", "f32", seed=19)
    ref = plain.backward(saved2)
    g.gdnt_scan_backward(c.dims, c.params, c.batch, g.StatePool(c.h0.to(DEV)), saved2, c.t["dh"], x=c.t["x"],
                         a=c.t["a"], b=c.t["b"], d_state=torch.from_numpy(c.d_state).to(DEV), out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, ref))
    assert float(wide["dx"][:, 64:].abs().max()) == 0
    del want


def test_a_checkpoint_beyond_four_gigabytes():
    """The last sequence of a batch whose checkpoint passes 32 bits gives the bits it gives alone (it begins on a
    kept state's row, so tiles and blocks are the same)."""
    g = gdn()
    C, n, first = 4096, 1000, 256 * 1400
    dims = g.ScanDims(C)
    assert g.gdnt_scan_saved_bytes(dims, first)[1] > 1 << 32
    rows = lambda v: torch.cat((torch.zeros((first, C), dtype=v.dtype, device=DEV), v))
    torch.manual_seed(3)
    x, a, b, dh = (torch.randn(n, C, device=DEV).bfloat16() for _ in range(4))
    params = g.ScanParams(torch.randn(C, device=DEV) * 0.1, torch.randn(C, device=DEV) - 3)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    h0, d_state = torch.randn(2, C, device=DEV), torch.randn(2, C, device=DEV)

    def step(x, a, b, dh, batch, ds):
        pool, out = g.StatePool(h0), g.StatePool(torch.zeros_like(h0))
        saved = g.ScanSaved.alloc(dims, batch.n_rows, DEV, ckpt=True)
        h = g.gdnt_scan_forward(dims, params, x, a, b, batch, pool, out, saved=saved)
        got = g.gdnt_scan_backward(dims, params, batch, pool, saved, dh, d_state=ds)
        torch.cuda.synchronize()
        return (h[-n:], out.buf[1], got.dx[-n:], got.da[-n:], got.db[-n:], got.d_state0[-1])
    want = step(x, a, b, dh, g.Batch(i32(0, n), i32(1), None, 0, n), d_state[1:])
    got = step(*(rows(v) for v in (x, a, b, dh)), g.Batch(i32(0, first, first + n), i32(0, 1), None, 0, first + n),
               d_state)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_one_row_of_any_stride():
    """A single row has no stride to speak of: views of wider buffers, a's and b's strides apart."""
    g = gdn()
    c = Case([1], 24, "bf16", "f32", seed=4)
    want = c.forward()
    for k, width in (("x", 24), ("a", 40), ("b", 1 << 25)):
        buf = torch.zeros((1, width), dtype=torch.bfloat16, device=DEV)
        buf[:, :24].copy_(c.t[k])
        c.t[k] = buf[:, :24]
    got = c.forward()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2].buf[c.pages], want[2].buf[c.pages])


def test_bad_batches_in_the_backward_pass():
    g = gdn()
    c = Case([300, 20, 40], 64, "f32", "f32", seed=6)
    saved = c.saved()
    c.forward(saved)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = g.Batch(torch.tensor([0, 300, 300 + 400, 360], dtype=torch.int32, device=DEV), c.batch.page_idx, None, 0,
                c.rows)
    out = c.backward(saved, batch=b, err=err)
    assert int(err.item()) == g.GDN_DEVERR_BATCH
    c.spans = [c.spans[0], None, None]  # [300, 700) passes n_rows, [700, 360) decreases
    c.owned[300:] = False
    check_grads(c, out, ora)


def test_empty_batches():
    g = gdn()
    c = Case([0, 0], 64, "bf16", "f32", seed=1)
    saved = c.saved()
    h, _, so = c.forward(saved)
    assert torch.isnan(so.buf.float()).all()
    out = c.backward(saved)
    assert float(out.d_a_log.abs().sum()) == 0 and float(out.d_dt_bias.abs().sum()) == 0
    assert np.array_equal(host(out.d_state0), c.d_state.astype(np.float64))
    none = g.Batch(torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), None,
                   0, 0)
    z = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    st = g.ScanSaved.alloc(c.dims, 0, DEV)
    got = g.gdnt_scan_backward(c.dims, c.params, none, g.StatePool(c.h0.to(DEV)), st, z, x=z, a=z, b=z)
    assert float(got.d_a_log.abs().sum()) == 0 and got.d_state0.shape == (0, 64)


def test_states_kept_are_the_states_before_every_256th_row():
    c = Case([600, 168, 300], 64, "f32", "f32", seed=9)
    saved = c.saved()
    h, _, _ = c.forward(saved)
    with np.errstate(invalid="ignore"):
        before = ora.scan(c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans, c.seq_h0())[2]
    st = host(saved.states)
    for r in (256, 512, 1024):
        assert np.abs(st[r // 256] - before[r]).max() <= c.tol() * (1 + np.abs(before[r]).max()) * 4
    assert np.isnan(st[[0, 3]]).all()  # row 0 and row 768 start sequences


def test_a_long_memory():
    """Decays within 1e-3 of 1 over thousands of rows: the gates' errors add up over the memory."""
    c = Case([3000], 64, "f32", "f32", seed=11, dt_lo=1e-4, dt_hi=1e-3)
    saved = c.saved()
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    check_grads(c, c.backward(saved), ora)


def test_extreme_gates():
    """a and b far out, the lowest bf16 and both infinities: the gates saturate, nothing becomes NaN."""
    c = Case([40, 300], 64, "bf16", "f32", seed=12)
    lo = torch.finfo(torch.bfloat16).min
    for k in "ab":
        t = c.t[k]
        t[3, :8] = lo
        t[4, 8:16] = -lo
        t[100, 16:24] = float("-inf")
        t[101, 24:32] = float("inf")
        t[200, :] = 60.0
        t[201, :] = -60.0
    saved = c.saved()
    h, _, so = c.forward(saved)
    with np.errstate(over="ignore", invalid="ignore"):
        ref, last, _ = ora.scan(c.f64("x"), np.clip(c.f64("a"), -1e4, 1e4), np.clip(c.f64("b"), -1e4, 1e4), c.a_log,
                                c.dt_bias, c.spans, c.seq_h0())
    got = host(h)
    assert not np.isnan(got).any()
    assert np.abs(got - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    out = c.backward(saved)
    for k in ("dx", "da", "db"):
        assert not torch.isnan(getattr(out, k)).any(), k


def test_nan_and_inf_stay_in_their_sequence_and_channel():
    c = Case([300, 290, 10], 64, "f32", "f32", seed=13)
    c.t["x"][20, 5] = float("inf")
    c.t["x"][310, 9] = float("nan")
    h, _, so = c.forward()
    clean = Case([300, 290, 10], 64, "f32", "f32", seed=13)
    ref, _, so2 = clean.forward()
    bad = ~torch.isfinite(h)
    want = torch.zeros_like(bad)
    want[20:300, 5] = True
    want[310:590, 9] = True
    assert torch.equal(bad, want)
    assert torch.equal(h[~want], ref[~want])


def test_gradients_against_differences():
    """The gradients predict how a random linear functional of h and the final states changes: central differences
    of the float64 oracle around the inputs, along one random direction for each input."""
    c = Case([33, 1, 270, 7], 12, "f32", "f32", seed=17)
    saved = c.saved()
    c.forward(saved)
    g = c.backward(saved)
    rng = np.random.default_rng(0)
    x, a, b = (c.f64(k) for k in "xab")
    h0, dh = c.seq_h0(), c.f64("dh")

    def value(x, a, b, a_log, dt_bias, h0):
        h, last, _ = ora.scan(x, a, b, a_log, dt_bias, c.spans, h0)
        return (h * dh).sum() + (last * c.d_state).sum()

    at = [x, a, b, c.a_log.astype(np.float64), c.dt_bias.astype(np.float64), h0]
    for k, (v, grad) in enumerate(zip(at, (g.dx, g.da, g.db, g.d_a_log, g.d_dt_bias, g.d_state0))):
        step = rng.standard_normal(v.shape)
        e = 1e-5
        up, down = ([w + s * e * step if i == k else w for i, w in enumerate(at)] for s in (1, -1))
        want = (value(*up) - value(*down)) / (2 * e)
        gr = host(grad)
        # the difference is off by e^2 of the third derivative and by 1e-16 / e of the value; each gradient by tol of
        # its terms, and they add up with random signs
        assert abs((gr * step).sum() - want) <= 1e-4 * np.sqrt((gr ** 2).sum()) + 1e-6 * abs(want), k


# ------------------------------------------------------------------ 8 bits


def decode(c, saved):
    """x, a, b that the checkpoint stands for, the raw integers and scales too, from its documented layout."""
    nb, n4 = -(-c.rows // 16), -(-c.C // 64) * 16
    raw = saved.ckpt.cpu().numpy()
    q = raw[:nb * 3 * n4 * 64].view(np.int8).reshape(nb, 3, n4, 16, 4)
    s = raw[nb * 3 * n4 * 64:].view(np.float32).reshape(nb, 3, n4)
    with np.errstate(invalid="ignore"):
        v = q.astype(np.float64) * s[:, :, :, None, None].astype(np.float64)
    v = v.transpose(1, 0, 3, 2, 4).reshape(3, nb * 16, n4 * 4)[:, :c.rows, :c.C]
    return v, q, s


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("lens,C", [([1], 1), ([17, 0, 300, 2], 64), ([600, 45], 70), ([256], 132)])
def test_checkpoint(lens, C, act):
    """The stored integers and scales equal the definition's; the gradients are those at the stored values."""
    c = Case(lens, C, act, "f32", skip=(1,) if len(lens) == 4 else (), tail=5, seed=C)
    with torch.no_grad():
        c.t["x"][0, :1] = 1e-38  # blocks too small to scale are stored as zeros
    plain, saved = c.saved(), c.saved(ckpt=True)
    h0, _, so0 = c.forward(plain)
    h, _, so = c.forward(saved)
    assert torch.equal(host_t(h), host_t(h0)) and torch.equal(host_t(so.buf), host_t(so0.buf))
    v, q, s = decode(c, saved)
    for k, name in enumerate("xab"):
        qr, sr = ora.quantise(c.f64(name), c.owned)
        nc = qr.shape[2]
        assert np.array_equal(s[:, k, :nc], sr.astype(np.float32)), name
        assert np.array_equal(q[:, k, :nc].transpose(0, 2, 1, 3), qr), name
    with np.errstate(invalid="ignore"):
        before = ora.scan(c.f64("x"), c.f64("a"), c.f64("b"), c.a_log, c.dt_bias, c.spans, c.seq_h0())[2]
        # decoding multiplies an integer by an fp32 scale: one more rounding, half an ulp, inside the bounds
        rb = ora.rebuilt(v[0], v[1], v[2], c.a_log, c.dt_bias, c.spans, before)
    check_grads(c, c.backward(saved, from_ckpt=True), ora, x=v[0], a=v[1], b=v[2], before=rb)


def test_checkpoint_of_values_that_are_not_finite():
    """A block with an Inf or NaN comes back as NaNs, its neighbours untouched."""
    c = Case([64], 64, "f32", "f32", seed=21)
    c.t["x"][5, 3] = float("inf")
    c.t["b"][40, 17] = float("nan")
    saved = c.saved(ckpt=True)
    c.forward(saved)
    v, _, _ = decode(c, saved)
    want = np.zeros((3, 64, 64), bool)
    want[0, 0:16, 0:4] = True
    want[2, 32:48, 16:20] = True
    assert np.array_equal(np.isnan(v), want)


# ---------------------------------------------------------- streams and graphs


def test_two_streams_with_workspaces_of_their_own():
    c1, c2 = Case([700, 5], 512, "bf16", "f32", seed=31), Case([3, 900], 512, "bf16", "f32", seed=32)
    want = [c.forward()[0] for c in (c1, c2)]
    g = gdn()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, s in zip((c1, c2), streams):
            with torch.cuda.stream(s):
                got.append((c, g.gdnt_scan_forward(c.dims, c.params, c.t["x"], c.t["a"], c.t["b"], c.batch,
                                                   g.StatePool(c.h0.to(DEV)), g.StatePool(c.h0.to(DEV)))))
    torch.cuda.synchronize()
    for c, h in got:
        assert torch.equal(h, want[0] if c is c1 else want[1])


def test_backward_calls_on_two_streams_at_once():
    """More tiles than the GPU holds workgroups, from both calls, with what each waits for in the other's way."""
    g = gdn()
    cs = [Case([5000, 3000, 200], 4096, "bf16", "f32", seed=s) for s in (51, 52)]
    saved = [c.saved(ckpt=True) for c in cs]
    for c, sv in zip(cs, saved):
        c.forward(sv)
    want = [c.backward(sv, from_ckpt=bool(i)) for i, (c, sv) in enumerate(zip(cs, saved))]
    pools = [g.StatePool(c.h0.to(DEV)) for c in cs]
    ds = [torch.from_numpy(c.d_state).to(DEV) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                xab = {} if i else {k: c.t[k] for k in "xab"}
                got.append((i, g.gdnt_scan_backward(c.dims, c.params, c.batch, pools[i], saved[i], c.t["dh"],
                                                    d_state=ds[i], **xab)))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


def test_decode_steps_replayed_from_a_graph_in_place():
    """The one-launch form with states in place: each replay goes on from the states the last one left."""
    g = gdn()
    c = Case([1] * 9 + [0, 2], 260, "bf16", "f32", skip=(4,), seed=43)
    b = g.Batch(c.batch.cu_seqlens, c.batch.page_idx, None, 2, c.rows)
    pool, ref = g.StatePool(c.h0.to(DEV)), g.StatePool(c.h0.to(DEV))
    h, want = c.empty_rows(), c.empty_rows()
    step = lambda p, out: g.gdnt_scan_forward(c.dims, c.params, c.t["x"], c.t["a"], c.t["b"], b, p, h=out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(pool, h)
    step(ref, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, h)
    own = torch.from_numpy(c.owned).to(DEV)
    gen = torch.Generator().manual_seed(2)
    for _ in range(4):
        for name in ("x", "a", "b"):
            c.t[name].copy_(torch.randn(c.rows, c.C, generator=gen).to(torch.bfloat16))
        step(ref, want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.buf, ref.buf) and torch.equal(h[own], want[own])
        assert torch.isnan(h[~own]).all()


def test_a_training_step_replayed_from_a_graph():
    """Forward with a checkpoint and backward captured once and replayed over changing inputs, eager work and
    synchronisations between: every replay equals the eager calls bit for bit."""
    g = gdn()
    c = Case([300, 0, 45, 1], 192, "bf16", "f32", seed=41)
    saved = c.saved(ckpt=True)
    si, so = g.StatePool(c.h0.to(DEV)), g.StatePool(c.h0.to(DEV))
    ws = torch.empty(g.gdnt_scan_workspace_bytes(c.dims, c.n, c.rows), dtype=torch.uint8, device=DEV)
    ds = torch.from_numpy(c.d_state).to(DEV)
    h, out = c.empty_rows(), c.grads_out()

    def step():
        g.gdnt_scan_forward(c.dims, c.params, c.t["x"], c.t["a"], c.t["b"], c.batch, si, so, h=h, saved=saved,
                            workspace=ws)
        g.gdnt_scan_backward(c.dims, c.params, c.batch, si, saved, c.t["dh"], d_state=ds, out=out, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator().manual_seed(1)
    for k in range(4):
        for name in ("x", "a", "b", "dh"):
            c.t[name].copy_(torch.randn(c.rows, c.C, generator=gen).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        used = torch.tensor([p for p, n in zip(c.pages, c.lens) if n], device=DEV)  # the pages a sequence ends in
        results = lambda: [t.clone() for t in (h, so.buf[used], *out)]
        want = results()
        for t in (h, so.buf, *out):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for w, t in zip(want, results()):
            assert torch.equal(w, t), k


def test_results_do_not_depend_on_the_run():
    c = Case([5000, 300, 2000], 320, "bf16", "f32", seed=51)
    saved = c.saved(ckpt=True)
    h, _, so = c.forward(saved)
    g0 = c.backward(saved)
    for _ in range(5):
        h2, _, so2 = c.forward(saved)
        g2 = c.backward(saved)
        assert torch.equal(h, h2) and torch.equal(host_t(so.buf), host_t(so2.buf))
        assert all(torch.equal(p, q) for p, q in zip(g0, g2))
