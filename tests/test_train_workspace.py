"""The workspace queries of include/gdn_train.h: one size serves every smaller
batch (CPU: sizes and refusals; GPU: a call in a larger batch's workspace)."""
import ctypes

import numpy as np
import pytest

FAKE = 0x10000
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def L():
    import os
    import linear_attention_ssm_gdn_amd._lib as lib
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libgdn.so not built")
    lib.load()
    return lib


def conv_bytes(L, heads, rows):
    d, ws = L.GdnDims(*heads, 4, 0, BF16, F32, 1.0, 1e-6), ctypes.c_size_t()
    assert L.load().gdnt_conv_workspace_bytes(ctypes.byref(d), 3, rows, ctypes.byref(ws)) == 0
    return ws.value


# 96, 672, 8192 channels, and so many that one strip is enough for the longest
HEADS = [(1, 1, 32, 32), (1, 1, 32, 608), (16, 32, 128, 128), (2048, 4096, 128, 128)]


@pytest.mark.parametrize("heads", HEADS)
def test_the_conv_workspace_never_shrinks_with_rows(L, heads):
    C = 2 * heads[0] * heads[2] + heads[1] * heads[3]
    strips = -(-2048 // -(-C // 256))  # of a column, for 2048 in all
    rows = {0, 1, 2, 255, 256, 257, 70000, 1 << 18}
    for own in (13, 25, 57):  # where the strips' length may change
        rows |= {max(0, (strips + k) * own + j) for k in (-2, -1, 0, 1) for j in range(-2, 3)}
    sizes = [conv_bytes(L, heads, r) for r in sorted(rows)]
    assert sizes == sorted(sizes)


def test_the_scan_workspace_never_shrinks_with_rows(L):
    ws = ctypes.c_size_t()
    for C in (1, 64, 65, 4096):
        d, last = L.GdntScanDims(C, BF16, F32), 0
        for rows in (0, 1, 127, 128, 129, 255, 256, 257, 5000, 70000):
            assert L.load().gdnt_scan_workspace_bytes(ctypes.byref(d), 3, rows, ctypes.byref(ws)) == 0
            assert ws.value >= last
            last = ws.value


def test_batches_beyond_one_launch_are_refused(L):
    """HIP launches fewer than 2^32 threads: 2^23 workgroups of 512 are too many.  Refused on the host, by the queries
    and the call, before anything is launched."""
    ws = ctypes.c_size_t()
    ask = lambda C, rows: L.load().gdnt_scan_workspace_bytes(ctypes.byref(L.GdntScanDims(C, BF16, F32)), 1, rows,
                                                             ctypes.byref(ws))
    for C, per_row in ((1, 1), (128, 1), (129, 2), (4096, 32)):
        rows = (1 << 23) // per_row * 128  # 2^23 blocks of 128 rows by 128 channels
        assert ask(C, rows - 256) == 0, C
        assert ask(C, rows) == 1, C
        d = L.GdntScanDims(C, BF16, F32)
        assert L.load().gdnt_scan_saved_bytes(ctypes.byref(d), rows, ctypes.byref(ws), None) == 1
    d, p = L.GdntScanDims(64, BF16, F32), L.GdntScanParams(FAKE, FAKE)
    b, s = L.GdnBatch(FAKE, FAKE, None, 2, 0, (1 << 30) + 1), L.GdnStatePool(FAKE, 64, 4)
    assert L.load().gdnt_scan_forward(ctypes.byref(d), ctypes.byref(p), FAKE, 64, FAKE, FAKE, 64, ctypes.byref(b), s, s,
                                      FAKE, 64, None, None, FAKE, 1 << 62, None, None) == 1
    # the one-launch form: 2^24 workgroups of 256
    C = 1 << 24
    d, b, s = L.GdntScanDims(C, BF16, F32), L.GdnBatch(FAKE, FAKE, None, 1024, 1, 1024), L.GdnStatePool(FAKE, C, 1024)
    assert L.load().gdnt_scan_forward(ctypes.byref(d), ctypes.byref(p), FAKE, C, FAKE, FAKE, C, ctypes.byref(b), s, s,
                                      FAKE, C, None, None, None, 0, None, None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3591, 3500, 1575, 30])
def test_a_smaller_batch_in_a_larger_ones_workspace(rows):
    """8192 channels, sized for 4096 rows; 3591 rows have shorter strips and so more partial sums than 4096 have."""
    import torch
    from gpu_util import DEV, gdn
    from test_gpu_conv_backward import Conv
    g = gdn()
    lens = [rows // 3, 0, rows - rows // 3]
    c = Conv(lens, (16, 32, 128, 128), act="bf16", ydt="bf16", seed=rows)
    size = g.gdnt_conv_workspace_bytes(c.dims, 8, 4096)
    assert size >= g.gdnt_conv_workspace_bytes(c.dims, c.n, rows)
    whole = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    assert whole.data_ptr() % 256 == 0
    want = c.run()
    got = g.gdnt_conv_backward(c.dims, c.w, c.x, c.dy, c.batch, g.ConvPool(c.win, None),
                               d_window=torch.from_numpy(c.d_window).to(DEV), workspace=whole[:size])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert bool((whole[size:] == 0xA5).all())
    assert np.isfinite(got.d_conv_w.cpu().numpy()).all()


@pytest.mark.gpu
def test_pools_of_different_sizes():
    """A page that one of the two pools lacks is skipped and flagged; a backward call told the smaller number skips
    the same sequence, whose gradients are then nobody's."""
    import oracle.train as ora
    import torch
    from gpu_util import DEV, gdn
    from train_util import Case, check_grads
    g = gdn()
    c = Case([40, 300, 9], 64, "f32", "f32", seed=73)
    few = int(c.pages.max())  # one page too few for one sequence
    gone = int(np.argmax(c.pages))
    pool, err = g.StatePool(c.h0.to(DEV)), torch.zeros(1, dtype=torch.int32, device=DEV)
    small, saved = g.StatePool(torch.full((few, 64), float("nan"), device=DEV)), c.saved()
    h = c.empty_rows()
    g.gdnt_scan_forward(c.dims, c.params, c.t["x"], c.t["a"], c.t["b"], c.batch, pool, small, h=h, saved=saved, err=err)
    assert int(err.item()) == g.GDN_DEVERR_PAGE
    span = c.spans[gone]
    assert bool(torch.isnan(h[span[0]:span[1]]).all())
    err.zero_()
    out = g.gdnt_scan_backward(c.dims, c.params, c.batch, g.StatePool(pool.buf[:few]), saved, c.t["dh"], x=c.t["x"],
                               a=c.t["a"], b=c.t["b"], d_state=torch.from_numpy(c.d_state).to(DEV), out=c.grads_out(),
                               err=err)
    assert int(err.item()) == g.GDN_DEVERR_PAGE
    c.spans[gone] = None
    check_grads(c, out, ora)
