"""CPU tests of include/gdn_train.h: the header and the ctypes mirror, the
exported symbols, the sizes of workspaces and checkpoints, and the host-side
refusals (no GPU is touched: every call here is refused, or empty)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_train.h")
FAKE = 0x10000  # non-null and 256-byte aligned: validation never dereferences it
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def L():
    import linear_attention_ssm_gdn_amd._lib as lib
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return lib


@pytest.fixture(scope="module")
def so(L):
    return L.load()


def test_header_compiles_as_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gdn_train.h"\nint main(void) { return GDNT_SCAN_BLOCK == 256 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.dirname(HEADER),
                    str(src), "-o", str(tmp_path / "h")], check=True)
    subprocess.run([str(tmp_path / "h")], check=True)


def test_every_declared_symbol_is_exported(so, L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdnt_\w+)\s*\(", text))
    assert names == {n for n in L.SYMBOLS if n.startswith("gdnt_")}
    out = subprocess.run(["nm", "-D", "--defined-only", L.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if l.split()[-1].startswith("gdnt_")} == names


def test_struct_layouts_match_c(L, tmp_path):
    structs = {"gdnt_scan_dims": L.GdntScanDims, "gdnt_scan_params": L.GdntScanParams}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gdn_train.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'  printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'  printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0; }"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    got = dict(l.rsplit(" ", 1) for l in out.splitlines())
    for c, py in structs.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset


def _dims(L, C=64, act=BF16, state=F32):
    return L.GdntScanDims(C, act, state)


def test_saved_and_workspace_sizes(so, L):
    st, q, ws = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    for rows, C in ((0, 64), (1, 1), (256, 64), (257, 65), (40000, 4096)):
        d = _dims(L, C)
        assert so.gdnt_scan_saved_bytes(ctypes.byref(d), rows, ctypes.byref(st), ctypes.byref(q)) == 0
        n4 = -(-C // 64) * 16
        assert st.value == -(-rows // 256) * C * 4
        assert q.value == -(-rows // 16) * 3 * n4 * (64 + 4)
        assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 3, rows, ctypes.byref(ws)) == 0
        assert ws.value >= -(-rows // 256) * 256 * 4 + 256 and ws.value % 256 == 0
    d = _dims(L)
    assert so.gdnt_scan_saved_bytes(ctypes.byref(d), 5, None, None) == 0
    for bad in (dict(C=0), dict(C=-4), dict(C=(1 << 24) + 1), dict(act=2), dict(state=7)):
        d = _dims(L, **bad)
        assert so.gdnt_scan_saved_bytes(ctypes.byref(d), 5, ctypes.byref(st), None) == 1
        assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 1, 5, ctypes.byref(ws)) == 1
    d = _dims(L)
    assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 1, -1, ctypes.byref(ws)) == 1
    assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), -1, 5, ctypes.byref(ws)) == 1
    assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 1, 5, None) == 1
    assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 1, 1 << 31, ctypes.byref(ws)) == 1
    # more workgroups than a launch is given
    d = _dims(L, C=1 << 24)
    assert so.gdnt_scan_workspace_bytes(ctypes.byref(d), 1, (1 << 31) - 600, ctypes.byref(ws)) == 1
    cd = L.GdnDims(1, 1, 32, 64, 4, 0, BF16, F32, 1.0, 1e-6)
    assert so.gdnt_conv_workspace_bytes(ctypes.byref(cd), 1, 300, ctypes.byref(ws)) == 0
    assert ws.value >= 2 * 256 * 4 + 6 * 4 * 128 * 4  # the row map, and a partial sum for every 52 rows
    cd.conv_w = 3
    assert so.gdnt_conv_workspace_bytes(ctypes.byref(cd), 1, 300, ctypes.byref(ws)) == 2


BIG = 1 << 30


def _forward(so, L, **kw):
    d = kw.pop("dims", _dims(L))
    a = dict(params=L.GdntScanParams(FAKE, FAKE), x=FAKE, xs=64, a=FAKE, b=FAKE, abs=64,
             batch=L.GdnBatch(FAKE, FAKE, None, 2, 0, 300), si=L.GdnStatePool(FAKE, 64, 4),
             sto=L.GdnStatePool(FAKE, 64, 4), h=FAKE, hs=64, states=None, ckpt=None, ws=FAKE, wsb=BIG)
    a.update(kw)
    ref = lambda v: ctypes.byref(v) if v is not None else None
    return so.gdnt_scan_forward(ref(d), ref(a["params"]), a["x"], a["xs"], a["a"], a["b"], a["abs"], ref(a["batch"]),
                                a["si"], a["sto"], a["h"], a["hs"], a["states"], a["ckpt"], a["ws"], a["wsb"], None,
                                None)


def test_forward_refusals(so, L):
    P, B, S = L.GdntScanParams, L.GdnBatch, L.GdnStatePool
    for bad in (dict(dims=None), dict(dims=_dims(L, 0)), dict(dims=_dims(L, act=3)), dict(params=None),
                dict(params=P(None, FAKE)), dict(params=P(FAKE, None)), dict(batch=None),
                dict(batch=B(FAKE, FAKE, None, -1, 0, 300)), dict(batch=B(FAKE, FAKE, None, 2, -1, 300)),
                dict(batch=B(FAKE, FAKE, None, 2, 0, -1)), dict(batch=B(None, FAKE, None, 2, 0, 300)),
                dict(batch=B(FAKE, None, None, 2, 0, 300)), dict(batch=B(FAKE, FAKE, None, 1 << 29, 0, 300)),
                dict(x=None), dict(a=None), dict(b=None), dict(h=None), dict(xs=(1 << 24) + 1), dict(xs=63), dict(abs=63), dict(hs=63),
                dict(x=FAKE + 1), dict(h=FAKE + 1), dict(si=S(None, 64, 4)), dict(sto=S(None, 64, 4)),
                dict(si=S(FAKE, 63, 4)), dict(sto=S(FAKE, 64, -1)), dict(si=S(FAKE + 2, 64, 4)),
                dict(ckpt=FAKE), dict(states=FAKE, ckpt=FAKE + 64), dict(states=FAKE + 4), dict(ws=None),
                dict(ws=FAKE + 16), dict(wsb=1000)):
        assert _forward(so, L, **bad) == 1, bad
    # nothing to do: no sequence at all
    assert _forward(so, L, batch=B(None, None, None, 0, 0, 300), x=None, ws=None, wsb=0) == 0
    # rows kept to 8 a sequence need no workspace, but those that keep states do
    assert _forward(so, L, batch=B(FAKE, FAKE, None, 2, 8, 16), states=FAKE, ws=None, wsb=0) == 1


def _backward(so, L, **kw):
    d = kw.pop("dims", _dims(L))
    a = dict(params=L.GdntScanParams(FAKE, FAKE), x=FAKE, xs=64, a=FAKE, b=FAKE, abs=64, ckpt=None,
             batch=L.GdnBatch(FAKE, FAKE, None, 2, 0, 300), si=L.GdnStatePool(FAKE, 64, 4), states=FAKE, dh=FAKE,
             dhs=64, ds=None, dx=FAKE, dxs=64, da=FAKE, db=FAKE, dabs=64, dA=FAKE, dB=FAKE, d0=None, ws=FAKE, wsb=BIG)
    a.update(kw)
    ref = lambda v: ctypes.byref(v) if v is not None else None
    return so.gdnt_scan_backward(ref(d), ref(a["params"]), a["x"], a["xs"], a["a"], a["b"], a["abs"], a["ckpt"],
                                 ref(a["batch"]), a["si"], a["states"], a["dh"], a["dhs"], a["ds"], a["dx"],
                                 a["dxs"], a["da"], a["db"], a["dabs"], a["dA"], a["dB"], a["d0"], a["ws"],
                                 a["wsb"], None, None)


def test_backward_refusals(so, L):
    P, B, S = L.GdntScanParams, L.GdnBatch, L.GdnStatePool
    for bad in (dict(dims=None), dict(params=P(FAKE, None)), dict(batch=None), dict(x=None), dict(a=None),
                dict(b=None), dict(xs=10), dict(abs=10), dict(ckpt=FAKE), dict(x=None, a=None, b=None, ckpt=FAKE + 8),
                dict(si=S(None, 64, 4)), dict(states=None), dict(states=FAKE + 4), dict(dh=None), dict(dhs=63),
                dict(dx=None), dict(da=None), dict(db=None), dict(dxs=1 << 25), dict(dxs=1), dict(dabs=1), dict(dA=None),
                dict(dB=None), dict(ws=None), dict(ws=FAKE + 1), dict(wsb=0), dict(dx=FAKE + 1),
                dict(batch=B(FAKE, FAKE, None, 2, 0, (1 << 31) - 1))):
        assert _backward(so, L, **bad) == 1, bad


def _conv(so, L, **kw):
    d = kw.pop("dims", L.GdnDims(1, 1, 32, 64, 4, 0, BF16, F32, 1.0, 1e-6))
    C = 128
    a = dict(w=FAKE, x=FAKE, xs=C, dy=FAKE, dyt=F32, dys=C, batch=L.GdnBatch(FAKE, FAKE, None, 2, 0, 300),
             conv=L.GdnConvPool(FAKE, 3 * C, 3, 4, None), act=1, dwin=None, dx=FAKE, dxs=C, dw=FAKE, d0=None,
             ws=FAKE, wsb=BIG)
    a.update(kw)
    ref = lambda v: ctypes.byref(v) if v is not None else None
    return so.gdnt_conv_backward(ref(d), a["w"], a["x"], a["xs"], a["dy"], a["dyt"], a["dys"], ref(a["batch"]),
                                 a["conv"], a["act"], a["dwin"], a["dx"], a["dxs"], a["dw"], a["d0"], a["ws"],
                                 a["wsb"], None, None)


def test_conv_backward_refusals(so, L):
    B, P = L.GdnBatch, L.GdnConvPool
    for bad in (dict(dims=None), dict(w=None), dict(x=None), dict(dy=None), dict(dx=None), dict(dw=None),
                dict(xs=127), dict(dys=127), dict(dxs=127), dict(dys=(1 << 24) + 1), dict(dyt=2), dict(act=2), dict(batch=None),
                dict(conv=P(FAKE, 3 * 128, 2, 4, None)), dict(conv=P(FAKE, 128, 3, 4, None)),
                dict(conv=P(FAKE, 3 * 128, 3, -1, None)), dict(conv=P(FAKE + 1, 3 * 128, 3, 4, None)),
                dict(ws=None), dict(wsb=100), dict(ws=FAKE + 128), dict(dy=FAKE + 2),
                dict(batch=B(FAKE, FAKE, None, 2, 0, -5))):
        assert _conv(so, L, **bad) == 1, bad
    d = L.GdnDims(1, 1, 48, 64, 4, 0, BF16, F32, 1.0, 1e-6)
    assert _conv(so, L, dims=d) == 2


def test_the_binding_refuses_what_the_pointers_cannot_show(L):
    import torch
    import linear_attention_ssm_gdn_amd as g
    dims = g.ScanDims(8, act_dtype="f32")
    t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    params = g.ScanParams(t(8), t(8))
    batch = g.Batch(t(2, dt=torch.int32), t(1, dt=torch.int32), None, 0, 4)
    pool = g.StatePool(t(1, 8))
    ok = dict(dims=dims, params=params, x=t(4, 8), a=t(4, 8), b=t(4, 8), batch=batch, state_in=pool)
    for bad in (dict(x=t(4, 8, dt=torch.bfloat16)), dict(x=t(4, 7)), dict(x=t(3, 8)), dict(a=t(8, 4).t()),
                dict(a=t(4, 16)[:, :8]),  # a and b with different strides
                dict(params=g.ScanParams(t(8, dt=torch.float64), t(8))), dict(params=g.ScanParams(t(7), t(8))),
                dict(state_in=g.StatePool(t(1, 8, dt=torch.bfloat16))), dict(state_in=g.StatePool(t(1, 9))),
                dict(batch=g.Batch(t(2, dt=torch.int64), t(1, dt=torch.int32), None, 0, 4)),
                dict(batch=g.Batch(t(3, dt=torch.int32), t(1, dt=torch.int32), None, 0, 4)),
                dict(h=t(4, 8, dt=torch.bfloat16)), dict(workspace=t(64)),
                dict(saved=g.ScanSaved(t(2, 8)))):
        with pytest.raises(ValueError):
            g.gdnt_scan_forward(**{**ok, **bad})
    saved = g.ScanSaved(t(1, 8))
    with pytest.raises(ValueError):  # neither activations nor a checkpoint
        g.gdnt_scan_backward(dims, params, batch, pool, saved, t(4, 8))
    with pytest.raises(ValueError):
        g.gdnt_scan_backward(dims, params, batch, pool, saved, t(4, 8), x=t(4, 8))
    cd = g.Dims(1, 1, 32, 32, act_dtype="f32")
    with pytest.raises(ValueError):
        g.gdnt_conv_backward(cd, t(96, 4), t(4, 96), t(4, 96, dt=torch.float64), batch)
    with pytest.raises(ValueError):
        g.gdnt_conv_backward(cd, t(96, 3), t(4, 96), t(4, 96), batch)


def test_the_binding_refuses_tensors_on_the_host(L):
    """Valid in every other respect: the last check before a launch."""
    import torch
    import linear_attention_ssm_gdn_amd as g
    t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    dims, params, pool = g.ScanDims(8, act_dtype="f32"), g.ScanParams(t(8), t(8)), g.StatePool(t(1, 8))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    batch = g.Batch(cu, t(1, dt=torch.int32), None, 0, 4)
    saved = g.ScanSaved(t(1, 8))
    with pytest.raises(ValueError, match="on a GPU"):
        g.gdnt_scan_forward(dims, params, t(4, 8), t(4, 8), t(4, 8), batch, pool)
    with pytest.raises(ValueError, match="on a GPU"):
        g.gdnt_scan_backward(dims, params, batch, pool, saved, t(4, 8), x=t(4, 8), a=t(4, 8), b=t(4, 8))
    with pytest.raises(ValueError, match="on a GPU"):
        g.gdnt_conv_backward(g.Dims(1, 1, 32, 32, act_dtype="f32"), t(96, 4), t(4, 96), t(4, 96), batch)
