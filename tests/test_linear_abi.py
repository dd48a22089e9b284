"""CPU tests of include/gdn_linear.h: the header and the ctypes mirror, the
exported symbols, sizes, and the host-side refusals (no GPU is touched: every
call here is refused, or empty)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_linear.h")
FAKE = 0x10000  # non-null and 256-byte aligned: validation never dereferences it
BF16, F32 = 1, 0
BIG = 1 << 40


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
    src.write_text('#include "gdn_linear.h"\nint main(void) { return GDNL_CACHE_COLS == 64 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.dirname(HEADER),
                    str(src), "-o", str(tmp_path / "h")], check=True)
    subprocess.run([str(tmp_path / "h")], check=True)


def test_every_declared_symbol_is_exported(so, L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdnl_\w+)\s*\(", text))
    assert names == {n for n in L.SYMBOLS if n.startswith("gdnl_")}
    out = subprocess.run(["nm", "-D", "--defined-only", L.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if l.split()[-1].startswith("gdnl_")} == names


def test_struct_layouts_and_constants_match_c(L, tmp_path):
    structs = {"gdnl_dims": L.GdnlDims, "gdnl_rotate_dims": L.GdnlRotateDims, "gdnl_cache": L.GdnlCache}
    names = ("GDNL_CACHE_COLS", "GDNL_NORM_RMS", "GDNL_NORM_L2", "GDNL_PAIRS_HALVES", "GDNL_PAIRS_NEIGHBOURS")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gdn_linear.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'  printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'  printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    lines += [f'  printf("{n} %d\\n", {n});' for n in names]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0; }"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    got = dict(l.rsplit(" ", 1) for l in out.splitlines())
    for c, py in structs.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset
    for n in names:
        assert int(got[n]) == getattr(L, n)


def _dims(L, hk=2, hv=4, dk=16, dv=32, act=BF16, state=F32, scale=1.0):
    return L.GdnlDims(hk, hv, dk, dv, act, state, scale)


BAD_DIMS = [(dict(hk=0), 1), (dict(hv=3), 1), (dict(dk=0), 1), (dict(dv=-1), 1), (dict(act=2), 1), (dict(state=5), 1),
            (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(hk=1 << 20, hv=1 << 20), 1),
            (dict(dk=129), 2), (dict(dv=256), 2)]


def test_workspace_sizes(so, L):
    out, more = ctypes.c_size_t(), ctypes.c_size_t()
    for back in (0, 1):
        for kw in (dict(), dict(hk=4), dict(hk=16, hv=32, dk=128, dv=128), dict(hk=1, hv=300)):
            d = _dims(L, **kw)
            last = 0
            for rows in (0, 1, 255, 256, 257, 3000, 32768, 32769, 70000, 1 << 20):  # never less for more rows
                assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), 5, rows, back, ctypes.byref(out)) == 0
                assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), 6, rows, back, ctypes.byref(more)) == 0
                assert last <= out.value <= more.value and out.value % 256 == 0
                last = out.value
    for kw, status in BAD_DIMS:
        d = _dims(L, **kw)
        assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), 1, 5, 0, ctypes.byref(out)) == status, kw
    d = _dims(L)
    for args in ((-1, 5, 0), (1, -5, 0), (1, 1 << 31, 0), (1, 5, 2), (1 << 28, 5, 0)):
        assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), *args, ctypes.byref(out)) == 1, args
    assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), 1, 5, 0, None) == 1
    assert so.gdnl_attend_workspace_bytes(None, 1, 5, 0, ctypes.byref(out)) == 1


def _call(so, L, back, **kw):
    d = kw.pop("dims", _dims(L))
    S = L.GdnStatePool
    a = dict(q=FAKE, qs=32, k=FAKE, ks=32, v=FAKE, vs=128, g=FAKE, gs=4, batch=L.GdnBatch(FAKE, FAKE, None, 2, 0, 300),
             si=S(FAKE, 2048, 4), sto=S(FAKE, 2048, 4), o=FAKE, os=128, ds=None, dq=FAKE, dqs=32, dk=FAKE, dks=32, dv=FAKE,
             dvs=128, dg=FAKE, d0=None, ws=FAKE, wsb=BIG)
    a.update(kw)
    ref = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    first = (ref(d), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"], a["gs"], ref(a["batch"]), a["si"])
    if back:
        return so.gdnl_attend_backward(*first, a["o"], a["os"], a["ds"], a["dq"], a["dqs"], a["dk"], a["dks"], a["dv"],
                                       a["dvs"], a["dg"], a["d0"], a["ws"], a["wsb"], None, None)
    return so.gdnl_attend_forward(*first, a["sto"], a["o"], a["os"], a["ws"], a["wsb"], None, None)


def _bad(L):
    B, S = L.GdnBatch, L.GdnStatePool
    return [dict(dims=None), dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(o=None), dict(qs=31), dict(ks=31),
            dict(vs=127), dict(os=127), dict(gs=3), dict(gs=-1), dict(q=FAKE + 1), dict(g=FAKE + 2), dict(o=FAKE + 1),
            dict(qs=(1 << 24) + 1), dict(batch=None), dict(batch=B(FAKE, FAKE, None, -1, 0, 300)),
            dict(batch=B(FAKE, FAKE, None, 2, -1, 300)), dict(batch=B(FAKE, FAKE, None, 2, 0, -1)),
            dict(batch=B(None, FAKE, None, 2, 0, 300)), dict(batch=B(FAKE, None, None, 2, 0, 300)),
            dict(batch=B(FAKE, FAKE, None, 2, 0, (1 << 31) - 1)), dict(batch=B(FAKE, FAKE, None, 1 << 28, 0, 300)),
            dict(si=S(None, 2048, 4)), dict(si=S(FAKE, 2047, 4)), dict(si=S(FAKE, 2048, -1)), dict(si=S(FAKE + 2, 2048, 4)),
            dict(si=S(FAKE, 2048, 1 << 29)), dict(ws=None), dict(ws=FAKE + 16), dict(wsb=1000)]


def test_forward_refusals(so, L):
    S, B = L.GdnStatePool, L.GdnBatch
    for kw in _bad(L) + [dict(sto=S(None, 2048, 4)), dict(sto=S(FAKE, 100, 4)), dict(sto=S(FAKE + 1, 2048, 4))]:
        assert _call(so, L, False, **kw) == 1, kw
    for kw, status in BAD_DIMS:
        assert _call(so, L, False, dims=_dims(L, **kw)) == status, kw
    assert _call(so, L, False, batch=B(FAKE, FAKE, None, 1 << 23, 1, 300)) == 1  # more workgroups than a launch has
    assert _call(so, L, False, batch=B(None, None, None, 0, 0, 300), q=None, ws=None) == 0  # no sequence at all


def test_more_workgroups_than_a_launch_has(so, L):
    """2^32 threads are too many: 2^23 workgroups of 512, those counted that round a key head's values up to every XCD."""
    B, out = L.GdnBatch, ctypes.c_size_t()
    for hk, hv, n, status in ((1, 1 << 16, 127, 1), (1, 1 << 16, 200, 1), (1 << 16, 1 << 16, 127, 1), (1 << 16, 1 << 16, 120, 0)):
        d = _dims(L, hk=hk, hv=hv, dk=1, dv=1)
        for back in (0, 1):
            assert so.gdnl_attend_workspace_bytes(ctypes.byref(d), n, 100, back, ctypes.byref(out)) == status
        if status == 0:
            continue
        S = L.GdnStatePool
        for back in (False, True):
            assert _call(so, L, back, dims=d, qs=hk, ks=hk, vs=hv, os=hv, dqs=hk, dks=hk, dvs=hv, gs=hv, si=S(FAKE, hv, 4),
                         sto=S(FAKE, hv, 4), batch=B(FAKE, FAKE, None, n, 0, 100)) == 1
    d = _dims(L)
    assert _call(so, L, False, batch=B(FAKE, FAKE, None, 1 << 21, 1, 300)) == 1  # row by row, a workgroup to a sequence and head


def test_backward_refusals(so, L):
    B = L.GdnBatch
    for kw in _bad(L) + [dict(dq=None), dict(dk=None), dict(dv=None), dict(dqs=31), dict(dks=31), dict(dvs=127),
                         dict(dq=FAKE + 1), dict(dg=FAKE + 2), dict(ds=FAKE + 1), dict(d0=FAKE + 2)]:
        assert _call(so, L, True, **kw) == 1, kw
    for kw, status in BAD_DIMS:
        assert _call(so, L, True, dims=_dims(L, **kw)) == status, kw
    assert _call(so, L, True, batch=B(None, None, None, 0, 0, 300), q=None, ws=None) == 0
    assert _call(so, L, True, batch=B(None, None, None, 0, 0, 0), gs=0, dg=None) == 0


def _rot(L, hq=2, hk=1, d=16, rot=8, act=BF16, norm=0, pairs=0, eps=1e-6):
    return L.GdnlRotateDims(hq, hk, d, rot, act, norm, pairs, eps)


BAD_ROT = [(dict(hq=-1), 1), (dict(hk=-1), 1), (dict(hq=1 << 16), 1), (dict(d=0), 1), (dict(d=15), 1), (dict(rot=18), 1),
           (dict(rot=7), 1), (dict(rot=-2), 1), (dict(act=2), 1), (dict(norm=2), 1), (dict(pairs=-1), 1), (dict(eps=-1e-6), 1),
           (dict(eps=float("nan")), 1), (dict(d=258), 2)]


def _rotate(so, L, back, **kw):
    d = kw.pop("dims", _rot(L))
    a = dict(q=FAKE, qs=32, k=FAKE, ks=16, wq=FAKE, wk=None, pos=FAKE, inv=FAKE, n=7, yq=FAKE + 0x10000, yqs=32,
             yk=FAKE + 0x20000, yks=16, dq=FAKE + 0x30000, dqs=32, dk=FAKE + 0x40000, dks=16, dwq=FAKE, dwk=None, ws=FAKE, wsb=BIG)
    a.update(kw)
    first = (ctypes.byref(d) if d is not None else None, a["q"], a["qs"], a["k"], a["ks"], a["wq"], a["wk"], a["pos"], a["inv"], a["n"],
             a["yq"], a["yqs"], a["yk"], a["yks"])
    if back:
        return so.gdnl_rotate_backward(*first, a["dq"], a["dqs"], a["dk"], a["dks"], a["dwq"], a["dwk"], a["ws"], a["wsb"], None)
    return so.gdnl_rotate_forward(*first, None)


def test_rotate_refusals(so, L):
    both = [dict(dims=None), dict(q=None), dict(k=None), dict(qs=31), dict(ks=15), dict(pos=None), dict(inv=None), dict(n=-1),
            dict(n=1 << 31), dict(yq=None), dict(yk=None), dict(yqs=31), dict(yks=15), dict(q=FAKE + 1), dict(wq=FAKE + 2),
            dict(pos=FAKE + 2), dict(inv=FAKE + 1)]
    for kw in both + [dict(yq=FAKE, yqs=40), dict(yk=FAKE, yks=17)]:
        assert _rotate(so, L, False, **kw) == 1, kw
    for kw in both + [dict(dq=None), dict(dk=None), dict(dqs=31), dict(dks=15), dict(dq=FAKE + 1), dict(dwq=FAKE + 1),
                      dict(ws=None), dict(ws=FAKE + 8), dict(wsb=10), dict(dq=FAKE + 0x10000, dqs=40)]:
        assert _rotate(so, L, True, **kw) == 1, kw
    out = ctypes.c_size_t()
    for kw, status in BAD_ROT:
        d = _rot(L, **kw)
        assert _rotate(so, L, False, dims=d) == status and _rotate(so, L, True, dims=d) == status, kw
        assert so.gdnl_rotate_workspace_bytes(ctypes.byref(d), 5, ctypes.byref(out)) == status
    assert _rotate(so, L, False, n=0, q=None, pos=None) == 0
    assert _rotate(so, L, False, dims=_rot(L, hq=0, hk=0), q=None, k=None) == 0
    assert _rotate(so, L, True, n=0, q=None, pos=None, dwq=None) == 0
    d = _rot(L)
    sizes = []
    for rows in (0, 1, 1023, 1024, 5000):
        assert so.gdnl_rotate_workspace_bytes(ctypes.byref(d), rows, ctypes.byref(out)) == 0
        sizes.append(out.value)
    assert sizes == sorted(sizes) and sizes[1] >= 2 * 16 * 4
    assert so.gdnl_rotate_workspace_bytes(ctypes.byref(d), 5, None) == 1


def test_cache_sizes_and_refusals(so, L):
    q, sc = ctypes.c_size_t(), ctypes.c_size_t()
    d = _dims(L, dk=40, dv=300)  # wider than the attend calls take
    assert so.gdnl_cache_bytes(ctypes.byref(d), 3, ctypes.byref(q), ctypes.byref(sc)) == 0
    assert q.value == 3 * 4 * 40 * 300 and sc.value == 3 * 4 * 40 * 5 * 4
    assert so.gdnl_cache_bytes(ctypes.byref(d), 0, None, None) == 0
    assert so.gdnl_cache_bytes(ctypes.byref(d), -1, None, None) == 1 and so.gdnl_cache_bytes(None, 1, None, None) == 1
    S, C = L.GdnStatePool, L.GdnlCache
    d = _dims(L)
    ok = dict(n=2, a=FAKE, b=FAKE, pool=S(FAKE, 2048, 4), cache=C(FAKE, FAKE, 4))
    for kw in (dict(n=-1), dict(a=None), dict(b=None), dict(pool=S(None, 2048, 4)), dict(pool=S(FAKE, 2047, 4)),
               dict(pool=S(FAKE + 2, 2048, 4)), dict(cache=C(None, FAKE, 4)), dict(cache=C(FAKE, None, 4)), dict(cache=C(FAKE + 2, FAKE, 4)),
               dict(cache=C(FAKE, FAKE + 1, 4)), dict(cache=C(FAKE, FAKE, -1)), dict(cache=None), dict(n=1 << 30)):
        a = {**ok, **kw}
        c = ctypes.byref(a["cache"]) if a["cache"] is not None else None
        assert so.gdnl_cache_store(ctypes.byref(d), a["n"], a["a"], a["b"], a["pool"], c, None, None) == 1, kw
        assert so.gdnl_cache_load(ctypes.byref(d), a["n"], a["a"], a["b"], c, a["pool"], None, None) == 1, kw
    c = C(None, None, 0)
    assert so.gdnl_cache_store(ctypes.byref(d), 0, None, None, S(None, 0, 0), ctypes.byref(c), None, None) == 0


# --------------------------------------------------------------- the binding


def _host_calls():
    """Arguments that are right but for being on the host, the last thing refused."""
    import torch
    import linear_attention_ssm_gdn_amd as g
    t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)  # noqa: E731
    dims = g.LinearDims(1, 2, 8, 16, act_dtype="f32")
    batch = g.Batch(torch.tensor([0, 4], dtype=torch.int32), t(1, dt=torch.int32), None, 0, 4)
    attend = dict(dims=dims, q=t(4, 8), k=t(4, 8), v=t(4, 32), g=t(4, 2), batch=batch, state_in=g.StatePool(t(1, 2, 8, 16)))
    rot = dict(dims=g.RotateDims(2, 1, 8, 4, act_dtype="f32"), q=t(4, 16), k=t(4, 8), wq=t(8), wk=None, pos=t(4, dt=torch.int32), inv_freq=t(2))
    cache = dict(dims=dims, page_idx=t(2, dt=torch.int32), entry=t(2, dt=torch.int32), state=g.StatePool(t(3, 2, 8, 16)),
                 cache=g.StateCache.alloc(dims, 4, "cpu"))
    return g, t, attend, rot, cache


def test_the_binding_refuses_what_the_pointers_cannot_show(L):
    import torch
    g, t, attend, rot, cache = _host_calls()
    bf = torch.bfloat16
    for bad in (dict(q=t(4, 8, dt=bf)), dict(q=t(4, 9)), dict(k=t(3, 8)), dict(v=t(32, 4).t()), dict(g=t(4, 2, dt=bf)), dict(g=t(3)),
                dict(g=t(4, 3)), dict(state_in=g.StatePool(t(1, 2, 8, 16, dt=bf))), dict(state_in=g.StatePool(t(1, 2, 16, 8))),
                dict(state_out=g.StatePool(t(1, 2, 8))), dict(o=t(4, 31)), dict(workspace=t(64)), dict(err=t(1)),
                dict(batch=g.Batch(t(2, dt=torch.int64), t(1, dt=torch.int32), None, 0, 4))):
        with pytest.raises(ValueError):
            g.gdnl_attend_forward(**{**attend, **bad})
    for bad in (dict(d_o=t(4, 31)), dict(d_state=t(1, 2, 8, 15)), dict(d_state=t(1, 2, 16, 8).transpose(2, 3)),
                dict(out=g.LinearGrads(t(4, 8), t(4, 8), t(4, 32), t(2), t(1, 2, 8, 16))),
                dict(out=g.LinearGrads(t(4, 7), t(4, 8), t(4, 32), t(4, 2), t(1, 2, 8, 16)))):
        with pytest.raises(ValueError):
            g.gdnl_attend_backward(**{**attend, "d_o": t(4, 32), **bad})
    for bad in (dict(q=t(4, 15)), dict(k=t(5, 8)), dict(wq=t(7)), dict(wk=t(8, dt=bf)), dict(pos=t(4)), dict(pos=None), dict(inv_freq=t(3)),
                dict(yq=t(4, 16, dt=bf))):
        with pytest.raises(ValueError):
            g.gdnl_rotate_forward(**{**rot, **bad})
    with pytest.raises(ValueError):
        g.gdnl_rotate_backward(**rot, d_yq=t(4, 16), d_yk=t(4, 9))
    for bad in (dict(page_idx=t(3, dt=torch.int32)), dict(entry=t(2)), dict(state=g.StatePool(t(3, 2, 8, 15))),
                dict(cache=g.StateCache(t(4, 2, 8, 16), t(4, 2, 8, 1))), dict(cache=g.StateCache(t(4, 2, 8, 16, dt=torch.int8), t(4, 2, 8, 2)))):
        with pytest.raises(ValueError):
            g.gdnl_cache_store(**{**cache, **bad})
    with pytest.raises(KeyError):
        g.RotateDims(1, 1, 8, 4, norm="batch").c()


def test_the_binding_refuses_tensors_on_the_host_and_lost_history(L):
    import torch
    g, t, attend, rot, cache = _host_calls()
    calls = [(g.gdnl_attend_forward, attend, ("q", "k", "v", "g")), (g.gdnl_attend_backward, {**attend, "d_o": t(4, 32), "d_state": t(1, 2, 8, 16)}, ("d_o", "d_state")),
             (g.gdnl_rotate_forward, rot, ("q", "k", "wq")), (g.gdnl_rotate_backward, {**rot, "d_yq": t(4, 16), "d_yk": t(4, 8)}, ("d_yq", "d_yk"))]
    for f, kw, names in calls:
        with pytest.raises(ValueError, match="on a GPU"):
            f(**kw)
        for n in names:
            with pytest.raises(ValueError, match="autograd"):
                f(**{**kw, n: kw[n].clone().requires_grad_()})
    with pytest.raises(ValueError, match="on a GPU"):
        g.gdnl_cache_store(**cache)
    with pytest.raises(ValueError, match="on a GPU"):
        g.gdnl_cache_load(**cache)
