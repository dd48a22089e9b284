"""Torch-facing binding of include/gdn_linear.h: linear attention with a decay
for each head, its backward pass, the head norms with the rotation by position
in front of it, and state pages in 8 bits.

As in train.py every function checks its tensors, turns them into device
pointers, strides and sizes, calls the C entry point on the current HIP stream
of the tensors' device and raises on a non-OK status.  Outputs and workspaces
that are not given are allocated.  Autograd records nothing here: a call whose
history would be lost in silence, forward or backward, is refused, be it that
gradients are enabled and an input requires one (the backward calls' inputs
too: they have no second derivative) or that an input has a forward-mode
tangent.  Call it under torch.no_grad(), with detached tensors, or from a
torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _lib as L
from .ops import _DT, _TORCH_DT, Batch, StatePool, _check
from .train import _call, _check_batch, _err, _flat, _no_history, _on, _p, _rows2

_NORMS = {"rms": L.GDNL_NORM_RMS, "l2": L.GDNL_NORM_L2}
_PAIRS = {"halves": L.GDNL_PAIRS_HALVES, "neighbours": L.GDNL_PAIRS_NEIGHBOURS}


@dataclasses.dataclass(frozen=True)
class LinearDims:
    h_k: int
    h_v: int
    d_k: int
    d_v: int
    act_dtype: str = "bf16"
    state_dtype: str = "f32"
    scale: float = 1.0

    @functools.cached_property
    def _c(self) -> L.GdnlDims:
        return L.GdnlDims(self.h_k, self.h_v, self.d_k, self.d_v, _DT[self.act_dtype], _DT[self.state_dtype],
                          self.scale)

    def c(self) -> L.GdnlDims:
        return self._c  # the library only reads it


@dataclasses.dataclass(frozen=True)
class RotateDims:
    h_q: int
    h_k: int
    d: int
    rot: int
    act_dtype: str = "bf16"
    norm: str = "rms"          # or "l2"
    pairs: str = "halves"      # or "neighbours"
    eps: float = 1e-6

    @functools.cached_property
    def _c(self) -> L.GdnlRotateDims:
        return L.GdnlRotateDims(self.h_q, self.h_k, self.d, self.rot, _DT[self.act_dtype], _NORMS[self.norm],
                                _PAIRS[self.pairs], self.eps)

    def c(self) -> L.GdnlRotateDims:
        return self._c


@dataclasses.dataclass
class StateCache:
    """State pages in 8 bits."""
    q: torch.Tensor      # [n_entries][h_v][d_k][d_v] int8
    scale: torch.Tensor  # [n_entries][h_v][d_k][ceil(d_v/64)] fp32

    @staticmethod
    def alloc(dims: LinearDims, n_entries: int, device) -> "StateCache":
        per = -(-dims.d_v // L.GDNL_CACHE_COLS)
        return StateCache(torch.zeros((n_entries, dims.h_v, dims.d_k, dims.d_v), dtype=torch.int8, device=device),
                          torch.zeros((n_entries, dims.h_v, dims.d_k, per), dtype=torch.float32, device=device))


class LinearGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dg: Optional[torch.Tensor]
    d_state0: torch.Tensor


class RotateGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dwq: Optional[torch.Tensor]
    dwk: Optional[torch.Tensor]


def gdnl_attend_workspace_bytes(dims: LinearDims, n_seqs: int, n_rows: int, backward: bool = False,
                                asks: Optional[tuple] = None) -> int:
    """asks: for backward calls alone that are given (dg, d_state, d_state0), three truth values."""
    out, d, what = ctypes.c_size_t(0), dims.c(), 1 if backward else 0
    if backward and asks is not None:
        what = L.GDNL_ASKS | sum(f for f, given in zip((L.GDNL_ASKS_DG, L.GDNL_ASKS_D_STATE, L.GDNL_ASKS_D_STATE0), asks) if given)
    _check("gdnl_attend_workspace_bytes",
           L.load().gdnl_attend_workspace_bytes(ctypes.byref(d), n_seqs, n_rows, what, ctypes.byref(out)))
    return int(out.value)


def gdnl_rotate_workspace_bytes(dims: RotateDims, n_rows: int) -> int:
    out, d = ctypes.c_size_t(0), dims.c()
    _check("gdnl_rotate_workspace_bytes",
           L.load().gdnl_rotate_workspace_bytes(ctypes.byref(d), n_rows, ctypes.byref(out)))
    return int(out.value)


def gdnl_cache_bytes(dims: LinearDims, n_entries: int) -> tuple:
    """(bytes of the 8-bit values, bytes of the scales)"""
    q, s, d = ctypes.c_size_t(0), ctypes.c_size_t(0), dims.c()
    _check("gdnl_cache_bytes", L.load().gdnl_cache_bytes(ctypes.byref(d), n_entries, ctypes.byref(q), ctypes.byref(s)))
    return int(q.value), int(s.value)


def _no_tangents(fn: str, *tensors: Optional[torch.Tensor]) -> None:
    """Within torch.autograd.forward_ad.dual_level() alone, which _current_level tells for less than a tensor's check."""
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            _no_history(fn)


def _check_pool(name: str, pool: StatePool, dims: LinearDims) -> None:
    t = pool.buf
    shape = (dims.h_v, dims.d_k, dims.d_v)
    if t.dtype is not _TORCH_DT[dims.state_dtype] or t.dim() != 4 or t.shape[1:] != shape or \
            not (t.is_contiguous() or t.shape[0] == 0 or t[0].is_contiguous()):  # t[0] costs 2 us
        raise ValueError(f"{name} must be [pages]{list(shape)} of {_TORCH_DT[dims.state_dtype]}, a page contiguous")


def _gates(g: torch.Tensor, rows: int, heads: int) -> int:
    """The row stride of g, 0 where it is one number for each head."""
    if g.dtype is not torch.float32:
        raise ValueError(f"g must be fp32, not {g.dtype}")
    if g.dim() == 1:
        _flat("g", g, (heads,), torch.float32)
        return 0
    return _rows2("g", g, rows, heads, torch.float32)


def _space(ws: Optional[torch.Tensor], size: int, dev: torch.device) -> torch.Tensor:
    if ws is None:
        return torch.empty(size, dtype=torch.uint8, device=dev)
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")  # its size is the library's to check
    _on(dev, workspace=ws)
    return ws


def _rows_out(name: str, t: Optional[torch.Tensor], like: torch.Tensor, rows: int, cols: int, dt: torch.dtype,
              dev: torch.device) -> tuple:
    """An output of [rows][cols] and its row stride: the caller's, checked, or a new one like `like`, checked before."""
    if t is None:
        return like.new_empty((rows, cols)), cols
    _on(dev, **{name: t})
    return t, _rows2(name, t, rows, cols, dt)


def gdnl_attend_forward(dims: LinearDims, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                        batch: Batch, state_in: StatePool, state_out: Optional[StatePool] = None,
                        o: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o [n_rows][h_v*d_v] (rows of no sequence and of padding left as they
    are); the final states go to state_out (default: state_in, in place).  g:
    fp32 [n_rows][h_v], or [h_v], the same for every row."""
    dev, n, dt = q.device, batch.n_rows, _TORCH_DT[dims.act_dtype]
    wk, wv = dims.h_k * dims.d_k, dims.h_v * dims.d_v
    state_out = state_in if state_out is None else state_out
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or g.requires_grad or
                                    state_in.buf.requires_grad):
        _no_history("gdnl_attend_forward")
    if forward_ad._current_level >= 0:
        _no_tangents("gdnl_attend_forward", q, k, v, g, state_in.buf)
    _on(dev, k=k, v=v, g=g, state_in=state_in.buf, state_out=state_out.buf, err=err)
    _check_batch(batch, dev)
    _check_pool("state_in", state_in, dims)
    if state_out is not state_in:
        _check_pool("state_out", state_out, dims)
    qs, ks = _rows2("q", q, n, wk, dt), _rows2("k", k, n, wk, dt)
    vs = _rows2("v", v, n, wv, dt)
    o, os_ = _rows_out("o", o, v, n, wv, dt, dev)
    gs = _gates(g, n, dims.h_v)
    if workspace is None and 0 < batch.max_seqlen <= L.GDNL_TOKEN_ROWS:
        ws, ws_bytes = None, 0  # row by row
    else:
        space = _space(workspace, 0 if workspace is not None else gdnl_attend_workspace_bytes(dims, batch.n_seqs, n), dev)
        ws, ws_bytes = space.data_ptr(), space.numel()
    d, bt = dims.c(), batch.c()
    _call("gdnl_attend_forward", dev,
          ctypes.byref(d), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), gs, ctypes.byref(bt),
          state_in.c(), state_out.c(), o.data_ptr(), os_, ws, ws_bytes, _err(err))
    return o


def gdnl_attend_backward(dims: LinearDims, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                         batch: Batch, state_in: StatePool, d_o: torch.Tensor, d_state: Optional[torch.Tensor] = None,
                         out: Optional[LinearGrads] = None, with_dg: bool = True,
                         workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None) -> LinearGrads:
    """The gradients of gdnl_attend_forward.  state_in: the pages as they were
    before the forward call; d_state [n_seqs][h_v][d_k][d_v] fp32: the gradient
    of the final states.  Rows of no sequence and of padding are left as they are
    in every output: give zeroed ones where something reads them.  An `out` whose
    dg is None, or with_dg False where there is no `out`: no gradient of the
    decays, which saves time."""
    dev, n, dt, s = q.device, batch.n_rows, _TORCH_DT[dims.act_dtype], batch.n_seqs
    wk, wv, one = dims.h_k * dims.d_k, dims.h_v * dims.d_v, g.dim() == 1
    state = (s, dims.h_v, dims.d_k, dims.d_v)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or g.requires_grad or
                                    state_in.buf.requires_grad or d_o.requires_grad or
                                    (d_state is not None and d_state.requires_grad)):
        _no_history("gdnl_attend_backward")
    if forward_ad._current_level >= 0:
        _no_tangents("gdnl_attend_backward", q, k, v, g, state_in.buf, d_o, d_state)
    _on(dev, k=k, v=v, g=g, d_o=d_o, d_state=d_state, state_in=state_in.buf, err=err)
    _check_batch(batch, dev)
    _check_pool("state_in", state_in, dims)
    qs, ks, vs = _rows2("q", q, n, wk, dt), _rows2("k", k, n, wk, dt), _rows2("v", v, n, wv, dt)
    os_, gs = _rows2("d_o", d_o, n, wv, dt), _gates(g, n, dims.h_v)
    if gs == 0 and not one:  # one row expanded over all: its gradient is each row's
        g, gs = g.contiguous(), dims.h_v
    _flat("d_state", d_state, state, torch.float32)
    if out is None:
        out = LinearGrads(q.new_empty((n, wk)), q.new_empty((n, wk)), q.new_empty((n, wv)),
                          g.new_empty((dims.h_v,) if one else (n, dims.h_v)) if with_dg else None, g.new_empty(state))
        dqs, dks, dvs = wk, wk, wv
    else:
        _on(dev, **out._asdict())
        dqs, dks, dvs = _rows2("dq", out.dq, n, wk, dt), _rows2("dk", out.dk, n, wk, dt), _rows2("dv", out.dv, n, wv, dt)
        _flat("dg", out.dg, (dims.h_v,) if one else (n, dims.h_v), torch.float32)
        _flat("d_state0", out.d_state0, state, torch.float32)
    asks = out.dg is not None, d_state is not None, out.d_state0 is not None
    space = _space(workspace, 0 if workspace is not None else gdnl_attend_workspace_bytes(dims, s, n, True, asks), dev)
    d, bt = dims.c(), batch.c()
    _call("gdnl_attend_backward", dev,
          ctypes.byref(d), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), gs, ctypes.byref(bt),
          state_in.c(), d_o.data_ptr(), os_, _p(d_state), out.dq.data_ptr(), dqs, out.dk.data_ptr(), dks,
          out.dv.data_ptr(), dvs, _p(out.dg), _p(out.d_state0), space.data_ptr(), space.numel(), _err(err))
    return out


def _rotate_inputs(dims: RotateDims, q, k, wq, wk, pos, inv_freq) -> tuple:
    n, dt, dev = q.shape[0], _TORCH_DT[dims.act_dtype], q.device
    _on(dev, k=k, wq=wq, wk=wk, pos=pos, inv_freq=inv_freq)
    _flat("wq", wq, (dims.d,), torch.float32)
    _flat("wk", wk, (dims.d,), torch.float32)
    _flat("pos", pos, (n,), torch.int32)
    _flat("inv_freq", inv_freq, (dims.rot // 2,), torch.float32)
    if dims.rot > 0 and (pos is None or inv_freq is None):
        raise ValueError("a rotation needs pos and inv_freq")
    return n, dt, dev, _rows2("q", q, n, dims.h_q * dims.d, dt), _rows2("k", k, n, dims.h_k * dims.d, dt)


def gdnl_rotate_forward(dims: RotateDims, q: torch.Tensor, k: torch.Tensor, wq: Optional[torch.Tensor],
                        wk: Optional[torch.Tensor], pos: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                        yq: Optional[torch.Tensor] = None, yk: Optional[torch.Tensor] = None) -> tuple:
    """(yq, yk): every head of q [n_rows][h_q*d] and k [n_rows][h_k*d] normed,
    weighted by wq or wk (fp32 [d], None: ones) and rotated by pos (int32
    [n_rows]) times inv_freq (fp32 [rot/2]).  yq may be q, and yk k."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, wq, wk)):
        _no_history("gdnl_rotate_forward")
    if forward_ad._current_level >= 0:
        _no_tangents("gdnl_rotate_forward", q, k, wq, wk)
    n, dt, dev, qs, ks = _rotate_inputs(dims, q, k, wq, wk, pos, inv_freq)
    yq, yqs = _rows_out("yq", yq, q, n, dims.h_q * dims.d, dt, dev)
    yk, yks = _rows_out("yk", yk, q, n, dims.h_k * dims.d, dt, dev)
    d = dims.c()
    _call("gdnl_rotate_forward", dev, ctypes.byref(d), q.data_ptr(), qs, k.data_ptr(), ks, _p(wq), _p(wk), _p(pos),
          _p(inv_freq), n, yq.data_ptr(), yqs, yk.data_ptr(), yks)
    return yq, yk


def gdnl_rotate_backward(dims: RotateDims, q: torch.Tensor, k: torch.Tensor, wq: Optional[torch.Tensor],
                         wk: Optional[torch.Tensor], pos: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                         d_yq: torch.Tensor, d_yk: torch.Tensor, out: Optional[RotateGrads] = None,
                         workspace: Optional[torch.Tensor] = None) -> RotateGrads:
    """The gradients of gdnl_rotate_forward at its inputs q and k.  out.dq may
    be d_yq and out.dk d_yk; an `out` whose dwq or dwk is None leaves it out, as
    does a weight of None."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, wq, wk, d_yq, d_yk)):
        _no_history("gdnl_rotate_backward")
    if forward_ad._current_level >= 0:
        _no_tangents("gdnl_rotate_backward", q, k, wq, wk, d_yq, d_yk)
    n, dt, dev, qs, ks = _rotate_inputs(dims, q, k, wq, wk, pos, inv_freq)
    nq, nk = dims.h_q * dims.d, dims.h_k * dims.d
    _on(dev, d_yq=d_yq, d_yk=d_yk)
    yqs, yks = _rows2("d_yq", d_yq, n, nq, dt), _rows2("d_yk", d_yk, n, nk, dt)
    if out is None:
        out = RotateGrads(q.new_empty((n, nq)), q.new_empty((n, nk)), None if wq is None else wq.new_empty(dims.d),
                          None if wk is None else wk.new_empty(dims.d))
        dqs, dks = nq, nk
    else:
        _on(dev, **out._asdict())
        dqs, dks = _rows2("dq", out.dq, n, nq, dt), _rows2("dk", out.dk, n, nk, dt)
        _flat("dwq", out.dwq, (dims.d,), torch.float32)
        _flat("dwk", out.dwk, (dims.d,), torch.float32)
    space = _space(workspace, 0 if workspace is not None else gdnl_rotate_workspace_bytes(dims, n), dev)
    d = dims.c()
    _call("gdnl_rotate_backward", dev, ctypes.byref(d), q.data_ptr(), qs, k.data_ptr(), ks, _p(wq), _p(wk), _p(pos),
          _p(inv_freq), n, d_yq.data_ptr(), yqs, d_yk.data_ptr(), yks, out.dq.data_ptr(), dqs, out.dk.data_ptr(), dks,
          _p(out.dwq), _p(out.dwk), space.data_ptr(), space.numel())
    return out


def _cache_call(fn: str, dims: LinearDims, first: tuple, second: tuple, pool: StatePool, cache: StateCache, err,
                store: bool) -> None:
    dev, n = pool.buf.device, first[1].numel()
    if torch.is_grad_enabled() and pool.buf.requires_grad:
        _no_history(fn)
    if forward_ad._current_level >= 0:
        _no_tangents(fn, pool.buf)
    _on(dev, **{first[0]: first[1], second[0]: second[1]}, q=cache.q, scale=cache.scale, err=err)
    for name, t in (first, second):
        _flat(name, t, (n,), torch.int32)
    _check_pool("state", pool, dims)
    e, per = cache.q.shape[0], -(-dims.d_v // L.GDNL_CACHE_COLS)
    _flat("cache.q", cache.q, (e, dims.h_v, dims.d_k, dims.d_v), torch.int8)
    _flat("cache.scale", cache.scale, (e, dims.h_v, dims.d_k, per), torch.float32)
    d, c = dims.c(), L.GdnlCache(cache.q.data_ptr(), cache.scale.data_ptr(), e)
    tail = (pool.c(), ctypes.byref(c)) if store else (ctypes.byref(c), pool.c())
    _call(fn, dev, ctypes.byref(d), n, first[1].data_ptr(), second[1].data_ptr(), *tail, _err(err))


def gdnl_cache_store(dims: LinearDims, page_idx: torch.Tensor, entry: torch.Tensor, state: StatePool,
                     cache: StateCache, err: Optional[torch.Tensor] = None) -> None:
    """Entry entry[i] <- state page page_idx[i]; an index < 0 in either (int32
    [n]) skips the pair.  Entries of one call must be distinct."""
    _cache_call("gdnl_cache_store", dims, ("page_idx", page_idx), ("entry", entry), state, cache, err, True)


def gdnl_cache_load(dims: LinearDims, entry: torch.Tensor, page_idx: torch.Tensor, cache: StateCache,
                    state: StatePool, err: Optional[torch.Tensor] = None) -> None:
    """State page page_idx[i] <- entry entry[i].  Pages of one call must be
    distinct."""
    _cache_call("gdnl_cache_load", dims, ("entry", entry), ("page_idx", page_idx), state, cache, err, False)
