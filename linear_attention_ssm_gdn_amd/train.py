"""Torch-facing binding of include/gdn_train.h: the vector-state gated
recurrence, its backward pass and the conv's backward pass.

As in ops.py every function checks its tensors, turns them into device
pointers, strides and sizes, calls the C entry point on the current HIP
stream of the tensors' device and raises on a non-OK status.  Outputs and
workspaces that are not given are allocated.

Autograd records nothing here: the backward pass is called by hand, or from
the backward of a torch.autograd.Function whose forward calls the forward
pass.  A call whose history would be lost in silence is refused: gradients
enabled, and a tensor that requires one among the inputs of the forward pass
(or among the gradients given to a backward pass, which has none of its own).
Call it under torch.no_grad() or with detached tensors.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .ops import _DT, _TORCH_DT, Batch, ConvPool, Dims, StatePool, _check

_NAMES = {v: k for k, v in _TORCH_DT.items()}


@dataclasses.dataclass(frozen=True)
class ScanDims:
    channels: int
    act_dtype: str = "bf16"
    state_dtype: str = "f32"

    @property
    def act_torch(self) -> torch.dtype:
        return _TORCH_DT[self.act_dtype]

    @property
    def state_torch(self) -> torch.dtype:
        return _TORCH_DT[self.state_dtype]

    @functools.cached_property
    def _c(self) -> L.GdntScanDims:
        return L.GdntScanDims(self.channels, _DT[self.act_dtype], _DT[self.state_dtype])

    def c(self) -> L.GdntScanDims:
        return self._c  # the library only reads it


@dataclasses.dataclass
class ScanParams:
    a_log: torch.Tensor    # [channels] fp32
    dt_bias: torch.Tensor  # [channels] fp32

    def c(self) -> L.GdntScanParams:
        return L.GdntScanParams(self.a_log.data_ptr(), self.dt_bias.data_ptr())


@dataclasses.dataclass
class ScanSaved:
    """What a forward call keeps for its backward call."""
    states: torch.Tensor                    # [ceil(n_rows/256)][channels] fp32
    ckpt: Optional[torch.Tensor] = None     # uint8: x, a and b in 8 bits

    @staticmethod
    def alloc(dims: ScanDims, n_rows: int, device, ckpt: bool = False) -> "ScanSaved":
        states, q = gdnt_scan_saved_bytes(dims, n_rows)
        return ScanSaved(torch.empty((states // (4 * dims.channels), dims.channels), dtype=torch.float32, device=device),
                         torch.empty(q, dtype=torch.uint8, device=device) if ckpt else None)


class ScanGrads(NamedTuple):
    dx: torch.Tensor
    da: torch.Tensor
    db: torch.Tensor
    d_a_log: torch.Tensor
    d_dt_bias: torch.Tensor
    d_state0: torch.Tensor


class ConvGrads(NamedTuple):
    dx: torch.Tensor
    d_conv_w: torch.Tensor
    d_window0: torch.Tensor


def gdnt_scan_workspace_bytes(dims: ScanDims, n_seqs: int, n_rows: int) -> int:
    out, d = ctypes.c_size_t(0), dims.c()
    _check("gdnt_scan_workspace_bytes",
           L.load().gdnt_scan_workspace_bytes(ctypes.byref(d), n_seqs, n_rows, ctypes.byref(out)))
    return int(out.value)


def gdnt_scan_saved_bytes(dims: ScanDims, n_rows: int) -> tuple:
    """(bytes of the kept states, bytes of the 8-bit checkpoint)"""
    st, q, d = ctypes.c_size_t(0), ctypes.c_size_t(0), dims.c()
    _check("gdnt_scan_saved_bytes",
           L.load().gdnt_scan_saved_bytes(ctypes.byref(d), n_rows, ctypes.byref(st), ctypes.byref(q)))
    return int(st.value), int(q.value)


def gdnt_conv_workspace_bytes(dims: Dims, n_seqs: int, n_rows: int) -> int:
    out, d = ctypes.c_size_t(0), dims.c()
    _check("gdnt_conv_workspace_bytes",
           L.load().gdnt_conv_workspace_bytes(ctypes.byref(d), n_seqs, n_rows, ctypes.byref(out)))
    return int(out.value)


def _on(dev: torch.device, **tensors) -> None:
    where = -1 if dev.index is None else dev.index  # the host's tensors give -1
    for name, t in tensors.items():
        if t is not None and t.get_device() != where:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _rows2(name: str, t: torch.Tensor, rows: int, cols: int, dt: torch.dtype) -> int:
    """The row stride of a [rows][cols] tensor."""
    if t.dtype is not dt:
        raise ValueError(f"{name} must be {dt}, not {t.dtype}")
    st = t.stride()
    if t.shape != (rows, cols) or (cols > 1 and st[1] != 1):
        raise ValueError(f"{name} must be [{rows}][{cols}] with unit inner stride")
    return st[0] if rows > 1 else cols


def _flat(name: str, t: Optional[torch.Tensor], shape: tuple, dt: torch.dtype) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not dt or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {list(shape)}")
    return t.data_ptr()


def _err(err: Optional[torch.Tensor]) -> Optional[int]:
    if err is not None and (err.dtype is not torch.int32 or err.numel() < 1):
        raise ValueError("err must be an int32 tensor")
    return _p(err)


def _no_history(fn: str) -> None:
    raise ValueError(f"{fn} records nothing for autograd, but one of its tensors requires a gradient: call it "
                     "under torch.no_grad() or with detached tensors, and the backward pass by hand")


def _check_batch(batch: Batch, dev: torch.device) -> None:
    n = batch.n_seqs
    _on(dev, cu_seqlens=batch.cu_seqlens, page_idx=batch.page_idx, has_init=batch.has_init)
    _flat("cu_seqlens", batch.cu_seqlens, (n + 1,), torch.int32)
    _flat("page_idx", batch.page_idx, (n,), torch.int32)
    _flat("has_init", batch.has_init, (n,), torch.uint8)


def _check_state_pool(name: str, pool: StatePool, dims: ScanDims) -> None:
    t = pool.buf
    if t.dtype is not dims.state_torch or t.dim() != 2 or t.shape[1] != dims.channels or \
            (dims.channels > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [pages][{dims.channels}] of {dims.state_torch} with unit inner stride")


def _check_params(params: ScanParams, dims: ScanDims) -> None:
    _flat("a_log", params.a_log, (dims.channels,), torch.float32)
    _flat("dt_bias", params.dt_bias, (dims.channels,), torch.float32)


def _workspace(ws: Optional[torch.Tensor], size, dims, n_seqs: int, n_rows: int, dev: torch.device) -> torch.Tensor:
    if ws is None:
        return torch.empty(size(dims, n_seqs, n_rows), dtype=torch.uint8, device=dev)
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")  # its size is the library's to check
    _on(dev, workspace=ws)
    return ws


def _call(fn: str, dev: torch.device, *args) -> None:
    """The C entry point on the current stream of `dev`, with `dev` current."""
    if dev.type != "cuda":  # a kernel would fault on host memory
        raise ValueError(f"{fn} takes tensors on a GPU, not on {dev}")
    f, here = getattr(L.load(), fn), torch.cuda.current_device()
    if dev.index is None or dev.index == here:
        st = f(*args, torch._C._cuda_getCurrentRawStream(here))  # 2 us less than through a Stream object
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        _check(fn, st)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_saved(saved: ScanSaved, dims: ScanDims, n_rows: int, dev: torch.device) -> None:
    states, q = gdnt_scan_saved_bytes(dims, n_rows)
    _on(dev, states=saved.states, ckpt=saved.ckpt)
    _flat("states", saved.states, (states // (4 * dims.channels), dims.channels), torch.float32)
    _flat("ckpt", saved.ckpt, (q,), torch.uint8)


def gdnt_scan_forward(dims: ScanDims, params: ScanParams, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                      batch: Batch, state_in: StatePool, state_out: Optional[StatePool] = None,
                      h: Optional[torch.Tensor] = None, saved: Optional[ScanSaved] = None,
                      workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h [n_rows][channels] (rows of no sequence and of padding left as they
    are); the final states go to state_out (default: state_in, in place).
    `saved` receives what gdnt_scan_backward needs, x, a and b in 8 bits among
    it where it has a ckpt."""
    dev, n, C, dt = x.device, batch.n_rows, dims.channels, dims.act_torch
    state_out = state_in if state_out is None else state_out
    if torch.is_grad_enabled() and (x.requires_grad or a.requires_grad or b.requires_grad or
                                    params.a_log.requires_grad or params.dt_bias.requires_grad or
                                    state_in.buf.requires_grad):
        _no_history("gdnt_scan_forward")
    if h is None:
        h = torch.empty((n, C), dtype=dt, device=dev)
    _on(dev, a=a, b=b, h=h, state_in=state_in.buf, state_out=state_out.buf, a_log=params.a_log,
        dt_bias=params.dt_bias, err=err)
    _check_params(params, dims)
    _check_batch(batch, dev)
    _check_state_pool("state_in", state_in, dims)
    _check_state_pool("state_out", state_out, dims)
    xs, hs = _rows2("x", x, n, C, dt), _rows2("h", h, n, C, dt)
    as_, bs = _rows2("a", a, n, C, dt), _rows2("b", b, n, C, dt)
    if as_ != bs:
        raise ValueError("a and b must share their row stride")
    if saved is not None:
        _check_saved(saved, dims, n, dev)
    ws = _workspace(workspace, gdnt_scan_workspace_bytes, dims, batch.n_seqs, n, dev)
    d, p, bt = dims.c(), params.c(), batch.c()
    _call("gdnt_scan_forward", dev,
          ctypes.byref(d), ctypes.byref(p), x.data_ptr(), xs, a.data_ptr(), b.data_ptr(), as_, ctypes.byref(bt),
          state_in.c(), state_out.c(), h.data_ptr(), hs, _p(saved.states) if saved is not None else None,
          _p(saved.ckpt) if saved is not None else None, ws.data_ptr(), ws.numel(), _err(err))
    return h


def gdnt_scan_backward(dims: ScanDims, params: ScanParams, batch: Batch, state_in: StatePool, saved: ScanSaved,
                       dh: torch.Tensor, x: Optional[torch.Tensor] = None, a: Optional[torch.Tensor] = None,
                       b: Optional[torch.Tensor] = None, d_state: Optional[torch.Tensor] = None,
                       out: Optional[ScanGrads] = None, workspace: Optional[torch.Tensor] = None,
                       err: Optional[torch.Tensor] = None) -> ScanGrads:
    """The gradients of gdnt_scan_forward, from x, a and b, or from the 8 bits
    in `saved` where these are not given.  state_in: the pages as they were
    before the forward call; d_state [n_seqs][channels] fp32: the gradient of
    the final states.  Rows of no sequence and of padding are left as they
    are in every output: give zeroed ones where something reads them."""
    dev, n, C, s, dt = dh.device, batch.n_rows, dims.channels, batch.n_seqs, dims.act_torch
    if torch.is_grad_enabled() and (dh.requires_grad or (d_state is not None and d_state.requires_grad)):
        _no_history("gdnt_scan_backward")
    given = [t is not None for t in (x, a, b)]
    if any(given) and not all(given):
        raise ValueError("x, a and b go together")
    if not any(given) and saved.ckpt is None:
        raise ValueError("a backward pass needs x, a and b, or a checkpoint")
    if out is None:
        out = ScanGrads(*(torch.empty((n, C), dtype=dt, device=dev) for _ in range(3)),
                        *(torch.empty(C, dtype=torch.float32, device=dev) for _ in range(2)),
                        torch.empty((s, C), dtype=torch.float32, device=dev))
    _on(dev, x=x, a=a, b=b, d_state=d_state, state_in=state_in.buf, a_log=params.a_log, dt_bias=params.dt_bias,
        err=err, **out._asdict())
    _check_params(params, dims)
    _check_batch(batch, dev)
    _check_state_pool("state_in", state_in, dims)
    _check_saved(saved, dims, n, dev)
    xs = as_ = bs = 0
    if all(given):
        xs, as_, bs = _rows2("x", x, n, C, dt), _rows2("a", a, n, C, dt), _rows2("b", b, n, C, dt)
    hs, dxs = _rows2("dh", dh, n, C, dt), _rows2("dx", out.dx, n, C, dt)
    das, dbs = _rows2("da", out.da, n, C, dt), _rows2("db", out.db, n, C, dt)
    if as_ != bs or das != dbs:
        raise ValueError("a and b, and da and db, must share their row stride")
    _flat("d_state", d_state, (s, C), torch.float32)
    _flat("d_a_log", out.d_a_log, (C,), torch.float32)
    _flat("d_dt_bias", out.d_dt_bias, (C,), torch.float32)
    _flat("d_state0", out.d_state0, (s, C), torch.float32)
    ws = _workspace(workspace, gdnt_scan_workspace_bytes, dims, s, n, dev)
    d, p, bt = dims.c(), params.c(), batch.c()
    _call("gdnt_scan_backward", dev,
          ctypes.byref(d), ctypes.byref(p), _p(x), xs, _p(a), _p(b), as_, None if all(given) else _p(saved.ckpt),
          ctypes.byref(bt), state_in.c(), saved.states.data_ptr(), dh.data_ptr(), hs, _p(d_state),
          out.dx.data_ptr(), dxs, out.da.data_ptr(), out.db.data_ptr(), das, out.d_a_log.data_ptr(),
          out.d_dt_bias.data_ptr(), out.d_state0.data_ptr(), ws.data_ptr(), ws.numel(), _err(err))
    return out


def gdnt_conv_backward(dims: Dims, conv_w: torch.Tensor, x: torch.Tensor, dy: torch.Tensor, batch: Batch,
                       conv: Optional[ConvPool] = None, activation: bool = True,
                       d_window: Optional[torch.Tensor] = None, out: Optional[ConvGrads] = None,
                       workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None) -> ConvGrads:
    """The gradients of gdn_conv_update.  conv: the windows as they were
    before the forward call (its sync words are not used), or None when no
    sequence has one; d_window [n_seqs][conv_w-1][C_conv] fp32: the gradient
    of the rolled windows.  Rows of no sequence and of padding are left as
    they are in dx: give a zeroed one where something reads them."""
    dev, n, C, s, k = x.device, batch.n_rows, dims.c_conv, batch.n_seqs, dims.conv_w - 1
    if torch.is_grad_enabled() and (dy.requires_grad or (d_window is not None and d_window.requires_grad)):
        _no_history("gdnt_conv_backward")
    if dy.dtype not in _NAMES:
        raise ValueError(f"dy must be fp32 or bf16, not {dy.dtype}")
    if out is None:
        out = ConvGrads(torch.empty((n, C), dtype=dims.act_torch, device=dev),
                        torch.empty((C, dims.conv_w), dtype=torch.float32, device=dev),
                        torch.empty((s, k, C), dtype=torch.float32, device=dev))
    _on(dev, conv_w=conv_w, dy=dy, conv=conv.buf if conv is not None else None, d_window=d_window, err=err,
        **out._asdict())
    _check_batch(batch, dev)
    _flat("conv_w", conv_w, (C, dims.conv_w), dims.act_torch)
    cp = L.GdnConvPool(None, 0, 0, 0, None)
    if conv is not None:
        t = conv.buf
        if t.dtype != dims.act_torch or t.dim() != 3 or t.shape[1] < k or t.shape[2] != C or \
                t.stride(2) != 1 or t.stride(1) != C:
            raise ValueError(f"conv must be [pages][>= {k}][{C}] of {dims.act_torch}, rows contiguous")
        cp = L.GdnConvPool(t.data_ptr(), t.stride(0), t.shape[1], t.shape[0], None)
    xs, dxs = _rows2("x", x, n, C, dims.act_torch), _rows2("dx", out.dx, n, C, dims.act_torch)
    ys = _rows2("dy", dy, n, C, dy.dtype)
    _flat("d_window", d_window, (s, k, C), torch.float32)
    _flat("d_conv_w", out.d_conv_w, (C, dims.conv_w), torch.float32)
    _flat("d_window0", out.d_window0, (s, k, C), torch.float32)
    ws = _workspace(workspace, gdnt_conv_workspace_bytes, dims, s, n, dev)
    d, bt = dims.c(), batch.c()
    _call("gdnt_conv_backward", dev,
          ctypes.byref(d), conv_w.data_ptr(), x.data_ptr(), xs, dy.data_ptr(), _DT[_NAMES[dy.dtype]], ys,
          ctypes.byref(bt), cp, 1 if activation else 0, _p(d_window), out.dx.data_ptr(), dxs,
          out.d_conv_w.data_ptr(), out.d_window0.data_ptr(), ws.data_ptr(), ws.numel(), _err(err))
    return out
