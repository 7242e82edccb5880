"""Operators around a recurrent layer: the short causal convolution, the
selective state-space scan, and the gradient norm with its clipping.

The e2ttt_* functions mirror the C entry points of include/e2ttt.h one to one
(torch tensors or raw device pointers, no checks of their own). The others take
torch tensors, check them (device, type, shape, contiguity: E2TTTError with
ERR_INVALID_ARG), allocate outputs and workspace with torch, and run on the
current stream of the tensors' device or on `stream` (a torch stream or a raw
handle; outputs are then allocated on it). None of them records autograd: the
gradients are functions of their own, as for chunk_scan_bwd.
"""
from __future__ import annotations

import contextlib
import ctypes
from array import array

import torch

from . import (BF16, ERR_INVALID_ARG, E2TTTError, F32, _check, _lib, _P, _ptr, _stream)


class e2ttt_conv_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "T", "d", "W", "act", "silu")]


class e2ttt_ssm_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "G", "T", "d_k", "d_v", "act")]


_C = ctypes.POINTER(e2ttt_conv_shape)
_M = ctypes.POINTER(e2ttt_ssm_shape)
_Z, _I = ctypes.c_size_t, ctypes.c_int
for _name, (_res, _args) in {
    "e2ttt_short_conv_workspace_bytes": (_Z, [_C]),
    "e2ttt_short_conv_fwd": (_I, [_C] + [_P] * 8),
    "e2ttt_short_conv_bwd": (_I, [_C] + [_P] * 12 + [_Z, _P]),
    "e2ttt_short_conv_step": (_I, [_C] + [_P] * 6),
    "e2ttt_ssm_workspace_bytes": (_Z, [_M, _I]),
    "e2ttt_ssm_saved_bytes": (_Z, [_M]),
    "e2ttt_ssm_scan_fwd": (_I, [_M] + [_P] * 12 + [_Z, _P]),
    "e2ttt_ssm_scan_bwd": (_I, [_M] + [_P] * 18 + [_Z, _P]),
    "e2ttt_ssm_step": (_I, [_M] + [_P] * 9),
    "e2ttt_grad_workspace_bytes": (_Z, [_I]),
    "e2ttt_grad_norm": (_I, [_P, _P, _P, _I, _P, _P, _Z, _P]),
    "e2ttt_clip_grad_norm": (_I, [_P, _P, _P, _P, _I, ctypes.c_float, _P, _P, _Z, _P]),
}.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

_ACT = {torch.bfloat16: BF16, torch.float32: F32}


# ---------------------------------------------------------------- C entry points
def make_conv_shape(B, H, T, d, W, act=BF16, silu=True) -> e2ttt_conv_shape:
    return e2ttt_conv_shape(B, H, T, d, W, act, int(silu))


def make_ssm_shape(B, H, G, T, d_k, d_v, act=BF16) -> e2ttt_ssm_shape:
    return e2ttt_ssm_shape(B, H, G, T, d_k, d_v, act)


def _nbytes(workspace):
    return workspace.numel() * workspace.element_size()


def _done(st, raw):
    if raw:
        return st
    _check(st)


def e2ttt_short_conv_workspace_bytes(shape) -> int:
    return _lib.e2ttt_short_conv_workspace_bytes(ctypes.byref(shape))


def e2ttt_short_conv_fwd(shape, x, w, bias, state, lengths, y, state_end, stream=None, raw=False):
    return _done(_lib.e2ttt_short_conv_fwd(
        ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(y),
        _ptr(state_end), _stream(stream) if not raw else stream), raw)


def e2ttt_short_conv_bwd(shape, x, w, bias, state, lengths, dy, dstate_end, dx, dw, dbias, dstate,
                         workspace, workspace_bytes=None, stream=None, raw=False):
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    return _done(_lib.e2ttt_short_conv_bwd(
        ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(dy),
        _ptr(dstate_end), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(dstate), _ptr(workspace),
        workspace_bytes, _stream(stream) if not raw else stream), raw)


def e2ttt_short_conv_step(shape, x, w, bias, state, y, stream=None, raw=False):
    return _done(_lib.e2ttt_short_conv_step(
        ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(y),
        _stream(stream) if not raw else stream), raw)


def e2ttt_ssm_workspace_bytes(shape, for_bwd=0) -> int:
    return _lib.e2ttt_ssm_workspace_bytes(ctypes.byref(shape), int(for_bwd))


def e2ttt_ssm_saved_bytes(shape) -> int:
    return _lib.e2ttt_ssm_saved_bytes(ctypes.byref(shape))


def e2ttt_ssm_scan_fwd(shape, q, k, v, dt, A, D, S0, lengths, y, S_end, saved_states, workspace,
                       workspace_bytes=None, stream=None, raw=False):
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    return _done(_lib.e2ttt_ssm_scan_fwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(A), _ptr(D), _ptr(S0),
        _ptr(lengths), _ptr(y), _ptr(S_end), _ptr(saved_states), _ptr(workspace), workspace_bytes,
        _stream(stream) if not raw else stream), raw)


def e2ttt_ssm_scan_bwd(shape, q, k, v, dt, A, D, lengths, saved_states, dy, dS_end, dq, dk, dv, ddt,
                       dA, dD, dS0, workspace, workspace_bytes=None, stream=None, raw=False):
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    return _done(_lib.e2ttt_ssm_scan_bwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(A), _ptr(D), _ptr(lengths),
        _ptr(saved_states), _ptr(dy), _ptr(dS_end), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ddt),
        _ptr(dA), _ptr(dD), _ptr(dS0), _ptr(workspace), workspace_bytes,
        _stream(stream) if not raw else stream), raw)


def e2ttt_ssm_step(shape, q, k, v, dt, A, D, S, y, stream=None, raw=False):
    return _done(_lib.e2ttt_ssm_step(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(A), _ptr(D), _ptr(S), _ptr(y),
        _stream(stream) if not raw else stream), raw)


def e2ttt_grad_workspace_bytes(count) -> int:
    return _lib.e2ttt_grad_workspace_bytes(int(count))


def _lists(g, out, n, act):
    """Host arrays of the lists: device pointers, element counts, types."""
    held = [array("Q", g), array("Q", out) if out is not None else None, array("Q", n),
            array("i", act)]
    return held, [h.buffer_info()[0] if h else None for h in held]


def e2ttt_grad_norm(g, n, act, norm, workspace, workspace_bytes=None, stream=None, raw=False):
    """g, n, act: equally long lists of device pointers, element counts and types."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    held, (pg, _, pn, pa) = _lists(g, None, n, act)
    return _done(_lib.e2ttt_grad_norm(pg, pn, pa, len(g), _ptr(norm), _ptr(workspace),
                                      workspace_bytes, _stream(stream) if not raw else stream), raw)


def e2ttt_clip_grad_norm(g, out, n, act, max_norm, norm, workspace, workspace_bytes=None,
                         stream=None, raw=False):
    """out: a list of device pointers (0: in place) or None (all in place)."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    held, (pg, po, pn, pa) = _lists(g, out, n, act)
    return _done(_lib.e2ttt_clip_grad_norm(pg, po, pn, pa, len(g), max_norm, _ptr(norm),
                                           _ptr(workspace), workspace_bytes,
                                           _stream(stream) if not raw else stream), raw)


# ---------------------------------------------------------------- checks
def _refuse(what):
    raise E2TTTError(ERR_INVALID_ARG, what)


def _need(name, t, shape, dtype, device):
    """t is a contiguous CUDA tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor):
        _refuse(f"{name} must be a tensor, got {type(t).__name__}")
    if t.shape != shape:
        _refuse(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        _refuse(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        _refuse(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")


def _may(name, t, shape, dtype, device):
    if t is not None:
        _need(name, t, shape, dtype, device)


def _first(name, t, dims):
    """The tensor that fixes sizes, type and device."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        _refuse(f"{name} must be a tensor of {dims} dimensions")
    if not t.is_cuda:
        _refuse(f"{name} must be on a CUDA device, got {t.device}")
    if t.dtype not in _ACT:
        _refuse(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


@contextlib.contextmanager
def _guard(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device)
            elif stream.device != device:
                _refuse(f"the stream is on {stream.device}, the tensors are on {device}")
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Makes `device` current, and `stream` where one is given."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _HERE
    return _guard(device, stream)


def _scratch(ws, need, device):
    if ws is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        _refuse(f"ws must be a contiguous tensor on {device}")
    return ws


# ---------------------------------------------------------------- short convolution
def _conv_check(x, w, bias, state, lengths, silu):
    B, H, T, d = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        _refuse("w must be [H, d, W]")
    W = w.shape[2]
    dev, f32 = x.device, torch.float32
    _need("x", x, x.shape, x.dtype, dev)
    _need("w", w, (H, d, W), f32, dev)
    _may("bias", bias, (H, d), f32, dev)
    _may("state", state, (B, H, W - 1, d), x.dtype, dev)
    _may("lengths", lengths, (B,), torch.int32, dev)
    return e2ttt_conv_shape(B, H, T, d, W, _ACT[x.dtype], 1 if silu else 0)


def short_conv_fwd(x, w, bias=None, state=None, lengths=None, *, silu=True, return_state=False,
                   stream=None):
    """Short causal depthwise convolution: x [B, H, T, d] (bf16 or fp32), w
    [H, d, W] and bias [H, d] fp32, state [B, H, W-1, d] (the inputs before the
    first token; None: zeros), lengths int32 [B] (a padded batch). Returns (y,
    state_end), state_end None unless return_state."""
    _first("x", x, 4)
    shape = _conv_check(x, w, bias, state, lengths, silu)
    with _on(x.device, stream):
        y = torch.empty_like(x)
        end = (torch.empty((shape.B, shape.H, shape.W - 1, shape.d), dtype=x.dtype, device=x.device)
               if return_state else None)
        e2ttt_short_conv_fwd(shape, x, w, bias, state, lengths, y, end)
    return y, end


def short_conv_bwd(x, w, dy, bias=None, state=None, dstate_end=None, lengths=None, *, silu=True,
                   ws=None, stream=None):
    """Gradients of short_conv_fwd for <dy, y> + <dstate_end, state_end>: a dict
    dx, dw, dbias (None without bias), dstate (None without state)."""
    _first("x", x, 4)
    shape = _conv_check(x, w, bias, state, lengths, silu)
    dev = x.device
    _need("dy", dy, x.shape, x.dtype, dev)
    _may("dstate_end", dstate_end, (shape.B, shape.H, shape.W - 1, shape.d), x.dtype, dev)
    with _on(dev, stream):
        g = dict(dx=torch.empty_like(x), dw=torch.empty_like(w),
                 dbias=None if bias is None else torch.empty_like(bias),
                 dstate=None if state is None else torch.empty_like(state))
        ws = _scratch(ws, _bytes(e2ttt_short_conv_workspace_bytes(shape)), dev)
        e2ttt_short_conv_bwd(shape, x, w, bias, state, lengths, dy, dstate_end, g["dx"], g["dw"],
                             g["dbias"], g["dstate"], ws)
    return g


def short_conv_step(x, state, w, bias=None, *, silu=True, out=None, stream=None):
    """One token per row: x [B, H, d], state [B, H, W-1, d] updated in place.
    Returns y [B, H, d] (`out` where given)."""
    _first("x", x, 3)
    B, H, d = x.shape
    dev = x.device
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        _refuse("w must be [H, d, W]")
    W = w.shape[2]
    _need("x", x, x.shape, x.dtype, dev)
    _need("w", w, (H, d, W), torch.float32, dev)
    _may("bias", bias, (H, d), torch.float32, dev)
    _need("state", state, (B, H, W - 1, d), x.dtype, dev)
    _may("out", out, x.shape, x.dtype, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x)
        e2ttt_short_conv_step(e2ttt_conv_shape(B, H, 1, d, W, _ACT[x.dtype], 1 if silu else 0), x, w,
                              bias, state, out)
    return out


# ---------------------------------------------------------------- state-space scan
def _ssm_check(q, k, v, dt, A, D, lengths):
    B, H, T, d_v = v.shape
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        _refuse("q must be [B, G, T, d_k]")
    G, d_k = q.shape[1], q.shape[3]
    dev, f32 = v.device, torch.float32
    _need("v", v, v.shape, v.dtype, dev)
    _need("q", q, (B, G, T, d_k), v.dtype, dev)
    _need("k", k, (B, G, T, d_k), v.dtype, dev)
    _need("dt", dt, (B, H, T), f32, dev)
    _need("A", A, (H,), f32, dev)
    _may("D", D, (H,), f32, dev)
    _may("lengths", lengths, (B,), torch.int32, dev)
    return e2ttt_ssm_shape(B, H, G, T, d_k, d_v, _ACT[v.dtype])


def _bytes(n):
    """A workspace size; 0 stands for a shape the library refuses, and it says why."""
    if n == 0:
        _check(ERR_INVALID_ARG)
    return n


def ssm_scan_fwd(q, k, v, dt, A, D=None, S0=None, lengths=None, *, save_states=False, ws=None,
                 stream=None):
    """Selective state-space scan S_t = exp(dt_t A) S_{t-1} + dt_t v_t k_t^T,
    y_t = S_t q_t + D v_t: v [B, H, T, d_v], q and k [B, G, T, d_k] (bf16 or
    fp32; H / G heads share a group), dt [B, H, T], A and D [H], S0
    [B, H, d_v, d_k] fp32, lengths int32 [B] (a padded batch). Returns (y, S_end,
    saved), saved (what ssm_scan_bwd needs) None unless save_states."""
    _first("v", v, 4)
    shape = _ssm_check(q, k, v, dt, A, D, lengths)
    dev = v.device
    state = (shape.B, shape.H, shape.d_v, shape.d_k)
    _may("S0", S0, state, torch.float32, dev)
    with _on(dev, stream):
        need = _bytes(e2ttt_ssm_workspace_bytes(shape, 0))
        y = torch.empty_like(v)
        S_end = torch.empty(state, dtype=torch.float32, device=dev)
        saved = (torch.empty(e2ttt_ssm_saved_bytes(shape) // 4, dtype=torch.float32, device=dev)
                 if save_states else None)
        e2ttt_ssm_scan_fwd(shape, q, k, v, dt, A, D, S0, lengths, y, S_end, saved,
                           _scratch(ws, need, dev))
    return y, S_end, saved


def ssm_scan_bwd(q, k, v, dt, A, saved, dy, D=None, dS_end=None, lengths=None, *, ws=None,
                 stream=None):
    """Gradients of ssm_scan_fwd for <dy, y> + <dS_end, S_end>: a dict dq, dk, dv,
    ddt, dA, dD (None without D), dS0. `saved` is the forward's; lengths must be
    the forward's too."""
    _first("v", v, 4)
    shape = _ssm_check(q, k, v, dt, A, D, lengths)
    dev, f32 = v.device, torch.float32
    state = (shape.B, shape.H, shape.d_v, shape.d_k)
    _need("dy", dy, v.shape, v.dtype, dev)
    _may("dS_end", dS_end, state, f32, dev)
    with _on(dev, stream):
        need = _bytes(e2ttt_ssm_workspace_bytes(shape, 1))
        _need("saved", saved, (e2ttt_ssm_saved_bytes(shape) // 4,), f32, dev)
        g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                 ddt=torch.empty_like(dt), dA=torch.empty_like(A),
                 dD=None if D is None else torch.empty_like(D),
                 dS0=torch.empty(state, dtype=f32, device=dev))
        e2ttt_ssm_scan_bwd(shape, q, k, v, dt, A, D, lengths, saved, dy, dS_end, g["dq"], g["dk"],
                           g["dv"], g["ddt"], g["dA"], g["dD"], g["dS0"], _scratch(ws, need, dev))
    return g


def ssm_step(q, k, v, dt, S, A, D=None, *, out=None, stream=None):
    """One token per row: q, k [B, G, d_k], v [B, H, d_v], dt [B, H], S
    [B, H, d_v, d_k] fp32 updated in place. Returns y [B, H, d_v] (`out` where
    given)."""
    _first("v", v, 3)
    B, H, d_v = v.shape
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _refuse("q must be [B, G, d_k]")
    G, d_k = q.shape[1:]
    dev, f32 = v.device, torch.float32
    _need("v", v, v.shape, v.dtype, dev)
    _need("q", q, (B, G, d_k), v.dtype, dev)
    _need("k", k, (B, G, d_k), v.dtype, dev)
    _need("dt", dt, (B, H), f32, dev)
    _need("A", A, (H,), f32, dev)
    _may("D", D, (H,), f32, dev)
    _need("S", S, (B, H, d_v, d_k), f32, dev)
    _may("out", out, v.shape, v.dtype, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v)
        e2ttt_ssm_step(e2ttt_ssm_shape(B, H, G, 1, d_k, d_v, _ACT[v.dtype]), q, k, v, dt, A, D, S, out)
    return out


# ---------------------------------------------------------------- gradient norm
def _grad_lists(tensors, name):
    """Pointers, counts, types and device of contiguous CUDA tensors on one device."""
    T = torch.Tensor
    try:
        act = [_ACT[t.dtype] for t in tensors]
        devs = set(map(T.get_device, tensors))
        fine = len(devs) == 1 and -1 not in devs and all(map(T.is_contiguous, tensors))
    except (KeyError, AttributeError, TypeError):
        fine = False
    if not fine:
        _refuse(f"{name} must be contiguous bfloat16 or float32 tensors on one CUDA device")
    return list(map(T.data_ptr, tensors)), list(map(T.numel, tensors)), act, tensors[0].device


def grad_norm(grads, *, ws=None, stream=None):
    """The global 2-norm of a list of gradient tensors (bf16 or fp32, any mix), as
    a float32 tensor of no dimensions on their device."""
    grads = list(grads)
    if not grads:
        _refuse("grads must not be empty")
    g, n, act, dev = _grad_lists(grads, "grads")
    with _on(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        e2ttt_grad_norm(g, n, act, norm, _scratch(ws, e2ttt_grad_workspace_bytes(len(g)), dev))
    return norm


def clip_grad_norm(grads, max_norm, *, out=None, ws=None, stream=None):
    """Scales a list of gradient tensors by min(1, max_norm / (norm + 1e-6)), norm
    their global 2-norm, in place or into `out` (tensors of the same types and
    sizes). Returns the norm (float32, on the device, before clipping)."""
    grads = list(grads)
    if not grads:
        _refuse("grads must not be empty")
    g, n, act, dev = _grad_lists(grads, "grads")
    o = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            _refuse(f"out has {len(out)} tensors, grads has {len(grads)}")
        o, on, oact, odev = _grad_lists(out, "out")
        if on != n or oact != act or odev != dev:
            _refuse("out must have the types, sizes and device of grads")
    with _on(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        e2ttt_clip_grad_norm(g, o, n, act, max_norm, norm,
                             _scratch(ws, e2ttt_grad_workspace_bytes(len(g)), dev))
    return norm
