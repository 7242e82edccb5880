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
import functools
from array import array

import torch

from . import BF16, ERR_INVALID_ARG, OK, E2TTTError, F32, _check, _lib, _P, _ptr, _stream


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
    "e2ttt_test_stall_next_scan": (None, [_I]),
    "e2ttt_grad_workspace_bytes": (_Z, [_I]),
    "e2ttt_grad_norm": (_I, [_P, _P, _P, _I, _P, _P, _Z, _P]),
    "e2ttt_clip_grad_norm": (_I, [_P, _P, _P, _P, _I, ctypes.c_float, _P, _P, _Z, _P]),
}.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

_ACT = {torch.bfloat16: BF16, torch.float32: F32}


# ---------------------------------------------------------------- C entry points
def _filled(kind, sizes):
    """A shape struct, whose fields are C ints: what does not fit one is refused (ctypes
    would keep the lower 32 bits)."""
    for (name, _), n in zip(kind._fields_, sizes):
        if not -2 ** 31 <= n < 2 ** 31:
            raise E2TTTError(ERR_INVALID_ARG, f"{name}={n} does not fit a shape")
    return kind(*sizes)


def make_conv_shape(B, H, T, d, W, act=BF16, silu=True) -> e2ttt_conv_shape:
    return _filled(e2ttt_conv_shape, (B, H, T, d, W, act, int(silu)))


def make_ssm_shape(B, H, G, T, d_k, d_v, act=BF16) -> e2ttt_ssm_shape:
    return _filled(e2ttt_ssm_shape, (B, H, G, T, d_k, d_v, act))


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


def e2ttt_test_stall_next_scan(wait: int) -> None:
    """Failure-detection test hook: wait number `wait` of the next tensor-core scan times out."""
    _lib.e2ttt_test_stall_next_scan(int(wait))


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


def _need(name, t, shape, dtype, dev):
    """t is a contiguous tensor of this shape and type on CUDA device number dev."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return
    except AttributeError:
        _refuse(f"{name} must be a tensor, got {type(t).__name__}")
    if t.shape != shape:
        _refuse(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        _refuse(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        _refuse(f"{name} must be on cuda:{dev}, got {t.device}")
    _refuse(f"{name} must be contiguous")


def _first(name, t, dims):
    """The tensor that fixes sizes, type and device; returns its device's number
    and its type's code."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        _refuse(f"{name} must be a tensor of {dims} dimensions")
    if not t.is_cuda:
        _refuse(f"{name} must be on a CUDA device, got {t.device}")
    act = _ACT.get(t.dtype)
    if act is None:
        _refuse(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")
    return t.get_device(), act


def _dims(name, t, dims, what):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        _refuse(f"{name} must be {what}")


@contextlib.contextmanager
def _guard(dev, stream):
    """Makes device number `dev` current, and `stream` where one is given."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            if isinstance(stream, int):
                # (0, the default stream's handle, would be a new stream to ExternalStream)
                stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            elif stream.device.index != dev:
                _refuse(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
            with torch.cuda.stream(stream):
                yield


def _elsewhere(dev, stream):
    """Whether the call has to change the current device or stream first."""
    return stream is not None or torch.cuda.current_device() != dev


# The current stream's handle, by the short way where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _p(t):
    return None if t is None else t.data_ptr()


def _run(fn, *args):
    st = fn(*args)
    if st != OK:
        _check(st)


def _scratch(ws, need, like):
    """The caller's workspace or a new one; (its pointer, its size, what keeps it)."""
    if ws is None:
        ws = like.new_empty(need, dtype=torch.uint8)
        return ws.data_ptr(), need, ws
    if not isinstance(ws, torch.Tensor) or ws.get_device() != like.get_device() or not ws.is_contiguous():
        _refuse(f"ws must be a contiguous tensor on {like.device}")
    return ws.data_ptr(), _nbytes(ws), ws


# Shapes and the sizes that follow from them, by value.
@functools.lru_cache(maxsize=1024)
def _conv_shape(*sizes):
    shape = _filled(e2ttt_conv_shape, sizes)
    return ctypes.byref(shape), e2ttt_short_conv_workspace_bytes(shape)


@functools.lru_cache(maxsize=1024)
def _ssm_shape(*sizes):
    shape = _filled(e2ttt_ssm_shape, sizes)
    return (ctypes.byref(shape), e2ttt_ssm_workspace_bytes(shape, 0), e2ttt_ssm_workspace_bytes(shape, 1),
            e2ttt_ssm_saved_bytes(shape))


def _known(sizes_of, *sizes):
    found = sizes_of(*sizes)
    if found[1] == 0:  # a shape the library refuses: asked again, it says why
        sizes_of.__wrapped__(*sizes)
        _check(ERR_INVALID_ARG)
    return found


# ---------------------------------------------------------------- short convolution
def _conv_check(x, w, bias, state, lengths, silu):
    dev, act = _first("x", x, 4)
    _dims("w", w, 3, "[H, d, W]")
    B, H, T, d = x.shape
    W = w.shape[2]
    f32 = torch.float32
    _need("w", w, (H, d, W), f32, dev)
    if bias is not None:
        _need("bias", bias, (H, d), f32, dev)
    if state is not None:
        _need("state", state, (B, H, W - 1, d), x.dtype, dev)
    if lengths is not None:
        _need("lengths", lengths, (B,), torch.int32, dev)
    shape, need = _known(_conv_shape, B, H, T, d, W, act, 1 if silu else 0)
    return dev, shape, need, (B, H, W - 1, d)


def short_conv_fwd(x, w, bias=None, state=None, lengths=None, *, silu=True, return_state=False,
                   stream=None):
    """Short causal depthwise convolution: x [B, H, T, d] (bf16 or fp32), w
    [H, d, W] and bias [H, d] fp32, state [B, H, W-1, d] (the inputs before the
    first token; None: zeros), lengths int32 [B] (a padded batch). Returns (y,
    state_end), state_end None unless return_state."""
    dev, shape, _, history = _conv_check(x, w, bias, state, lengths, silu)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return short_conv_fwd(x, w, bias, state, lengths, silu=silu, return_state=return_state)
    y = torch.empty_like(x)
    end = x.new_empty(history) if return_state else None
    _run(_lib.e2ttt_short_conv_fwd, shape, x.data_ptr(), w.data_ptr(), _p(bias), _p(state), _p(lengths),
         y.data_ptr(), _p(end), _raw_stream(dev))
    return y, end


def short_conv_bwd(x, w, dy, bias=None, state=None, dstate_end=None, lengths=None, *, silu=True,
                   ws=None, stream=None):
    """Gradients of short_conv_fwd for <dy, y> + <dstate_end, state_end>: a dict
    dx, dw, dbias (None without bias), dstate (None without state)."""
    dev, shape, need, history = _conv_check(x, w, bias, state, lengths, silu)
    _need("dy", dy, x.shape, x.dtype, dev)
    if dstate_end is not None:
        _need("dstate_end", dstate_end, history, x.dtype, dev)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return short_conv_bwd(x, w, dy, bias, state, dstate_end, lengths, silu=silu, ws=ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dbias = None if bias is None else torch.empty_like(bias)
    dstate = None if state is None else torch.empty_like(state)
    wp, wn, _keep = _scratch(ws, need, x)
    _run(_lib.e2ttt_short_conv_bwd, shape, x.data_ptr(), w.data_ptr(), _p(bias), _p(state), _p(lengths),
         dy.data_ptr(), _p(dstate_end), dx.data_ptr(), dw.data_ptr(), _p(dbias), _p(dstate), wp, wn,
         _raw_stream(dev))
    return dict(dx=dx, dw=dw, dbias=dbias, dstate=dstate)


def short_conv_step(x, state, w, bias=None, *, silu=True, out=None, stream=None):
    """One token per row: x [B, H, d], state [B, H, W-1, d] updated in place.
    Returns y [B, H, d] (`out` where given)."""
    dev, act = _first("x", x, 3)
    _dims("w", w, 3, "[H, d, W]")
    B, H, d = x.shape
    W = w.shape[2]
    _need("w", w, (H, d, W), torch.float32, dev)
    if bias is not None:
        _need("bias", bias, (H, d), torch.float32, dev)
    _need("state", state, (B, H, W - 1, d), x.dtype, dev)
    if out is not None:
        _need("out", out, x.shape, x.dtype, dev)
    shape, _ = _known(_conv_shape, B, H, 1, d, W, act, 1 if silu else 0)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return short_conv_step(x, state, w, bias, silu=silu, out=out)
    if out is None:
        out = torch.empty_like(x)
    _run(_lib.e2ttt_short_conv_step, shape, x.data_ptr(), w.data_ptr(), _p(bias), state.data_ptr(),
         out.data_ptr(), _raw_stream(dev))
    return out


# ---------------------------------------------------------------- state-space scan
def _ssm_check(q, k, v, dt, A, D, lengths):
    dev, act = _first("v", v, 4)
    _dims("q", q, 4, "[B, G, T, d_k]")
    B, H, T, d_v = v.shape
    G, d_k = q.shape[1], q.shape[3]
    f32, qk = torch.float32, (B, G, T, d_k)
    _need("q", q, qk, v.dtype, dev)
    _need("k", k, qk, v.dtype, dev)
    _need("dt", dt, (B, H, T), f32, dev)
    _need("A", A, (H,), f32, dev)
    if D is not None:
        _need("D", D, (H,), f32, dev)
    if lengths is not None:
        _need("lengths", lengths, (B,), torch.int32, dev)
    return dev, _known(_ssm_shape, B, H, G, T, d_k, d_v, act), (B, H, d_v, d_k)


def ssm_scan_fwd(q, k, v, dt, A, D=None, S0=None, lengths=None, *, save_states=False, ws=None,
                 stream=None):
    """Selective state-space scan S_t = exp(dt_t A) S_{t-1} + dt_t v_t k_t^T,
    y_t = S_t q_t + D v_t: v [B, H, T, d_v], q and k [B, G, T, d_k] (bf16 or
    fp32; H / G heads share a group), dt [B, H, T] >= 0, A and D [H], S0
    [B, H, d_v, d_k] fp32, lengths int32 [B] (a padded batch). Returns (y, S_end,
    saved), saved (what ssm_scan_bwd needs) None unless save_states."""
    dev, (shape, need, _, n_saved), state = _ssm_check(q, k, v, dt, A, D, lengths)
    if S0 is not None:
        _need("S0", S0, state, torch.float32, dev)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return ssm_scan_fwd(q, k, v, dt, A, D, S0, lengths, save_states=save_states, ws=ws)
    y = torch.empty_like(v)
    S_end = dt.new_empty(state)
    saved = dt.new_empty(n_saved // 4) if save_states else None
    wp, wn, _keep = _scratch(ws, need, v)
    _run(_lib.e2ttt_ssm_scan_fwd, shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(),
         A.data_ptr(), _p(D), _p(S0), _p(lengths), y.data_ptr(), S_end.data_ptr(), _p(saved), wp, wn,
         _raw_stream(dev))
    return y, S_end, saved


def ssm_scan_bwd(q, k, v, dt, A, saved, dy, D=None, dS_end=None, lengths=None, *, ws=None,
                 stream=None):
    """Gradients of ssm_scan_fwd for <dy, y> + <dS_end, S_end>: a dict dq, dk, dv,
    ddt, dA, dD (None without D), dS0. `saved` is the forward's; lengths must be
    the forward's too."""
    dev, (shape, _, need, n_saved), state = _ssm_check(q, k, v, dt, A, D, lengths)
    _need("dy", dy, v.shape, v.dtype, dev)
    _need("saved", saved, (n_saved // 4,), torch.float32, dev)
    if dS_end is not None:
        _need("dS_end", dS_end, state, torch.float32, dev)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return ssm_scan_bwd(q, k, v, dt, A, saved, dy, D, dS_end, lengths, ws=ws)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ddt, dA = torch.empty_like(dt), torch.empty_like(A)
    dD = None if D is None else torch.empty_like(D)
    dS0 = dt.new_empty(state)
    wp, wn, _keep = _scratch(ws, need, v)
    _run(_lib.e2ttt_ssm_scan_bwd, shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(),
         A.data_ptr(), _p(D), _p(lengths), saved.data_ptr(), dy.data_ptr(), _p(dS_end), dq.data_ptr(),
         dk.data_ptr(), dv.data_ptr(), ddt.data_ptr(), dA.data_ptr(), _p(dD), dS0.data_ptr(), wp, wn,
         _raw_stream(dev))
    return dict(dq=dq, dk=dk, dv=dv, ddt=ddt, dA=dA, dD=dD, dS0=dS0)


def ssm_step(q, k, v, dt, S, A, D=None, *, out=None, stream=None):
    """One token per row: q, k [B, G, d_k], v [B, H, d_v], dt [B, H], S
    [B, H, d_v, d_k] fp32 updated in place. Returns y [B, H, d_v] (`out` where
    given)."""
    dev, act = _first("v", v, 3)
    _dims("q", q, 3, "[B, G, d_k]")
    B, H, d_v = v.shape
    G, d_k = q.shape[1], q.shape[2]
    f32, qk = torch.float32, (B, G, d_k)
    _need("q", q, qk, v.dtype, dev)
    _need("k", k, qk, v.dtype, dev)
    _need("dt", dt, (B, H), f32, dev)
    _need("A", A, (H,), f32, dev)
    if D is not None:
        _need("D", D, (H,), f32, dev)
    _need("S", S, (B, H, d_v, d_k), f32, dev)
    if out is not None:
        _need("out", out, v.shape, v.dtype, dev)
    shape = _known(_ssm_shape, B, H, G, 1, d_k, d_v, act)[0]
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return ssm_step(q, k, v, dt, S, A, D, out=out)
    if out is None:
        out = torch.empty_like(v)
    _run(_lib.e2ttt_ssm_step, shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(),
         A.data_ptr(), _p(D), S.data_ptr(), out.data_ptr(), _raw_stream(dev))
    return out


# ---------------------------------------------------------------- gradient norm
def _grad_lists(tensors, name):
    """Pointers, counts and types (host arrays) and device number of contiguous
    CUDA tensors on one device."""
    T = torch.Tensor
    try:
        act = array("i", [_ACT[t.dtype] for t in tensors])
        devs = set(map(T.get_device, tensors))
        fine = len(devs) == 1 and -1 not in devs and all(map(T.is_contiguous, tensors))
    except (KeyError, AttributeError, TypeError):
        fine = False
    if not fine:
        _refuse(f"{name} must be contiguous bfloat16 or float32 tensors on one CUDA device")
    return array("Q", map(T.data_ptr, tensors)), array("Q", map(T.numel, tensors)), act, devs.pop()


def _at(a):
    return None if a is None else a.buffer_info()[0]


def grad_norm(grads, *, ws=None, stream=None):
    """The global 2-norm of a list of gradient tensors (bf16 or fp32, any mix), as
    a float32 tensor of no dimensions on their device."""
    grads = list(grads)
    if not grads:
        _refuse("grads must not be empty")
    g, n, act, dev = _grad_lists(grads, "grads")
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return grad_norm(grads, ws=ws)
    norm = grads[0].new_empty((), dtype=torch.float32)
    wp, wn, _keep = _scratch(ws, e2ttt_grad_workspace_bytes(len(g)), norm)
    _run(_lib.e2ttt_grad_norm, _at(g), _at(n), _at(act), len(g), norm.data_ptr(), wp, wn, _raw_stream(dev))
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
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return clip_grad_norm(grads, max_norm, out=out, ws=ws)
    norm = grads[0].new_empty((), dtype=torch.float32)
    wp, wn, _keep = _scratch(ws, e2ttt_grad_workspace_bytes(len(g)), norm)
    _run(_lib.e2ttt_clip_grad_norm, _at(g), _at(o), _at(n), _at(act), len(g), max_norm, norm.data_ptr(),
         wp, wn, _raw_stream(dev))
    return norm
