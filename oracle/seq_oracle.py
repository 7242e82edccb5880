"""fp64 oracle of the operators around a recurrent layer: the short causal
convolution, the selective state-space scan (token by token) and the gradient
norm. Written from the definitions, without the library's chunk form."""
from __future__ import annotations

import numpy as np


def _lengths(lengths, B, T):
    if lengths is None:
        return np.full(B, T, int)
    return np.clip(np.asarray(lengths, int), 0, T)


def _present(x, lens, axis=2):
    """x with the tokens behind each batch row's length set to zero (whatever they hold)."""
    x = np.array(x, np.float64)
    for b, n in enumerate(lens):
        x[b][(slice(None),) * (axis - 1) + (slice(n, None),)] = 0.0
    return x


# ------------------------------------------------------------------ convolution
def conv_fwd(x, w, bias=None, state=None, lengths=None, silu=True):
    """y, state_end. x [B,H,T,d], w [H,d,W]."""
    B, H, T, d = x.shape
    W = w.shape[2]
    lens = _lengths(lengths, B, T)
    seq = np.zeros((B, H, W - 1 + T, d))
    if state is not None:
        seq[:, :, :W - 1] = state
    seq[:, :, W - 1:] = _present(x, lens)
    z = np.zeros((B, H, T, d))
    for t in range(T):
        for j in range(W):
            z[:, :, t] += w[:, :, j] * seq[:, :, t + j]
    if bias is not None:
        z += bias[:, None]
    y = z / (1 + np.exp(-z)) if silu else z
    end = np.stack([seq[b, :, n:n + W - 1] for b, n in enumerate(lens)])
    return _present(y, lens), end


def conv_bwd(x, w, dy, bias=None, state=None, dstate_end=None, lengths=None, silu=True):
    """dict dx, dw, dbias, dstate of <dy, y> + <dstate_end, state_end>."""
    B, H, T, d = x.shape
    W = w.shape[2]
    lens = _lengths(lengths, B, T)
    seq = np.zeros((B, H, W - 1 + T, d))
    if state is not None:
        seq[:, :, :W - 1] = state
    seq[:, :, W - 1:] = _present(x, lens)
    dy = _present(dy, lens)
    dseq, dw, db = np.zeros_like(seq), np.zeros(w.shape), np.zeros((H, d))
    for t in range(T):
        z = sum(w[:, :, j] * seq[:, :, t + j] for j in range(W)) + (0 if bias is None else bias)
        s = 1 / (1 + np.exp(-z))
        dz = dy[:, :, t] * (s + z * s * (1 - s) if silu else 1.0)
        db += dz.sum(0)
        for j in range(W):
            dw[:, :, j] += (dz * seq[:, :, t + j]).sum(0)
            dseq[:, :, t + j] += w[:, :, j] * dz
    if dstate_end is not None:
        for b, n in enumerate(lens):
            dseq[b, :, n:n + W - 1] += dstate_end[b]
    return dict(dx=_present(dseq[:, :, W - 1:], lens), dw=dw, dbias=db, dstate=dseq[:, :, :W - 1])


# ------------------------------------------------------------------ scan
def ssm_fwd(q, k, v, dt, A, D=None, S0=None, lengths=None, keep=False):
    """y, S_end (and with keep the state before each token and after it)."""
    B, H, T, P = v.shape
    G, N = q.shape[1], q.shape[3]
    lens = _lengths(lengths, B, T)
    q, k = (np.repeat(_present(a, lens), H // G, axis=1) for a in (q, k))
    v, dt = _present(v, lens), _present(dt, lens)
    S = np.zeros((B, H, P, N)) if S0 is None else np.array(S0, np.float64)
    y, path = np.zeros((B, H, T, P)), [S]
    for t in range(T):
        S = S * np.exp(dt[:, :, t] * A)[..., None, None] \
            + (dt[:, :, t, None] * v[:, :, t])[..., None] * k[:, :, t, None]
        y[:, :, t] = np.einsum("bhpn,bhn->bhp", S, q[:, :, t])
        path.append(S)
    if D is not None:
        y += np.asarray(D)[:, None, None] * v
    y = _present(y, lens)
    return (y, S, path) if keep else (y, S)


def ssm_bwd(q, k, v, dt, A, dy, D=None, S0=None, dS_end=None, lengths=None):
    """dict dq, dk, dv, ddt, dA, dD, dS0 of <dy, y> + <dS_end, S_end>, and the two
    parts of ddt = de + A dl: the gradient of dt as a factor and of the log decay."""
    B, H, T, P = v.shape
    G, N = q.shape[1], q.shape[3]
    lens = _lengths(lengths, B, T)
    _, _, path = ssm_fwd(q, k, v, dt, A, D, S0, lengths, keep=True)
    q, k = (np.repeat(_present(a, lens), H // G, axis=1) for a in (q, k))
    v, dt, dy = _present(v, lens), _present(dt, lens), _present(dy, lens)
    X = np.zeros((B, H, P, N)) if dS_end is None else np.array(dS_end, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    de, dl = np.zeros_like(dt), np.zeros_like(dt)
    for t in reversed(range(T)):
        X = X + dy[:, :, t, :, None] * q[:, :, t, None]
        dq[:, :, t] = np.einsum("bhpn,bhp->bhn", path[t + 1], dy[:, :, t])
        u = np.einsum("bhpn,bhn->bhp", X, k[:, :, t])
        dv[:, :, t] = dt[:, :, t, None] * u
        dk[:, :, t] = np.einsum("bhpn,bhp->bhn", X, dt[:, :, t, None] * v[:, :, t])
        X = X * np.exp(dt[:, :, t] * A)[..., None, None]
        dl[:, :, t] = (X * path[t]).sum((-1, -2))
        de[:, :, t] = (u * v[:, :, t]).sum(-1)
    if D is not None:
        dv += np.asarray(D)[:, None, None] * dy
    group = lambda a: _present(a.reshape(B, G, H // G, T, N).sum(2), lens)  # noqa: E731
    return dict(dq=group(dq), dk=group(dk), dv=_present(dv, lens), de=_present(de, lens), dl=_present(dl, lens),
                ddt=_present(de + np.asarray(A)[:, None] * dl, lens), dA=(dt * dl).sum((0, 2)),
                dD=(dy * v).sum((0, 2, 3)), dS0=X)


# ------------------------------------------------------------------ gradient norm
def grad_norm(grads):
    return float(np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads)))


def clip_grads(grads, max_norm):
    n = grad_norm(grads)
    c = min(1.0, max_norm / (n + 1e-6))
    return n, [np.asarray(g, np.float64) * c for g in grads]
