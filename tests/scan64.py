"""The state-space scan and its gradients token by token in 64 bits with torch, on
whatever device the inputs are on: the definitions of oracle/seq_oracle.py for
sizes where numpy on the host takes too long."""
import torch


def _present(x, lens):
    """x [B, heads, T, ..] with the tokens from each batch row's length on set to zero."""
    x = x.double()
    if lens is None:
        return x
    there = torch.arange(x.shape[2], device=x.device) < torch.as_tensor(lens, device=x.device)[:, None]
    return torch.where(there[:, None].reshape(x.shape[0], 1, -1, *[1] * (x.dim() - 3)), x, 0.0)


def scan64(x, lens=None, absolute=False):
    """dict y, S_end, dq, dk, dv, de, dl, ddt, dA, dD, dS0 of <dy, y> + <dS_end, S_end>;
    de and dl are the parts of ddt = de + A dl. `absolute`: of the inputs' absolute
    values (but for A), which bounds the sums of the absolute terms."""
    x = {n: None if t is None else t.double() for n, t in x.items()}
    if absolute:
        x = {n: t if t is None or n == "A" else t.abs() for n, t in x.items()}
    B, H, T, P = x["v"].shape
    G, N = x["q"].shape[1], x["q"].shape[3]
    per = H // G
    q, k = (_present(x[n], lens).repeat_interleave(per, 1) for n in ("q", "k"))
    v, dt, dy = (_present(x[n], lens) for n in ("v", "dt", "dy"))
    A = x["A"]
    dec = torch.exp(dt * A[:, None])
    S = v.new_zeros(B, H, P, N) if x["S0"] is None else x["S0"]
    path, y = [S], torch.zeros_like(v)
    for t in range(T):
        S = S * dec[:, :, t, None, None] + (dt[:, :, t, None] * v[:, :, t])[..., None] * k[:, :, t, None]
        y[:, :, t] = (S @ q[:, :, t, :, None])[..., 0]
        path.append(S)
    if x["D"] is not None:
        y = y + x["D"][:, None, None] * v
    X = v.new_zeros(B, H, P, N) if x["dS_end"] is None else x["dS_end"]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    de, dl = torch.zeros_like(dt), torch.zeros_like(dt)
    for t in reversed(range(T)):
        X = X + dy[:, :, t, :, None] * q[:, :, t, None]
        dq[:, :, t] = (dy[:, :, t, None] @ path[t + 1])[:, :, 0]
        u = (X @ k[:, :, t, :, None])[..., 0]
        dv[:, :, t] = dt[:, :, t, None] * u
        dk[:, :, t] = ((dt[:, :, t, None] * v[:, :, t])[:, :, None] @ X)[:, :, 0]
        de[:, :, t] = (u * v[:, :, t]).sum(-1)
        X = X * dec[:, :, t, None, None]
        dl[:, :, t] = (X * path[t]).sum((-1, -2))
    if x["D"] is not None:
        dv = dv + x["D"][:, None, None] * dy
    group = lambda a: _present(a.view(B, G, per, T, N).sum(2), lens)  # noqa: E731
    de, dl = _present(de, lens), _present(dl, lens)
    return dict(y=_present(y, lens), S_end=S, dq=group(dq), dk=group(dk), dv=_present(dv, lens), de=de, dl=dl,
                ddt=de + A[:, None] * dl, dA=(dt * dl).sum((0, 2)), dD=(dy * v).sum((0, 2, 3)), dS0=X)
