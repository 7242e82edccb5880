"""The fp64 oracle of the convolution and the scan: its gradients against
central differences of its own forward, and the forward against closed forms."""
import numpy as np
import pytest

from oracle import seq_oracle as O

H_STEP = 1e-5  # central differences of smooth functions of order one: error ~ h^2 + eps / h


def _differences(f, args, name, got, rng, n=12):
    x = args[name]
    for _ in range(min(n, x.size)):
        at = tuple(rng.integers(0, s) for s in x.shape)
        keep = x[at]
        x[at] = keep + H_STEP
        hi = f(**args)
        x[at] = keep - H_STEP
        lo = f(**args)
        x[at] = keep
        num = (hi - lo) / (2 * H_STEP)
        assert abs(num - got[at]) <= 1e-7 * max(1.0, abs(num)) + 1e-7, (name, at, num, got[at])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W,T,lengths", [(4, 9, None), (4, 2, [2, 1]), (3, 7, [0, 5]), (1, 3, None)])
def test_conv_gradients_against_differences(W, T, lengths, silu):
    rng = np.random.default_rng(W * 10 + T)
    B, H, d = 2, 2, 3
    a = dict(x=rng.normal(size=(B, H, T, d)), w=rng.normal(size=(H, d, W)), bias=rng.normal(size=(H, d)),
             state=rng.normal(size=(B, H, W - 1, d)))
    dy, de = rng.normal(size=(B, H, T, d)), rng.normal(size=(B, H, W - 1, d))

    def f(**k):
        y, end = O.conv_fwd(lengths=lengths, silu=silu, **k)
        return (y * dy).sum() + (end * de).sum()

    g = O.conv_bwd(dy=dy, dstate_end=de, lengths=lengths, silu=silu, **a)
    for n in ("x", "w", "bias", "state"):
        if a[n].size:
            _differences(f, a, n, g["d" + n], rng)


@pytest.mark.parametrize("G,lengths", [(1, None), (2, [5, 0]), (4, [3, 6])])
def test_scan_gradients_against_differences(G, lengths):
    rng = np.random.default_rng(G)
    B, H, T, P, N = 2, 4, 6, 3, 2
    a = dict(q=rng.normal(size=(B, G, T, N)), k=rng.normal(size=(B, G, T, N)), v=rng.normal(size=(B, H, T, P)),
             dt=rng.uniform(0.05, 0.5, size=(B, H, T)), A=-rng.uniform(0.5, 3, size=H), D=rng.normal(size=H),
             S0=rng.normal(size=(B, H, P, N)))
    dy, dS = rng.normal(size=(B, H, T, P)), rng.normal(size=(B, H, P, N))

    def f(**k):
        y, S = O.ssm_fwd(lengths=lengths, **k)
        return (y * dy).sum() + (S * dS).sum()

    g = O.ssm_bwd(dy=dy, dS_end=dS, lengths=lengths, **a)
    for n in a:
        _differences(f, a, n, g["d" + n], rng)


def test_scan_without_decay_is_a_running_sum():
    """A = 0: S_t is the sum of dt_s v_s k_s^T, so y_t = sum_{s<=t} dt_s (q_t.k_s) v_s."""
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 5, 3))
    v, dt = rng.normal(size=(1, 1, 5, 4)), rng.uniform(0, 1, size=(1, 1, 5))
    y, S = O.ssm_fwd(q, k, v, dt, np.zeros(1))
    M = np.tril(q[0, 0] @ k[0, 0].T) * dt[0, 0]
    np.testing.assert_allclose(y[0, 0], M @ v[0, 0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(S[0, 0], (v[0, 0] * dt[0, 0, :, None]).T @ k[0, 0], rtol=1e-12, atol=1e-13)


def test_scan_in_two_parts_is_one_scan():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 8, 3))
    v, dt, A = rng.normal(size=(1, 2, 8, 4)), rng.uniform(0, 1, size=(1, 2, 8)), np.array([-1.0, -2.0])
    y, S = O.ssm_fwd(q, k, v, dt, A)
    y1, S1 = O.ssm_fwd(q[:, :, :3], k[:, :, :3], v[:, :, :3], dt[:, :, :3], A)
    y2, S2 = O.ssm_fwd(q[:, :, 3:], k[:, :, 3:], v[:, :, 3:], dt[:, :, 3:], A, S0=S1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 2), y, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-13)


def test_rows_behind_a_length_are_not_read():
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(2, 2, 1, 5, 3))
    v, dt = rng.normal(size=(2, 1, 5, 4)), rng.uniform(0, 1, size=(2, 1, 5))
    for a in (q, k, v, dt):
        a[1, :, 2:] = np.nan
    y, S = O.ssm_fwd(q, k, v, dt, -np.ones(1), lengths=[5, 2])
    assert np.isfinite(y).all() and np.isfinite(S).all() and (y[1, :, 2:] == 0).all()


def test_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    n, out = O.clip_grads(g, 1.0)
    assert n == 5.0 and abs(O.grad_norm(out) - 1.0) < 1e-6
    assert O.clip_grads(g, 6.0)[1][0][0] == 3.0
