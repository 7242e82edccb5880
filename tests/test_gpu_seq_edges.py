"""Calls at the edges of the operators around a recurrent layer: raw stream handles,
NaN and infinities in valid places, roundings that lean one way, states carried over
thousands of single tokens."""
import numpy as np
import pytest

pytest.importorskip("torch")
import torch

from test_gpu_seq import scan_inputs

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    return E


def test_stream_handle_of_the_default_stream(E, monkeypatch):
    """stream=0, the default stream's raw handle, is that stream, whichever is current."""
    from test_weight_layers_chunk_b200 import sequence
    x = torch.randn(1, 1, 4, 8, device="cuda")
    w = torch.randn(1, 8, 2, device="cuda")
    used = []
    run = sequence._run
    monkeypatch.setattr(sequence, "_run", lambda fn, *args: (used.append(args[-1]), run(fn, *args)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            for stream in (0, torch.cuda.default_stream()):
                E.short_conv_fwd(x, w, stream=stream)
                E.grad_norm([x, w], stream=stream)
            E.short_conv_fwd(x, w, stream=side)
            E.short_conv_fwd(x, w, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert used == ([0] * 4 + [side.cuda_stream] * 2) * 2


SPREAD = [  # act, B, H, G, T, P, N: one chunk and several, several heads a block, both tile widths, and fp32
    ("bf16", 1, 3, 3, 1, 64, 64), ("bf16", 74, 6, 2, 40, 64, 64), ("bf16", 74, 6, 2, 140, 40, 128),
    ("bf16", 1, 3, 1, 300, 24, 200), ("f32", 2, 3, 1, 140, 24, 20),
]


def with_nan(E, case, what):
    """What the scan and its gradients give without and with a NaN in head 0's decay,
    step, state or input, the token that it is in, and the inputs."""
    act, B, H, G, T, P, N = case
    x = scan_inputs(act, B, H, G, T, P, N, True, True, True, seed=T + N)
    g = {n: t.cuda() for n, t in x.items()}

    def run():
        y, S, saved = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"], save_states=True)
        return dict(E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved, g["dy"], g["D"], g["dS_end"]),
                    y=y, S_end=S)

    clean, at = run(), T // 2
    nan = float("nan")
    if what == "A":
        g["A"][0], at = nan, 0
    elif what == "dt":
        g["dt"][:, 0, at] = nan
    elif what == "S0":
        g["S0"][:, 0], at = nan, 0
    else:
        g["v"][:, 0, at] = nan
    return clean, run(), at, g


@pytest.mark.parametrize("what", ["A", "dt", "S0", "v"])
@pytest.mark.parametrize("case", SPREAD, ids=[f"{c[0]}-{'x'.join(map(str, c[1:]))}" for c in SPREAD])
def test_nan_stays_with_its_head(E, case, what):
    """The other heads' results are those without it, bit for bit."""
    clean, got, _, _ = with_nan(E, case, what)
    for n in ("y", "S_end", "dv", "ddt", "dS0"):
        assert torch.equal(got[n][:, 1:], clean[n][:, 1:]), n
    for n in ("dA", "dD"):
        assert torch.equal(got[n][1:], clean[n][1:]), n


@pytest.mark.parametrize("what", ["A", "dt", "S0", "v"])
@pytest.mark.parametrize("case", SPREAD, ids=[f"{c[0]}-{'x'.join(map(str, c[1:]))}" for c in SPREAD])
def test_nan_reaches_what_follows(E, case, what):
    """Its own head's state is lost from there on; it does not count as no state at all."""
    _, got, at, g = with_nan(E, case, what)
    assert got["S_end"][:, 0].isnan().all()
    assert got["y"][:, 0, at:].isnan().all()
    if what in ("A", "dt"):  # the gradients pass every decay on the way to the row's start
        assert got["dS0"][:, 0].isnan().all() and got["ddt"][:, 0, :at + 1].isnan().all() and got["dA"][0].isnan()
    if what == "A":  # and a single token does the same
        state = g["S0"].clone()
        state[state.isnan()] = 0.0
        E.ssm_step(*(g[n][:, :, 0].contiguous() for n in ("q", "k", "v", "dt")), state, g["A"])
        assert state[:, 0].isnan().all() and not state[:, 1:].isnan().any()


@pytest.mark.parametrize("N", [64, 128])
def test_state_gradient_is_rounded_not_cut_off(E, N):
    """dv = dt X k with X of one value just below 1 + 2^-7, a bf16 value: X rounded to
    bf16 is that value, and dv = 2^-3 64 (1 + 2^-7) is one too; cut off, X would be 1."""
    B, H, T, P = 1, 2, 128, 64
    X = 1 + 2.0 ** -7 - 2.0 ** -20
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, v = z(B, 1, T, N), z(B, 1, T, N), z(B, H, T, P)
    k[..., :64] = 1
    dt, A = torch.full((B, H, T), 0.125, device="cuda"), torch.zeros(H, device="cuda")
    dS = torch.full((B, H, P, N), X, device="cuda")
    dS[:, 1] = -X
    _, _, saved = E.ssm_scan_fwd(q, k, v, dt, A, save_states=True)
    dv = E.ssm_scan_bwd(q, k, v, dt, A, saved, torch.zeros_like(v), dS_end=dS)["dv"]
    want = torch.tensor([8 * X, -8 * X], device="cuda", dtype=torch.float64).bfloat16()
    assert torch.equal(dv, want[None, :, None, None].expand_as(dv))


@pytest.mark.parametrize("N", [64, 128])
def test_state_gradient_does_not_lean(E, N):
    """dv = dt X k of random X. Each X has one rounding to bf16, of root mean square
    0.43 2^-8 and either sign; projected on dv, B H P N >= 2^15 independent ones (a
    token's share doubled, as k k^T is not quite diagonal) leave 2 0.43 2^-8 2^-7.5 =
    1.9e-5; held to six times that. Cut off, they would leave 2.8e-3."""
    B, H, T, P = 2, 4, 128, 64
    x = scan_inputs("bf16", B, H, 1, T, P, N, False, False, True, seed=N)
    g = {n: None if t is None else t.cuda() for n, t in x.items()}
    g["dy"].zero_()
    g["A"].zero_()
    _, _, saved = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], save_states=True)
    dv = E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved, g["dy"], dS_end=g["dS_end"])["dv"].double()
    want = g["dt"].double()[..., None] * (g["k"].double() @ g["dS_end"].double().transpose(-1, -2))
    assert abs(float(((dv - want) * want).sum() / want.square().sum())) <= 6 * 2 * 0.43 * UBF * 2.0 ** -7.5


@pytest.mark.parametrize("N", [16, 18, 128])
@pytest.mark.parametrize("log", [1e-3, 1e-4])
def test_long_generation_keeps_the_decay(E, log, N):
    """n single tokens that add nothing: S = S0 e^{n dt A}. Each of the n states is
    rounded once, by 2^-24 and either sign: sqrt(n) 2^-24, held to six times that. A
    decay that is itself off by half a unit, 2^-25, would be off n times the same way."""
    B, H, P, n = 1, 32, 4, 4000
    r = torch.Generator().manual_seed(N)
    A = -(0.5 + torch.rand(H, generator=r)).cuda()
    dt = torch.full((B, H), log, device="cuda")
    S0 = torch.randn(B, H, P, N, generator=r).cuda()
    S, v, k = S0.clone(), torch.zeros(B, H, P, device="cuda"), torch.ones(B, 1, N, device="cuda")
    for _ in range(n):
        E.ssm_step(k, k, v, dt, S, A)
    want = S0.double() * torch.exp(n * dt.double() * A.double())[..., None, None]
    off = ((S.double() - want) / want).abs()
    assert float(off.max()) <= 6 * n ** 0.5 * U32, float(off.max())


def test_steps_of_an_infinite_state(E):
    """An infinite state stays infinite under a decay, and under none (dt = 0)."""
    for dt in (0.0, 0.1, 2.0):
        S = torch.full((1, 1, 2, 8), float("inf"), device="cuda")
        S[:, :, 1] = 1.0
        one = torch.ones(1, 1, 8, device="cuda")
        E.ssm_step(one, one, torch.ones(1, 1, 2, device="cuda"), torch.full((1, 1), dt, device="cuda"), S,
                   torch.tensor([-1.0], device="cuda"))
        assert S[0, 0, 0].isinf().all() and S[0, 0, 1].isfinite().all()


def test_status_of_workspaces_without_waits(E):
    """The convolution's gradients and the gradient norm reset the status word too,
    whatever the workspace held: nothing of theirs can have given up."""
    x, w = torch.randn(2, 3, 50, 12, device="cuda"), torch.randn(3, 12, 4, device="cuda")
    grads, empty = [torch.randn(5000, device="cuda"), torch.randn(9, device="cuda")], [torch.empty(0, device="cuda")]
    out = [torch.empty_like(t) for t in grads]
    conv, norm = E.e2ttt_short_conv_workspace_bytes(E.make_conv_shape(2, 3, 50, 12, 4, E.F32)), E.e2ttt_grad_workspace_bytes(2)
    for need, call in ((conv, lambda ws: E.short_conv_bwd(x, w, x, ws=ws)["dw"]),
                       (norm, lambda ws: E.grad_norm(grads, ws=ws)),
                       (norm, lambda ws: E.grad_norm(empty, ws=ws)),
                       (norm, lambda ws: E.clip_grad_norm(grads, 1.0, out=out, ws=ws)),
                       (norm, lambda ws: E.clip_grad_norm(empty, 1.0, ws=ws)),
                       (norm, lambda ws: E.clip_grad_norm(grads * 300, 1.0, out=[t.clone() for t in grads * 300], ws=ws))):
        if need == norm:
            need = max(need, E.e2ttt_grad_workspace_bytes(600))
        ws = [torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda") for fill in (0xff, 0)]
        got = [call(t[:need]) for t in ws]
        assert all(E.e2ttt_workspace_status(t, raw=True, stream=torch.cuda.current_stream().cuda_stream) == E.OK for t in ws)
        assert torch.equal(*got)
        assert (ws[0][need:] == 0xff).all()  # nothing behind it
