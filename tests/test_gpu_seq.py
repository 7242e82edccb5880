"""The short convolution, the state-space scan and their single-token forms on
the GPU against the fp64 oracle.

Tolerances. Every output of the scan but ddt is a sum of products of the inputs
and of positive decays, so a run of the oracle on the inputs' absolute values
bounds the sum of the absolute terms, and each value may be off by that bound
times the terms' relative errors:
  gamma32 = (N + P + 2 Q + 8 chunks + heads of a group + 64) 2^-24: one rounding
    for each addition of the dot products and of the states' passage, and a
    few for each exponential (2^-22 by the instruction's documented error);
  bf16 inputs: operands that are not inputs (the decayed scores, the states) may
    be rounded to bf16 once where the result is bf16, 2^-8 (half a step), and to
    a pair of bf16 values (2^-16) where it is fp32; plus the result's own
    rounding, 2^-8 of its value.
ddt_t = A dl_t + de_t, where dl_t is a part of the sum over all (source, reader)
pairs of the row, and is formed from sums of up to all of them.
"""
import numpy as np
import pytest

pytest.importorskip("torch")
import torch

from oracle import seq_oracle as O

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    return E


ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rounded(x, act):
    return torch.from_numpy(np.ascontiguousarray(x)).to(ACT[act])


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, want, tol):
    got = host(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(off)), float(np.max(off / np.maximum(tol, 1e-300))),
                           np.argwhere(bad)[:3].tolist())


# ------------------------------------------------------------------ convolution
CONV = [  # act, B, H, T, d, W, bias, silu, state, lengths
    ("bf16", 1, 1, 1, 8, 4, True, True, True, None),
    ("bf16", 2, 3, 1, 64, 4, True, True, False, [0, 1]),
    ("f32", 2, 2, 2, 4, 4, False, True, True, [2, 0]),
    ("bf16", 2, 2, 33, 72, 3, True, False, True, [33, 7]),
    ("f32", 3, 2, 50, 33, 2, True, True, True, [0, -3, 99]),
    ("bf16", 1, 2, 257, 33, 4, True, True, True, [200]),
    ("f32", 1, 3, 300, 256, 4, True, True, False, None),
    ("bf16", 2, 1, 129, 128, 8, True, True, True, [128, 3]),
    ("f32", 2, 2, 17, 20, 1, True, True, False, [16, 4]),
    ("bf16", 1, 2, 40, 2056, 4, False, True, True, None),
    ("f32", 1, 1, 21, 300, 5, True, False, True, [19]),
    ("bf16", 1, 2, 64, 16, 6, True, True, True, None),
    ("f32", 1, 2, 19, 12, 7, True, True, True, [18]),
]


def conv_inputs(act, B, H, T, d, W, bias, state, lengths, seed):
    r = np.random.default_rng(seed)
    x = dict(x=rounded(r.normal(size=(B, H, T, d)), act), w=torch.from_numpy(r.normal(size=(H, d, W))).float(),
             bias=torch.from_numpy(r.normal(size=(H, d))).float() if bias else None,
             state=rounded(r.normal(size=(B, H, W - 1, d)), act) if state else None,
             dy=rounded(r.normal(size=(B, H, T, d)), act), dend=rounded(r.normal(size=(B, H, W - 1, d)), act))
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return x, lens


def conv_tol(x, lengths, silu, act, W, T, B):
    """The absolute sums behind each output, times their roundings. The logistic
    function and its derivative add a few units on values of at most about z."""
    a = {n: None if t is None else np.abs(host(t)) for n, t in x.items()}
    zabs, _ = O.conv_fwd(a["x"], a["w"], a["bias"], a["state"], lengths, silu=False)
    u = U32
    step = UBF if act == "bf16" else U32
    gz = (W + 2 + (40 if silu else 0)) * u  # ex2 and rcp: 2 and 1 units of 2^-23, the argument's own error |z| 2^-24
    y = gz * zabs * (1 + zabs if silu else 1)
    # dz = dy f(z), |f| <= 1.1, |f'| <= 0.5: relative (40 + |z| error) units
    dzt = a["dy"] * 1.1 * (gz * (1 + zabs) if silu else u)
    n = B * T
    g = O.conv_bwd(a["x"], a["w"], a["dy"] * 1.1, a["bias"], a["state"], a["dend"], lengths, silu=False)
    e = O.conv_bwd(a["x"], a["w"], dzt, a["bias"], a["state"], None, lengths, silu=False)
    grow = (W + 4) * u
    # sums over tokens: at most 64 in a row in one thread's register per block of a
    # few hundred; bounded here by one unit for each of the n terms
    return step, y, {k: e[k] + (grow if k in ("dx", "dstate") else (n + 4) * u) * g[k] for k in g}


@pytest.mark.parametrize("case", CONV, ids=[f"{c[0]}-{'x'.join(map(str, c[1:6]))}" for c in CONV])
def test_conv(E, case):
    act, B, H, T, d, W, bias, silu, state, lengths = case
    x, lens = conv_inputs(act, B, H, T, d, W, bias, state, lengths, seed=T * 100 + d)
    step, ytol, gtol = conv_tol(x, lengths, silu, act, W, T, B)
    h = {n: host(t) for n, t in x.items()}
    want, wend = O.conv_fwd(h["x"], h["w"], h["bias"], h["state"], lengths, silu)
    wg = O.conv_bwd(h["x"], h["w"], h["dy"], h["bias"], h["state"], h["dend"], lengths, silu)
    g = {n: None if t is None else t.cuda() for n, t in x.items()}
    if lengths is not None:  # what is behind a row's length may be anything
        for b, n in enumerate(np.clip(lengths, 0, T)):
            g["x"][b, :, n:] = float("nan")
            g["dy"][b, :, n:] = float("inf")
    lens = None if lens is None else lens.cuda()
    y, end = E.short_conv_fwd(g["x"], g["w"], g["bias"], g["state"], lens, silu=silu, return_state=True)
    got = E.short_conv_bwd(g["x"], g["w"], g["dy"], g["bias"], g["state"], g["dend"], lens, silu=silu)
    again = E.short_conv_bwd(g["x"], g["w"], g["dy"], g["bias"], g["state"], g["dend"], lens, silu=silu)
    close("y", y, want, ytol + step * np.abs(want) + 1e-30)
    close("state_end", end, wend, np.zeros_like(wend))
    for n in ("dx", "dw", "dbias", "dstate"):
        if got[n] is None:
            continue
        s = step if n in ("dx", "dstate") else U32
        close(n, got[n], wg[n], gtol[n] + s * np.abs(wg[n]) + 1e-30)
        assert torch.equal(got[n], again[n]), n  # the sums' order is fixed


def test_conv_saturated(E):
    """silu far out: 0 for large negative z, z for large positive, gradients 0 and 1."""
    x = torch.tensor([-1e4, -200.0, -90.0, 0.0, 90.0, 1e4, 3e38, -3e38], device="cuda").view(1, 1, 8, 1)
    w = torch.ones(1, 1, 1, device="cuda")
    y, _ = E.short_conv_fwd(x, w)
    want = torch.where(x > 0, x, torch.zeros_like(x))
    assert torch.allclose(y, want, rtol=1e-6, atol=1e-36)
    g = E.short_conv_bwd(x, w, torch.ones_like(x))
    assert torch.allclose(g["dx"].flatten(), torch.tensor([0, 0, 0, 0.5, 1, 1, 1, 0], device="cuda"), atol=1e-6)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("d,W", [(64, 4), (33, 3), (16, 1)])
def test_conv_steps_continue_a_prompt(E, act, d, W):
    """A prompt of 5 tokens and 4 single tokens give the rows of one pass, bit for bit
    (the same sums in the same order)."""
    x, _ = conv_inputs(act, 2, 3, 9, d, W, True, False, None, seed=d)
    g = {n: None if t is None else t.cuda() for n, t in x.items()}
    whole, wend = E.short_conv_fwd(g["x"], g["w"], g["bias"], return_state=True)
    y, state = E.short_conv_fwd(g["x"][:, :, :5].contiguous(), g["w"], g["bias"], return_state=True)
    assert torch.equal(y, whole[:, :, :5])
    for t in range(5, 9):
        assert torch.equal(E.short_conv_step(g["x"][:, :, t].contiguous(), state, g["w"], g["bias"]), whole[:, :, t])
    assert torch.equal(state, wend)


def test_conv_unaligned(E):
    """Views that start off a 16-byte boundary take the single-channel form, with the same sums."""
    x, _ = conv_inputs("bf16", 1, 2, 20, 16, 4, True, True, None, seed=3)
    g = {n: t.cuda() for n, t in x.items()}
    off = torch.empty(x["x"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(x["x"].shape)
    off.copy_(g["x"])
    assert off.data_ptr() % 16
    a, _ = E.short_conv_fwd(g["x"], g["w"], g["bias"], g["state"])
    b, _ = E.short_conv_fwd(off, g["w"], g["bias"], g["state"])
    assert torch.equal(a, b)
    ga = E.short_conv_bwd(g["x"], g["w"], g["dy"], g["bias"], g["state"])
    gb = E.short_conv_bwd(off, g["w"], g["dy"], g["bias"], g["state"])
    assert torch.equal(ga["dx"], gb["dx"])


# ------------------------------------------------------------------ scan
SCAN = [  # act, B, H, G, T, P (d_v), N (d_k), D, S0, dS_end, lengths
    ("f32", 1, 1, 1, 1, 1, 1, True, False, True, None),
    ("bf16", 1, 2, 1, 1, 64, 128, True, True, True, None),
    ("f32", 2, 4, 2, 70, 24, 20, True, True, True, [70, 0]),
    ("bf16", 3, 4, 1, 130, 64, 64, True, True, True, [1, 64, 129]),
    ("bf16", 1, 2, 2, 200, 64, 128, False, False, False, None),
    ("bf16", 2, 3, 3, 65, 128, 128, True, True, True, [65, -4]),
    ("bf16", 1, 2, 1, 129, 48, 40, True, False, True, None),
    ("bf16", 1, 2, 1, 100, 33, 17, True, True, True, [99]),
    ("f32", 1, 2, 1, 63, 100, 200, True, True, False, [1000]),
    ("bf16", 1, 2, 1, 70, 200, 256, True, True, True, None),
    ("bf16", 1, 4, 4, 64, 96, 16, False, True, True, None),
    ("f32", 2, 2, 1, 128, 64, 64, True, False, True, [128, 65]),
    ("bf16", 1, 16, 1, 300, 32, 128, True, False, True, None),
    ("bf16", 2, 8, 2, 513, 64, 128, True, True, False, [513, 300]),
]


def scan_inputs(act, B, H, G, T, P, N, D, S0, dS, seed, fast=False):
    r = np.random.default_rng(seed)
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).float()  # noqa: E731
    top = 3.0 if fast else 0.1
    return dict(q=rounded(r.normal(size=(B, G, T, N)), act), k=rounded(r.normal(size=(B, G, T, N)), act),
                v=rounded(r.normal(size=(B, H, T, P)), act),
                dt=f(np.exp(r.uniform(np.log(1e-3), np.log(top), size=(B, H, T)))),
                A=f(-r.uniform(1, 16, size=H)), D=f(r.normal(size=H)) if D else None,
                S0=f(r.normal(size=(B, H, P, N))) if S0 else None,
                dy=rounded(r.normal(size=(B, H, T, P)), act),
                dS_end=f(r.normal(size=(B, H, P, N))) if dS else None)


def scan_check(act, x, lengths, y, S_end, g=None):
    h = {n: host(t) for n, t in x.items()}
    a = {n: None if t is None else np.abs(t) for n, t in h.items()}
    a["A"] = h["A"]
    B, H, T, P = h["v"].shape
    G, N = h["q"].shape[1], h["q"].shape[3]
    f = ("q", "k", "v", "dt", "A", "D", "S0")
    g32 = (N + P + 128 + 8 * (T // 32 + 1) + H // G + 64) * U32
    lo, hi = (g32 + UBF, g32 + 2 * UBF ** 2) if act == "bf16" else (g32, g32)
    step = UBF if act == "bf16" else U32
    wy, wS = O.ssm_fwd(*(h[n] for n in f), lengths)
    ay, aS = O.ssm_fwd(*(a[n] for n in f), lengths)
    close("y", y, wy, lo * ay + step * np.abs(wy) + 1e-30)
    close("S_end", S_end, wS, hi * aS + U32 * np.abs(wS) + 1e-30)
    if g is None:
        return
    w = O.ssm_bwd(*(h[n] for n in ("q", "k", "v", "dt", "A", "dy", "D", "S0", "dS_end")), lengths)
    m = O.ssm_bwd(*(a[n] for n in ("q", "k", "v", "dt", "A", "dy", "D", "S0", "dS_end")), lengths)
    for n in ("dq", "dk", "dv"):
        close(n, g[n], w[n], lo * m[n] + step * np.abs(w[n]) + 1e-30)
    close("dS0", g["dS0"], w["dS0"], hi * m["dS0"] + 1e-30)
    # all (source, reader) pairs of a row; tokens behind its length add none
    pairs = np.abs(O._present(a["dy"], O._lengths(lengths, B, T)) *
                   O.ssm_fwd(*(a[n] for n in ("q", "k", "v", "dt", "A")), None, a["S0"], lengths)[0]).sum((2, 3))
    if a["dS_end"] is not None:
        pairs = pairs + (a["dS_end"] * aS).sum((2, 3))
    dt = O._present(a["dt"], O._lengths(lengths, B, T))
    close("ddt", g["ddt"], w["ddt"], hi * (np.abs(h["A"])[:, None] * pairs[..., None] + m["de"]) + 1e-30)
    close("dA", g["dA"], w["dA"], hi * (dt.sum(2) * pairs).sum(0) + 1e-30)
    if h["D"] is not None:
        close("dD", g["dD"], w["dD"], hi * m["dD"] + 1e-30)


def to_gpu(x, lengths, T):
    g = {n: None if t is None else t.cuda() for n, t in x.items()}
    if lengths is not None:
        for b, n in enumerate(np.clip(lengths, 0, T)):
            g["q"][b, :, n:] = float("nan")
            g["k"][b, :, n:] = float("inf")
            g["v"][b, :, n:] = float("nan")
            g["dt"][b, :, n:] = float("nan")
            g["dy"][b, :, n:] = float("-inf")
    return g, None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def run_scan(E, g, lens, grads=True):
    y, S, saved = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"], lens, save_states=grads)
    return y, S, E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved, g["dy"], g["D"], g["dS_end"],
                                lens) if grads else None


@pytest.mark.parametrize("case", SCAN, ids=[f"{c[0]}-{'x'.join(map(str, c[1:7]))}" for c in SCAN])
def test_scan(E, case):
    act, B, H, G, T, P, N, D, S0, dS, lengths = case
    x = scan_inputs(act, B, H, G, T, P, N, D, S0, dS, seed=T * 1000 + N)
    g, lens = to_gpu(x, lengths, T)
    y, S, grads = run_scan(E, g, lens)
    scan_check(act, x, lengths, y, S, grads)
    y2, S2, again = run_scan(E, g, lens)
    y3, S3, _ = run_scan(E, g, lens, grads=False)  # without saved states: the same results
    assert torch.equal(y, y2) and torch.equal(S, S2) and torch.equal(y, y3) and torch.equal(S, S3)
    for n, t in grads.items():
        assert t is None or torch.equal(t, again[n]), n


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_scan_strong_decay(E, act):
    """Logarithms that sum to thousands within a chunk: decays between neighbours of
    every size, none of them lost to the size of the sums."""
    x = scan_inputs(act, 1, 4, 1, 150, 64, 64, True, True, True, seed=7, fast=True)
    g, _ = to_gpu(x, None, 150)
    y, S, grads = run_scan(E, g, None)
    scan_check(act, x, None, y, S, grads)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_scan_no_decay_and_growth(E, act):
    """A = 0 and a small positive A."""
    x = scan_inputs(act, 1, 2, 1, 140, 64, 64, True, True, True, seed=8)
    x["A"] = torch.tensor([0.0, 0.5])
    g, _ = to_gpu(x, None, 140)
    y, S, grads = run_scan(E, g, None)
    scan_check(act, x, None, y, S, grads)


@pytest.mark.parametrize("act,T,P,N", [("f32", 500, 64, 64), ("f32", 100, 40, 200), ("bf16", 500, 64, 128),
                                       ("bf16", 77, 48, 40), ("bf16", 200, 33, 17)])
def test_scan_skip_gradient_of_one_head(E, act, T, P, N):
    """dD = sum dy v of one row, whose terms cancel: products and sums are fp64 (fp32
    over at most 16 exact products of bf16, 16 roundings), then dD is rounded once."""
    x = scan_inputs(act, 1, 1, 1, T, P, N, True, False, False, seed=T + P)
    x["dy"][:, :, 1::2] = -x["dy"][:, :, :-1:2]
    x["v"][:, :, 1::2] = x["v"][:, :, :-1:2].clone()  # pairs cancel; what is left
    x["dy"][0, 0, 3, 5] += 0.5                               # is one element's change
    g, _ = to_gpu(x, None, T)
    terms = host(x["dy"]) * host(x["v"])
    bound = T * P * 2.0 ** -53 + (16 * U32 if act == "bf16" else 0.0)
    got = run_scan(E, g, None)[2]["dD"]
    close("dD", got, terms.sum()[None], bound * np.abs(terms).sum() + U32 * np.abs(terms.sum()) + 1e-30)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_scan_zero_steps(E, act):
    """dt = 0: the token leaves the state as it is, and its gradients are those of that."""
    x = scan_inputs(act, 1, 2, 1, 80, 64, 64, True, True, True, seed=9)
    x["dt"][:, :, 10:70] = 0.0
    g, _ = to_gpu(x, None, 80)
    y, S, grads = run_scan(E, g, None)
    scan_check(act, x, None, y, S, grads)


def test_scan_finite_differences(E):
    """Gradients against differences of the fp32 forward itself, in double sums:
    step h = 2^-6 on values of order one; truncation h^2 f'''/6 and rounding
    2^-24 / h relative to the objective's absolute sum are both below 1e-3 of it."""
    x = scan_inputs("f32", 1, 2, 1, 70, 16, 16, True, True, True, seed=11)
    g, _ = to_gpu(x, None, 70)
    _, _, grads = run_scan(E, g, None)

    def objective():
        y, S, _ = run_scan(E, g, None, grads=False)
        return float((y.double() * g["dy"].double()).sum() + (S.double() * g["dS_end"].double()).sum())

    r = np.random.default_rng(0)
    for n, step in (("q", 2.0 ** -6), ("k", 2.0 ** -6), ("v", 2.0 ** -6), ("S0", 2.0 ** -6), ("D", 2.0 ** -6),
                    ("A", 2.0 ** -8), ("dt", 2.0 ** -12)):
        flat = g[n].view(-1)
        way = torch.from_numpy(r.choice([-1.0, 1.0], size=flat.numel())).float().cuda()
        keep = flat.clone()
        flat.copy_(keep + step * way)
        hi = objective()
        flat.copy_(keep - step * way)
        lo = objective()
        flat.copy_(keep)
        num, dot = (hi - lo) / (2 * step), float((grads["d" + n].view(-1).double() * way.double()).sum())
        scale = float(grads["d" + n].double().norm())
        assert abs(num - dot) <= 0.02 * scale, (n, num, dot, scale)


@pytest.mark.parametrize("act,H,G,P,N", [("bf16", 4, 2, 64, 128), ("f32", 2, 1, 33, 20), ("bf16", 2, 2, 128, 64),
                                         ("bf16", 2, 1, 24, 256)])
def test_steps_continue_a_prompt(E, act, H, G, P, N):
    """A prompt, then single tokens from its end state, against the oracle over all of it."""
    B, T, n = 2, 90, 70
    x = scan_inputs(act, B, H, G, T, P, N, True, True, False, seed=N)
    g, _ = to_gpu(x, None, T)
    y, S, _ = E.ssm_scan_fwd(*(g[m][:, :, :n].contiguous() for m in ("q", "k", "v", "dt")), g["A"], g["D"], g["S0"])
    rows = [y]
    for t in range(n, T):
        rows.append(E.ssm_step(*(g[m][:, :, t].contiguous() for m in ("q", "k", "v", "dt")), S, g["A"],
                               g["D"])[:, :, None])
    scan_check(act, x, None, torch.cat(rows, 2), S)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prompt_of_one_token_is_a_step(E, act):
    x = scan_inputs(act, 3, 4, 2, 1, 64, 128, True, True, False, seed=5)
    g, _ = to_gpu(x, None, 1)
    y, S, _ = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"])
    state = g["S0"].clone()
    ys = E.ssm_step(*(g[m][:, :, 0].contiguous() for m in ("q", "k", "v", "dt")), state, g["A"], g["D"])
    scan_check(act, x, None, y, S)
    scan_check(act, x, None, ys[:, :, None], state)


def test_scan_padding_does_not_matter(E):
    """A padded row equals the same row alone, bit for bit (chunks start at the row's start)."""
    x = scan_inputs("bf16", 2, 4, 1, 200, 64, 64, True, True, False, seed=13)
    g, lens = to_gpu(x, [200, 77], 200)
    y, S, _ = run_scan(E, g, lens, grads=False)
    cut = {n: None if t is None else t[1:, :, :77].contiguous() if n in ("q", "k", "v", "dt") else t for n, t in g.items()}
    y1, S1, _ = E.ssm_scan_fwd(cut["q"], cut["k"], cut["v"], cut["dt"], g["A"], g["D"], g["S0"][1:].contiguous())
    assert torch.equal(y[1:, :, :77], y1) and torch.equal(S[1:], S1)
    assert not y[1, :, 77:].any()


def test_scan_unaligned(E):
    x = scan_inputs("bf16", 1, 2, 1, 70, 64, 64, True, True, True, seed=14)
    g, _ = to_gpu(x, None, 70)
    for n in ("q", "k", "v", "dy"):
        t = torch.empty(g[n].numel() + 1, dtype=g[n].dtype, device="cuda")[1:].view(g[n].shape)
        g[n] = t.copy_(g[n])
    y, S, grads = run_scan(E, g, None)
    scan_check("bf16", x, None, y, S, grads)


def test_scan_graph_and_streams(E):
    """Captured and replayed on new values, and run on a stream of its own."""
    x = scan_inputs("bf16", 1, 4, 1, 300, 64, 128, True, True, True, seed=15)
    g, _ = to_gpu(x, None, 300)
    want = run_scan(E, g, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_scan(E, g, None)
    g["v"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[0], want[0])
    g["v"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n, t in want[2].items():
        assert torch.equal(t, got[2][n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, S, saved = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"], save_states=True, stream=side)
    grads = E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved, g["dy"], g["D"], g["dS_end"],
                           stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(S, want[1]) and torch.equal(grads["dk"], want[2]["dk"])
    torch.cuda.synchronize()


@pytest.mark.parametrize("act,N", [("bf16", 64), ("f32", 64), ("bf16", 200)])
def test_scan_workspace_and_status(E, act, N):
    """A caller's workspace, whatever it holds; its status word says that no wait gave up."""
    x = scan_inputs(act, 1, 2, 1, 150, 64, N, True, True, True, seed=16)
    g, _ = to_gpu(x, None, 150)
    want = run_scan(E, g, None)
    shape = E.make_ssm_shape(1, 2, 1, 150, N, 64, E.BF16 if act == "bf16" else E.F32)
    for fill in (0xff, 0x7f):
        ws = [torch.full((E.e2ttt_ssm_workspace_bytes(shape, i),), fill, dtype=torch.uint8, device="cuda") for i in (0, 1)]
        y, S, saved = E.ssm_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"], save_states=True, ws=ws[0])
        assert E.e2ttt_workspace_status(ws[0], raw=True, stream=torch.cuda.current_stream().cuda_stream) == E.OK
        grads = E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved, g["dy"], g["D"], g["dS_end"], ws=ws[1])
        assert E.e2ttt_workspace_status(ws[1], raw=True, stream=torch.cuda.current_stream().cuda_stream) == E.OK
        assert torch.equal(y, want[0]) and torch.equal(S, want[1])
        for n, t in grads.items():
            assert torch.equal(t, want[2][n]), n


def test_scan_many_state_tiles_and_long_rows(E):
    """Sixteen tiles of state rows, and more chunks than one batch of the carry."""
    for act, B, H, G, T, P, N in (("bf16", 1, 2, 1, 130, 1024, 16), ("f32", 1, 1, 1, 70, 520, 8), ("bf16", 1, 1, 1, 2300, 16, 16),
                                  ("f32", 1, 1, 1, 1200, 8, 8)):
        x = scan_inputs(act, B, H, G, T, P, N, True, True, True, seed=T)
        g, _ = to_gpu(x, None, T)
        scan_check(act, x, None, *run_scan(E, g, None))


# ------------------------------------------------------------------ refusals that need a device
def test_conveniences_refuse(E):
    x = scan_inputs("bf16", 1, 4, 2, 8, 16, 16, True, True, True, seed=1)
    g, _ = to_gpu(x, None, 8)
    good = [g["q"], g["k"], g["v"], g["dt"], g["A"], g["D"], g["S0"]]
    E.ssm_scan_fwd(*good)
    bad = {0: g["q"].float(), 1: g["k"][:, :1], 2: g["v"].transpose(2, 3), 3: g["dt"].double(), 4: g["A"].cpu(),
           5: g["D"][:2], 6: g["S0"].bfloat16()}
    for i, t in bad.items():
        with pytest.raises(E.E2TTTError) as err:
            E.ssm_scan_fwd(*[t if j == i else a for j, a in enumerate(good)])
        assert err.value.status == E.ERR_INVALID_ARG
    with pytest.raises(E.E2TTTError):  # 4 heads are not a multiple of 3 groups
        E.ssm_scan_fwd(g["q"].repeat(1, 2, 1, 1)[:, :3].contiguous(), g["k"].repeat(1, 2, 1, 1)[:, :3].contiguous(),
                       *good[2:])
    with pytest.raises(E.E2TTTError):
        E.ssm_scan_fwd(*good, lengths=torch.tensor([8], device="cuda"))  # int64
    with pytest.raises(E.E2TTTError):
        E.ssm_scan_fwd(*good, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    _, _, saved = E.ssm_scan_fwd(*good, save_states=True)
    with pytest.raises(E.E2TTTError):
        E.ssm_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], saved[:-1], g["dy"], g["D"])
    with pytest.raises(E.E2TTTError):
        E.ssm_step(g["q"][:, :, 0], g["k"][:, :, 0], g["v"][:, :, 0].contiguous(), g["dt"][:, :, 0].contiguous(), g["S0"], g["A"])
    c, _ = conv_inputs("bf16", 1, 2, 8, 16, 4, True, True, None, seed=1)
    c = {n: t.cuda() for n, t in c.items()}
    E.short_conv_fwd(c["x"], c["w"], c["bias"], c["state"])
    for a in ((c["x"], c["w"].bfloat16()), (c["x"], c["w"][:1]), (c["x"].half(), c["w"]),
              (c["x"], c["w"], c["bias"], c["state"][:, :, :2]), (c["x"].transpose(1, 2), c["w"])):
        with pytest.raises(E.E2TTTError):
            E.short_conv_fwd(*a)
    with pytest.raises(E.E2TTTError):  # a state that is the input
        E.short_conv_step(c["x"][:, :, 0].contiguous(), c["state"], c["w"], out=c["state"][:, :, 0])
