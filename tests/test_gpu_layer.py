"""The operators together, as a recurrent layer uses them: short convolutions in
front of q, k and v, the scan, their gradients, and the clipping of all of them; a
padded batch of prompts followed by single tokens; the convolution and clipping
around the chunk scan. Against the fp64 oracle run through the same chain.

Tolerance. Between the operators the GPU chain rounds to bf16 (2^-8 of each
value, half a step), which the oracle chain repeats on its own values; where the
two differ by an operator's error (2^-8 relative for a bf16 result with one
rounded operand), the next operator passes it on. A chain of n operators is held,
in the 2-norm, to (2 n) 2^-8: twice one step for each, since a sum of rounded
terms of either sign stays within the terms' own relative error in the 2-norm
and the products with fixed matrices keep relative errors of this order."""
import numpy as np
import pytest

pytest.importorskip("torch")
import torch

from oracle import seq_oracle as O

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    return E


def host(t):
    return t.detach().double().cpu().numpy()


def rel(got, want):
    return np.linalg.norm(host(got) - want) / np.linalg.norm(want)


def bf(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


def layer(seed, B, H, G, T, P, N, W=4):
    r = np.random.default_rng(seed)
    c = lambda *s: torch.from_numpy(r.normal(size=s)).bfloat16().cuda()  # noqa: E731
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).float().cuda()  # noqa: E731
    taps = lambda h, d: (f(r.normal(size=(h, d, W)) / W ** 0.5), f(0.1 * r.normal(size=(h, d))))  # noqa: E731
    x = dict(q=c(B, G, T, N), k=c(B, G, T, N), v=c(B, H, T, P))
    par = dict(q=taps(G, N), k=taps(G, N), v=taps(H, P), A=f(-r.uniform(1, 8, size=H)), D=f(r.normal(size=H)))
    dt = f(np.exp(r.uniform(np.log(1e-2), np.log(0.3), size=(B, H, T))))
    return x, par, dt, c(B, H, T, P)


@pytest.mark.parametrize("lengths", [None, [150, 37, 0]])
def test_training_step(E, lengths):
    B, H, G, T, P, N = 3, 4, 2, 150, 64, 64
    x, par, dt, dy = layer(1, B, H, G, T, P, N)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    conv = {n: E.short_conv_fwd(x[n], *par[n], lengths=lens)[0] for n in x}
    y, S, saved = E.ssm_scan_fwd(conv["q"], conv["k"], conv["v"], dt, par["A"], par["D"], lengths=lens, save_states=True)
    g = E.ssm_scan_bwd(conv["q"], conv["k"], conv["v"], dt, par["A"], saved, dy, par["D"], lengths=lens)
    back = {n: E.short_conv_bwd(x[n], par[n][0], g["d" + n], par[n][1], lengths=lens) for n in x}
    grads = [back[n][m] for n in x for m in ("dw", "dbias")] + [g["dA"], g["dD"], g["ddt"]]
    grads += [back[n]["dx"] for n in x]
    before = [host(t) for t in grads]
    norm = E.clip_grad_norm(grads, 1.0)

    hx = {n: host(t) for n, t in x.items()}
    hp = {n: tuple(host(t) for t in par[n]) for n in x}
    A, D, hdt, hdy = host(par["A"]), host(par["D"]), host(dt), host(dy)
    oc = {n: bf(O.conv_fwd(hx[n], *hp[n], lengths=lengths)[0]) for n in x}
    oy, oS = O.ssm_fwd(oc["q"], oc["k"], oc["v"], hdt, A, D, lengths=lengths)
    og = O.ssm_bwd(oc["q"], oc["k"], oc["v"], hdt, A, hdy, D, lengths=lengths)
    ob = {n: O.conv_bwd(hx[n], hp[n][0], bf(og["d" + n]), hp[n][1], lengths=lengths) for n in x}
    assert rel(y, oy) <= 4 * STEP and rel(S, oS) <= 4 * STEP
    want = [ob[n][m] for n in x for m in ("dw", "dbias")] + [og["dA"], og["dD"], og["ddt"]] + [ob[n]["dx"] for n in x]
    for b, w in zip(before, want):
        assert np.linalg.norm(b - w) <= 6 * STEP * np.linalg.norm(w)
    n, clipped = O.clip_grads(before, 1.0)
    assert abs(float(norm) - n) <= 1e-6 * n
    for t, w in zip(grads, clipped):
        assert np.linalg.norm(host(t) - w) <= STEP * np.linalg.norm(w) + 1e-12
    assert O.grad_norm([host(t) for t in grads]) <= 1.0 + STEP


def test_prompts_then_single_tokens(E):
    """A padded batch of prompts (one of them empty) and the tokens after them give
    what each row's whole sequence gives."""
    B, H, G, T, P, N, more = 3, 4, 1, 140, 64, 128, 5
    lengths = [140, 0, 61]
    x, par, dt, _ = layer(2, B, H, G, T + more, P, N)
    # row b: its prompt, then `more` tokens directly behind it
    ends = np.array(lengths)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    head = {n: t[:, :, :T].contiguous() for n, t in x.items()}
    hdt = dt[:, :, :T].contiguous()
    state, conv = {}, {}
    for n in x:
        conv[n], state[n] = E.short_conv_fwd(head[n], *par[n], lengths=lens, return_state=True)
    y, S, _ = E.ssm_scan_fwd(conv["q"], conv["k"], conv["v"], hdt, par["A"], par["D"], lengths=lens)
    rows = []
    for j in range(more):
        at = {n: torch.stack([x[n][b, :, e + j] for b, e in enumerate(ends)]).contiguous() for n in x}
        dtj = torch.stack([dt[b, :, e + j] for b, e in enumerate(ends)]).contiguous()
        c = {n: E.short_conv_step(at[n], state[n], *par[n]) for n in x}
        rows.append(E.ssm_step(c["q"], c["k"], c["v"], dtj, S, par["A"], par["D"]))
    rows = torch.stack(rows, 2)
    whole = (ends + more).tolist()
    oc = {n: bf(O.conv_fwd(host(x[n]), *(host(t) for t in par[n]), lengths=whole)[0]) for n in x}
    oy, oS = O.ssm_fwd(oc["q"], oc["k"], oc["v"], host(dt), host(par["A"]), host(par["D"]), lengths=whole)
    for b, e in enumerate(ends):
        if e:
            assert rel(y[b, :, :e], oy[b, :, :e]) <= 4 * STEP
        assert rel(rows[b], oy[b, :, e:e + more]) <= 4 * STEP
        assert rel(S[b], oS[b]) <= 4 * STEP


def test_two_calls_at_once(E):
    """The same calls on two streams at the same time, with workspaces of their own."""
    x, par, dt, dy = layer(3, 2, 4, 1, 600, 64, 128)
    def run():
        c = {n: E.short_conv_fwd(x[n], *par[n])[0] for n in x}
        y, S, saved = E.ssm_scan_fwd(c["q"], c["k"], c["v"], dt, par["A"], par["D"], save_states=True)
        g = E.ssm_scan_bwd(c["q"], c["k"], c["v"], dt, par["A"], saved, dy, par["D"])
        return [y, S] + [g[n] for n in sorted(g) if g[n] is not None]
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_around_the_chunk_scan(E):
    """Convolutions in front of the chunk scan's q, k and v (the same layouts), and
    the clipping of its gradients."""
    r = np.random.default_rng(4)
    B, H, T, d, dh = 1, 2, 256, 128, 128
    c = lambda *s: torch.from_numpy(0.1 * r.normal(size=s)).bfloat16().cuda()  # noqa: E731
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).float().cuda()  # noqa: E731
    x = {n: c(B, H, T, d) for n in "qkv"}
    w = {n: f(r.normal(size=(H, d, 4)) / 2) for n in "qkv"}
    gate = lambda lo, hi: f(r.uniform(lo, hi, size=(B, H, T)))  # noqa: E731
    lr, mom, decay = gate(0.001, 0.01), gate(0.8, 0.95), gate(0.95, 0.999)
    W0 = f(0.05 * r.normal(size=(B, H, 3 * d * dh)))
    y = {n: E.short_conv_fwd(x[n], w[n])[0] for n in x}
    out, W_end, _, saved = E.chunk_scan_fwd(y["q"], y["k"], y["v"], lr, mom, decay, W0, C=128, d_h=dh, save_states=True)
    g = E.chunk_scan_bwd(y["q"], y["k"], y["v"], lr, mom, decay, saved, torch.ones_like(out), C=128, d_h=dh)
    back = [E.short_conv_bwd(x[n], w[n], g["d" + n]) for n in x]
    grads = [b["dw"] for b in back] + [g[n] for n in ("dlr", "dmom", "ddecay", "dW0")]
    before = [host(t) for t in grads]
    n = E.clip_grad_norm(grads, 0.1)
    want, clipped = O.clip_grads(before, 0.1)
    assert abs(float(n) - want) <= 1e-6 * want and want > 0.1
    for t, c_ in zip(grads, clipped):
        assert np.allclose(host(t), c_, rtol=1e-6, atol=1e-12)
    # the convolution's gradient against its oracle, given the scan's
    ob = O.conv_bwd(host(x["v"]), host(w["v"]), host(g["dv"]))
    assert np.linalg.norm(before[2] - ob["dw"]) <= 1e-4 * np.linalg.norm(ob["dw"])
