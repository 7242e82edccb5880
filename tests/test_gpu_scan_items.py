"""The state-space scan where a block works through many items: several heads and
tiles of state rows one after the other, in both streams of the forward's kernels and
in the gradients', so that every buffer, barrier phase and running sum is used again.
How many items a block takes follows from the sizes; these take 2 to 12 of them. And
the gradients of dt and A, held head by head in the 2-norm.

Tolerances. Elementwise, as a sum's roundings bound it: (gamma + 2^-8) of the sum of
the absolute terms for bf16 results (one rounded operand a term) and half a step of
the result. In the 2-norm of a head, roundings add up like independent errors:
  bf16 results: 0.43 2^-8 (the root mean square of half a step, over a binade) for the
    result and as much for the operand of each term, so 0.6 2^-8; held to 2^-8.
  fp32 results: K = N + P + 256 + 16 chunks roundings of 2^-24 (the dot products, the
    running sums over a chunk's tokens, the states' passage and the exponentials),
    together sqrt(K) 2^-24; held to 4 times that, some 5e-6. The operands of these
    results enter with all 24 bits: one term of eight bits less would cost 2^-16.
ddt = de + A dl is held to that share of |A| ||dl|| + ||de||, dA to that of the sum of
dt |dl| over the head's tokens, since its parts cancel."""
import pytest

pytest.importorskip("torch")
import torch

from scan64 import scan64
from test_gpu_seq import ACT, scan_inputs

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    return E


# act, B, H, G, T, P, N, lengths given     items of a block: forward, gradients
CASES = [
    ("bf16", 16, 32, 1, 130, 64, 128, False),  # 8 in two streams, 8 (parts of dq and dk)
    ("bf16", 40, 8, 1, 257, 33, 17, True),     # 8, 8 (dq and dk directly), odd sizes
    ("bf16", 50, 6, 1, 130, 40, 40, True),     # 6, 6 directly, 64 columns
    ("bf16", 75, 5, 1, 129, 104, 72, True),    # 10 with two tiles of rows, 2
    ("bf16", 38, 12, 3, 130, 64, 128, True),   # 4, 4 directly, grouped
    ("bf16", 74, 6, 2, 7, 72, 128, True),      # 6, 6 directly, with two tiles of rows
    ("bf16", 74, 6, 2, 7, 70, 100, False),     # the same without vectors
    ("bf16", 5, 96, 1, 257, 16, 64, True),     # 12, 11
    ("bf16", 80, 7, 1, 129, 33, 128, False),   # 4 (a last block of 3), 1
    ("bf16", 1, 3, 1, 1500, 64, 128, False),   # few heads, many chunks
    ("f32", 3, 6, 2, 300, 48, 40, True),
    ("f32", 1, 2, 1, 200, 80, 136, False),
    ("bf16", 2, 4, 2, 300, 48, 200, True),     # beyond the tensor cores' columns
]


def norms(t):
    """2-norms by head (the second axis; the first of a vector of heads)."""
    t = t.double()
    return t.abs() if t.dim() == 1 else t.transpose(0, 1).reshape(t.shape[1], -1).norm(dim=1)


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{'x'.join(map(str, c[1:7]))}" for c in CASES])
def test_many_items(E, case):
    act, B, H, G, T, P, N, padded = case
    x = {n: None if t is None else t.cuda()
         for n, t in scan_inputs(act, B, H, G, T, P, N, True, True, True, seed=B * 100 + T).items()}
    lengths = None
    if padded:
        r = torch.Generator().manual_seed(B)
        lengths = torch.randint(0, T + 1, (B,), generator=r).tolist()
        lengths[0], lengths[-1] = T, 0
    want, most = scan64(x, lengths), scan64(x, lengths, absolute=True)
    lens = None
    if padded:
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lengths):
            for name in ("q", "k", "v", "dt", "dy"):
                x[name][b, :, n:] = float("nan")
    y, S, saved = E.ssm_scan_fwd(x["q"], x["k"], x["v"], x["dt"], x["A"], x["D"], x["S0"], lens, save_states=True)
    y2, S2, _ = E.ssm_scan_fwd(x["q"], x["k"], x["v"], x["dt"], x["A"], x["D"], x["S0"], lens)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    g = E.ssm_scan_bwd(x["q"], x["k"], x["v"], x["dt"], x["A"], saved, x["dy"], x["D"], x["dS_end"], lens)
    got = dict(g, y=y, S_end=S)
    chunks = -(-T // (128 if act == "bf16" else 32))
    gamma = (N + P + 256 + 16 * chunks + H // G) * U32
    share = 4 * (N + P + 256 + 16 * chunks + H // G) ** 0.5 * U32
    op, half = (UBF, UBF) if act == "bf16" else (0.0, U32)
    for n in ("y", "dq", "dk", "dv"):
        assert got[n].dtype == ACT[act]
        off = (got[n].double() - want[n]).abs()
        assert (off <= (gamma + op) * most[n] + half * want[n].abs()).all(), n
        part = UBF if act == "bf16" else share
        assert (norms(off) <= part * norms(want[n])).all(), (n, norms(off) / norms(want[n]))
    for n in ("S_end", "dS0"):
        off = (got[n].double() - want[n]).abs()
        assert (off <= gamma * most[n]).all(), n
        assert (norms(off) <= share * norms(want[n])).all(), (n, norms(off) / norms(want[n]))
    off = got["ddt"].double() - want["ddt"]
    scale = x["A"].double().abs() * norms(want["dl"]) + norms(want["de"])
    assert (norms(off) <= share * scale).all(), ("ddt", (norms(off) / scale).tolist())
    dt = torch.where(want["dl"] != 0, x["dt"].double(), 0.0)
    scale = (dt * want["dl"]).abs().sum((0, 2))
    off = (got["dA"].double() - want["dA"]).abs()
    assert (off <= share * scale).all(), ("dA", (off / scale).tolist())
    off = (got["dD"].double() - want["dD"]).abs()
    assert (off <= 16 * U32 * most["dD"]).all(), "dD"
