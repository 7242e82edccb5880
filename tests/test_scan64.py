"""The 64-bit scan in torch (scan64.py) against the numpy oracle."""
import numpy as np
import pytest

pytest.importorskip("torch")
import torch

from oracle import seq_oracle as O
from scan64 import scan64


@pytest.mark.parametrize("absolute", [False, True])
@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_against_the_oracle(lengths, absolute):
    r = np.random.default_rng(1)
    B, H, G, T, P, N = 3, 4, 2, 9, 5, 3
    x = dict(q=r.normal(size=(B, G, T, N)), k=r.normal(size=(B, G, T, N)), v=r.normal(size=(B, H, T, P)),
             dt=r.uniform(0, 1, size=(B, H, T)), A=-r.uniform(1, 3, size=H), D=r.normal(size=H),
             S0=r.normal(size=(B, H, P, N)), dy=r.normal(size=(B, H, T, P)), dS_end=r.normal(size=(B, H, P, N)))
    got = scan64({n: torch.from_numpy(a) for n, a in x.items()}, lengths, absolute)
    if absolute:
        x = {n: a if n == "A" else np.abs(a) for n, a in x.items()}
    y, S = O.ssm_fwd(*(x[n] for n in ("q", "k", "v", "dt", "A", "D", "S0")), lengths)
    want = O.ssm_bwd(*(x[n] for n in ("q", "k", "v", "dt", "A", "dy", "D", "S0", "dS_end")), lengths)
    # of B T sums of at most P N products, in 64 bits on both sides
    if lengths is not None:  # dD and y count the tokens that are there
        x["dy"] = O._present(x["dy"], O._lengths(lengths, B, T))
        want["dD"] = (x["dy"] * x["v"]).sum((0, 2, 3))
    for n, w in dict(want, y=y, S_end=S).items():
        assert np.allclose(got[n].numpy(), w, rtol=1e-12, atol=1e-12), n
