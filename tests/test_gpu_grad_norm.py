"""Gradient norm and clipping on the GPU against fp64. The norm's squares are
summed in fp32 over at most 8 values and in fp64 beyond: relative error of the
sum at most 8 * 2^-24, half of it in the root, and one rounding of the result;
the clipped values add the factor's rounding (4 units) and their own."""
import numpy as np
import pytest

pytest.importorskip("torch")
import torch

from oracle import seq_oracle as O

pytestmark = pytest.mark.gpu
NORM_TOL = 6 * 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    return E


def tensors(sizes, seed, kinds=(torch.bfloat16, torch.float32), scale=0.02):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(kinds[i % len(kinds)]).cuda() for i, n in enumerate(sizes)]


def check(E, grads, max_norm, out=None):
    before = [g.double().cpu().numpy() for g in grads]
    n, want = O.clip_grads(before, max_norm)
    got = E.clip_grad_norm(grads, max_norm, out=out)
    assert got.dim() == 0 and abs(float(got) - n) <= NORM_TOL * n + 1e-45
    # the norm alone, of copies: a start off a 16-byte boundary only changes which values share a vector
    alone = float(E.grad_norm([torch.from_numpy(b).to(g.dtype).cuda() for b, g in zip(before, grads)]))
    assert abs(alone - float(got)) <= 2 * NORM_TOL * n
    for g, b, w, o in zip(grads, before, want, grads if out is None else out):
        r = o.double().cpu().numpy()
        assert np.all(np.abs(r - w) <= (STEP[g.dtype] + NORM_TOL + 4 * 2.0 ** -24) * np.abs(w) + 1e-44)
        if out is not None:
            assert np.array_equal(g.double().cpu().numpy(), b)


SIZES = [[1], [7], [0, 5, 0], [8192], [8193, 1, 3], [100_001, 8, 64, 31], list(range(1, 600)), [517] * 481 + [9000],
         [(1 << 20) + 3]]


@pytest.mark.parametrize("sizes", SIZES, ids=[f"{len(s)}x{max(s)}" for s in SIZES])
@pytest.mark.parametrize("max_norm", [1e-3, 0.0, 1e6])
def test_clip_in_place_and_out(E, sizes, max_norm):
    check(E, tensors(sizes, 1), max_norm)
    grads = tensors(sizes, 2)
    check(E, grads, max_norm, [torch.full_like(g, float("nan")) for g in grads])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_unaligned_views(E, kind):
    """Tensors cut from one buffer at every offset, and outputs at other offsets."""
    flat, other = tensors([4000], 3, (kind,))[0], torch.zeros(4100, dtype=kind, device="cuda")
    cuts = [1, 2, 3, 5, 70, 333, 1001, 900, 1000]
    at = np.concatenate([[3], 3 + np.cumsum(cuts)])
    grads = [flat[a:a + c] for a, c in zip(at, cuts)]
    out = [other[a + 5:a + 5 + c] for a, c in zip(at, cuts)]
    check(E, grads, 0.5, out)
    assert not other[:8].any() and not other[at[-1] + 5:].any()  # nothing beside the outputs
    keep = flat[:3].clone(), flat[at[-1]:].clone()
    check(E, grads, 0.5)
    assert torch.equal(flat[:3], keep[0]) and torch.equal(flat[at[-1]:], keep[1])


def test_within_the_norm_nothing_changes(E):
    grads = tensors([1000, 33], 4)
    keep = [g.clone() for g in grads]
    E.clip_grad_norm(grads, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))


def test_empty_tensors_only(E):
    grads = [torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=torch.bfloat16)]
    assert float(E.clip_grad_norm(grads, 1.0)) == 0.0 and float(E.grad_norm(grads)) == 0.0


def test_large_and_small_values(E):
    """Squares beyond fp32's range, and below it."""
    for scale in (1e30, 1e-30, 1e-42):
        g = [torch.tensor([3 * scale, 0.0, 4 * scale] * 5, device="cuda"), torch.zeros(9, device="cuda")]
        n = O.grad_norm([t.double().cpu().numpy() for t in g])
        # 1e-42 is a denormal of a few bits; the norm's own rounding is half a step of 2^-149
        assert abs(float(E.grad_norm(g)) - n) <= NORM_TOL * n + 2.0 ** -150
    assert float(E.grad_norm([torch.zeros(100, device="cuda")])) == 0.0


def test_nonfinite(E):
    for bad in (float("nan"), float("inf"), -float("inf")):
        grads = tensors([5000, 40], 5, (torch.float32,))
        grads[1][7] = bad
        n = E.clip_grad_norm(grads, 1.0)
        if np.isnan(bad):
            assert torch.isnan(n) and torch.isnan(grads[0]).all()
        else:
            assert torch.isinf(n) and not grads[0].any() and torch.isnan(grads[1][7])


def test_repeatable_and_captured(E):
    grads = tensors([300_000, 17, 8200], 6)
    out = [torch.empty_like(g) for g in grads]
    a = E.clip_grad_norm(grads, 0.1, out=out)
    assert torch.equal(a, E.clip_grad_norm(grads, 0.1, out=out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = E.clip_grad_norm(grads, 0.1, out=out)
    for g in grads:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert float(n) == 2 * float(a)  # doubling is exact in every step


def test_refusals(E):
    g = tensors([100, 50], 7)
    half = torch.zeros(4, dtype=torch.float16, device="cuda")
    for bad in ([], [half], [g[0].cpu()], [g[0].view(10, 10).t()], [g[0], g[0]], [g[0], g[0][10:]]):
        with pytest.raises(E.E2TTTError):
            E.clip_grad_norm(bad, 1.0)
    for out in ([g[0]], [g[1], g[0]], [torch.empty_like(g[0]), g[0][:50].clone()],
                [g[0], torch.empty(25, dtype=torch.float32, device="cuda")]):
        with pytest.raises(E.E2TTTError):
            E.clip_grad_norm(g, 1.0, out=out)
    for m in (-1.0, float("nan"), float("inf")):
        with pytest.raises(E.E2TTTError):
            E.clip_grad_norm(g, m)
    E.grad_norm([g[0], g[0]])  # reading a tensor twice is fine
