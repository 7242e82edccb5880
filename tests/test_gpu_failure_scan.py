"""Failure detection of the state-space scan's tensor-core kernels without a fault. The
test hook e2ttt_test_stall_next_scan makes one block, mostly one thread of it alone, take
a wait for run out: the block records that, waits for its own copies and products in
flight, frees its tensor memory and ends. The status word says so although the other
waits succeeded, and a normal call afterwards gives the results of one before, bit for bit.
(That a wait itself runs out is tested with the chunk scan, whose waits these are.)"""
import pytest

pytest.importorskip("torch")
import torch

from test_gpu_seq import scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available()
    import test_weight_layers_chunk_b200 as E
    yield E
    E.e2ttt_test_stall_next_scan(0)


# B, H, G, T, P, N: several items in each stream of a block (copies in flight for the
# next one), both tile widths, with and without vectors; and a single item
SIZES = [(16, 32, 1, 130, 64, 128), (40, 8, 1, 257, 40, 64), (40, 8, 1, 130, 33, 17), (1, 1, 1, 5, 64, 64)]
FORWARD, BACKWARD = {"states": 1, "scores": 2, "rows": 3, "outputs": 4}, {"adjoint": 1, "dots": 5, "pairs": 6, "results": 7}


@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_a_wait_runs_out(E, size):
    B, H, G, T, P, N = size
    x = {n: t.cuda() for n, t in scan_inputs("bf16", *size, True, True, True, seed=T).items()}
    shape = E.make_ssm_shape(B, H, G, T, N, P)
    ws = [torch.empty(E.e2ttt_ssm_workspace_bytes(shape, i), dtype=torch.uint8, device="cuda") for i in (0, 1)]
    stream = torch.cuda.current_stream().cuda_stream

    def forward():
        return E.ssm_scan_fwd(x["q"], x["k"], x["v"], x["dt"], x["A"], x["D"], x["S0"], save_states=True, ws=ws[0])

    def backward():
        return E.ssm_scan_bwd(x["q"], x["k"], x["v"], x["dt"], x["A"], saved, x["dy"], x["D"], x["dS_end"], ws=ws[1])

    y, S, saved = forward()
    g = backward()
    vectors = N % 8 == 0 and P % 8 == 0  # loads by the threads have no wait of their own
    for i, (call, waits) in enumerate(((forward, FORWARD), (backward, BACKWARD))):
        for name, number in waits.items():
            if name == "rows" and not vectors:
                continue
            E.e2ttt_test_stall_next_scan(number)
            call()
            st = E.e2ttt_workspace_status(ws[i], raw=True, stream=stream)
            assert st == E.ERR_TIMEOUT and "gave up" in E.e2ttt_last_error(), name
            again = call()  # the hook has disarmed itself, the status word is reset
            assert E.e2ttt_workspace_status(ws[i], raw=True, stream=stream) == E.OK, name
            if i == 0:
                assert torch.equal(again[0], y) and torch.equal(again[1], S) and torch.equal(again[2], saved), name
            else:
                assert all(torch.equal(again[n], t) for n, t in g.items()), name
