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
