"""The C entry points of the convolution, the scan and the gradient norm without
a GPU: every bad argument is refused on the host, with a message, and nothing is
launched."""
import ctypes

import pytest

from test_abi import E  # noqa: F401  (the fixture that builds and loads the library)

FAKE, STEP = 1 << 40, 1 << 32  # never dereferenced


def _conv(E, shape, fn, **over):
    names = {"fwd": ("x", "w", "bias", "state", "lengths", "y", "state_end"),
             "bwd": ("x", "w", "bias", "state", "lengths", "dy", "dstate_end", "dx", "dw", "dbias", "dstate",
                     "workspace"),
             "step": ("x", "w", "bias", "state", "y")}[fn]
    args = {n: FAKE + i * STEP for i, n in enumerate(names)}
    if fn == "bwd":
        args["workspace_bytes"] = E.e2ttt_short_conv_workspace_bytes(shape)
    args.update(over)
    return getattr(E, "e2ttt_short_conv_" + fn)(shape, raw=True, stream=None, **args)


def _ssm(E, shape, fn, **over):
    names = {"fwd": ("q", "k", "v", "dt", "A", "D", "S0", "lengths", "y", "S_end", "saved_states", "workspace"),
             "bwd": ("q", "k", "v", "dt", "A", "D", "lengths", "saved_states", "dy", "dS_end", "dq", "dk", "dv", "ddt",
                     "dA", "dD", "dS0", "workspace"),
             "step": ("q", "k", "v", "dt", "A", "D", "S", "y")}[fn]
    args = {n: FAKE + i * STEP for i, n in enumerate(names)}
    if fn != "step":
        args["workspace_bytes"] = E.e2ttt_ssm_workspace_bytes(shape, int(fn == "bwd"))
    args.update(over)
    call = E.e2ttt_ssm_step if fn == "step" else getattr(E, "e2ttt_ssm_scan_" + fn)
    return call(shape, raw=True, stream=None, **args)


def _refused(E, st, *words):
    assert st == E.ERR_INVALID_ARG
    assert all(w in E.e2ttt_last_error() for w in words), E.e2ttt_last_error()


def test_conv_shapes(E):
    ok = dict(B=2, H=3, T=5, d=8, W=4)
    for over in (dict(B=0), dict(H=0), dict(T=0), dict(d=0), dict(W=0), dict(W=9), dict(act=2), dict(B=70000),
                 dict(T=(1 << 24) + 1), dict(H=60000, B=1, d=1 << 15), dict(d=(1 << 20) + 1)):
        s = E.make_conv_shape(**(ok | over))
        assert E.e2ttt_short_conv_workspace_bytes(s) == 0
        for fn in ("fwd", "bwd"):
            _refused(E, _conv(E, s, fn), "e2ttt_short_conv_" + fn)
    bad = E.make_conv_shape(**ok)
    bad.silu = 2
    _refused(E, _conv(E, bad, "fwd"), "silu")
    assert E.e2ttt_short_conv_workspace_bytes(E.make_conv_shape(**ok)) > 0


def test_conv_arguments(E):
    s = E.make_conv_shape(2, 3, 5, 8, 4)
    for n in ("x", "w", "y"):
        _refused(E, _conv(E, s, "fwd", **{n: None}), "NULL")
    for n in ("x", "w", "dy", "dx", "dw", "workspace"):
        _refused(E, _conv(E, s, "bwd", **{n: None}), "NULL")
    _refused(E, _conv(E, s, "fwd", y=FAKE + 2), "y overlaps input x")
    _refused(E, _conv(E, s, "fwd", state_end=FAKE + 3 * STEP), "state_end overlaps input state")
    _refused(E, _conv(E, s, "fwd", x=FAKE + 1), "aligned")
    _refused(E, _conv(E, s, "fwd", w=FAKE + STEP + 2), "aligned")
    _refused(E, _conv(E, s, "bwd", dx=FAKE + 5 * STEP), "dx overlaps input dy")
    _refused(E, _conv(E, s, "bwd", workspace=FAKE + 7 * STEP), "workspace")
    _refused(E, _conv(E, s, "bwd", workspace_bytes=8), "too small")
    _refused(E, _conv(E, s, "bwd", workspace=FAKE + 11 * STEP + 64), "256-byte")
    one = E.make_conv_shape(2, 3, 1, 8, 4)
    _refused(E, _conv(E, s, "step"), "T must be 1")
    for n in ("x", "w", "state", "y"):
        _refused(E, _conv(E, one, "step", **{n: None}), "NULL")
    _refused(E, _conv(E, one, "step", y=FAKE), "overlaps")
    _refused(E, _conv(E, one, "step", y=FAKE + 3 * STEP), "overlaps")


def test_scan_shapes(E):
    ok = dict(B=2, H=4, G=2, T=70, d_k=16, d_v=8)
    for over in (dict(B=0), dict(H=0), dict(G=0), dict(G=3), dict(T=0), dict(d_k=0), dict(d_v=0), dict(d_k=257),
                 dict(d_v=1025), dict(act=5), dict(B=40000), dict(T=(1 << 24) + 1),
                 dict(B=16000, T=1 << 24)):
        s = E.make_ssm_shape(**(ok | over))
        assert E.e2ttt_ssm_workspace_bytes(s, 0) == E.e2ttt_ssm_workspace_bytes(s, 1) == 0
        assert E.e2ttt_ssm_saved_bytes(s) == 0
        for fn in ("fwd", "bwd"):
            _refused(E, _ssm(E, s, fn), "e2ttt_ssm_scan_" + fn)
    s = E.make_ssm_shape(**ok)
    assert E.e2ttt_ssm_saved_bytes(s) >= 4 * 2 * 4 * 16 * 8
    assert E.e2ttt_ssm_workspace_bytes(s, 1) > 0 < E.e2ttt_ssm_workspace_bytes(s, 0)


def test_scan_arguments(E):
    s = E.make_ssm_shape(2, 4, 2, 70, 16, 8)
    for n in ("q", "k", "v", "dt", "A", "y", "S_end", "workspace"):
        _refused(E, _ssm(E, s, "fwd", **{n: None}), "NULL")
    for n in ("q", "k", "v", "dt", "A", "saved_states", "dy", "dq", "dk", "dv", "ddt", "dA", "workspace"):
        _refused(E, _ssm(E, s, "bwd", **{n: None}), "NULL")
    _refused(E, _ssm(E, s, "bwd", D=None), "dD")
    _refused(E, _ssm(E, s, "bwd", dD=None), "dD")
    _refused(E, _ssm(E, s, "fwd", y=FAKE + 2 * STEP), "y overlaps input v")
    _refused(E, _ssm(E, s, "fwd", S_end=FAKE + 6 * STEP), "S_end overlaps input S0")
    _refused(E, _ssm(E, s, "fwd", saved_states=FAKE + 11 * STEP), "overlaps")
    _refused(E, _ssm(E, s, "bwd", dk=FAKE + 10 * STEP), "overlaps")
    _refused(E, _ssm(E, s, "fwd", q=FAKE + 1), "aligned")
    _refused(E, _ssm(E, s, "fwd", dt=FAKE + 3 * STEP + 2), "aligned")
    _refused(E, _ssm(E, s, "fwd", workspace_bytes=0), "too small")
    _refused(E, _ssm(E, s, "bwd", workspace_bytes=0), "too small")
    _refused(E, _ssm(E, s, "step"), "T must be 1")
    one = E.make_ssm_shape(2, 4, 2, 1, 16, 8)
    for n in ("q", "k", "v", "dt", "A", "S", "y"):
        _refused(E, _ssm(E, one, "step", **{n: None}), "NULL")
    _refused(E, _ssm(E, one, "step", y=FAKE + 6 * STEP + 4), "overlaps")


def test_null_shape(E):
    from test_weight_layers_chunk_b200 import _lib
    assert _lib.e2ttt_ssm_scan_fwd(None, *[FAKE] * 12, 0, None) == E.ERR_INVALID_ARG
    assert _lib.e2ttt_short_conv_fwd(None, *[FAKE] * 8) == E.ERR_INVALID_ARG
    assert _lib.e2ttt_ssm_workspace_bytes(None, 0) == 0


def _clip(E, g, n=None, act=None, out=None, norm=FAKE - STEP, ws=FAKE - 2 * STEP, max_norm=1.0, ws_bytes=None):
    n = n or [100] * len(g)
    act = act or [E.F32] * len(g)
    return E.e2ttt_clip_grad_norm(g, out, n, act, max_norm, norm, ws,
                                  E.e2ttt_grad_workspace_bytes(len(g)) if ws_bytes is None else ws_bytes, raw=True)


def test_grad_arguments(E):
    g = [FAKE, FAKE + STEP]
    _refused(E, _clip(E, g, norm=None), "norm")
    _refused(E, _clip(E, g, ws=None), "workspace")
    _refused(E, _clip(E, g, ws_bytes=0), "too small")
    _refused(E, _clip(E, g, ws=FAKE - 2 * STEP + 8), "256-byte")
    for m in (-1.0, float("nan"), float("inf")):
        _refused(E, _clip(E, g, max_norm=m), "max_norm")
    _refused(E, _clip(E, [FAKE, 0]), "gradient 1 is NULL")
    _refused(E, _clip(E, [FAKE, FAKE + 2]), "aligned")
    _refused(E, _clip(E, [FAKE, FAKE + 40]), "overlaps")             # in place, and they meet
    _refused(E, _clip(E, g, out=[0, FAKE + 40]), "overlaps")         # into another gradient
    _refused(E, _clip(E, g, out=[FAKE + 8, FAKE + 2 * STEP]), "overlaps")  # into its own, shifted
    _refused(E, _clip(E, g, out=[FAKE + 2 * STEP] * 2), "overlaps")
    _refused(E, _clip(E, g, norm=FAKE + 16), "overlaps")
    _refused(E, _clip(E, g, act=[E.F32, 7]), "dtype")
    _refused(E, _clip(E, g, n=[1 << 41, 1]), "2^40")
    assert E.e2ttt_grad_workspace_bytes(-1) == 0
    assert E.e2ttt_grad_norm([FAKE], [4], [E.F32], None, FAKE + STEP, 1 << 20, raw=True) == E.ERR_INVALID_ARG


def test_overlap_is_found_behind_a_long_tensor(E):
    """A range that ends inside an earlier, longer one, with others between them."""
    g = [FAKE, FAKE + 4000, FAKE + 8000, FAKE + 39_000]
    _refused(E, _clip(E, g, n=[10_000, 1, 1, 1], out=[FAKE + STEP, FAKE + 2 * STEP, FAKE + 3 * STEP, 0]), "overlaps")


@pytest.mark.parametrize("name", ["short_conv_fwd", "short_conv_step", "ssm_scan_fwd", "ssm_step"])
def test_conveniences_refuse_cpu_tensors(E, name):
    import torch
    dims = 3 if name.endswith("step") else 4
    z = torch.zeros((1,) * dims)
    args = {"short_conv_fwd": (z, z), "short_conv_step": (z, z, z), "ssm_scan_fwd": (z,) * 5,
            "ssm_step": (z,) * 6}[name]
    with pytest.raises(E.E2TTTError, match="CUDA"):
        getattr(E, name)(*args)
    with pytest.raises(E.E2TTTError):
        E.clip_grad_norm([z], 1.0)
    with pytest.raises(E.E2TTTError):
        E.grad_norm([])
    assert ctypes.sizeof(E.e2ttt_ssm_shape) == 28 and ctypes.sizeof(E.e2ttt_conv_shape) == 28
