"""Sizes beyond a C int are refused, not cut to their lower 32 bits."""
import pytest

from test_abi import E  # noqa: F401  (the fixture that builds and loads the library)

BIG = (1 << 32) + 1


def test_shapes(E):
    conv, ssm = dict(B=1, H=2, T=3, d=4, W=2), dict(B=1, H=2, G=1, T=3, d_k=4, d_v=5)
    for make, ok in ((E.make_conv_shape, conv), (E.make_ssm_shape, ssm)):
        make(**ok)
        for n in ok:
            for size in (BIG, 1 << 31, -BIG):
                with pytest.raises(E.E2TTTError, match=n) as err:
                    make(**{**ok, n: size})
                assert err.value.status == E.ERR_INVALID_ARG


@pytest.mark.gpu
def test_tensors(E):
    """A tensor of 2^32 + 1 tokens (or rows) of one value each."""
    import torch
    x = torch.empty(BIG, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 1, 1, device="cuda")
    for call in (lambda: E.short_conv_fwd(x.view(1, 1, BIG, 1), w),
                 lambda: E.short_conv_step(x.view(BIG, 1, 1), x.new_empty(BIG, 1, 0, 1), w, out=x.view(BIG, 1, 1)),
                 lambda: E.ssm_scan_fwd(*[x.view(1, 1, BIG, 1)] * 3, torch.empty(1, 1, BIG, device="cuda"), w.view(1))):
        with pytest.raises(E.E2TTTError) as err:
            call()
        assert err.value.status == E.ERR_INVALID_ARG
