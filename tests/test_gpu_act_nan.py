"""What is not finite in the input of the gated activation shows in its gradient too: the 8-bit
checkpoint between them loses no NaN, wherever it lies in a block of 128 columns."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def both(ep, h):
    """(a, h_q, h_scale, grad_h, a again) of rows of one expert, for gradients of 1."""
    h = torch.as_tensor(h).bfloat16().cuda()
    n, I = h.shape[0], h.shape[1] // 2
    seg = (torch.zeros(1, dtype=torch.int32, device="cuda"),
           torch.full((1,), n, dtype=torch.int32, device="cuda"), n)
    a, q, s = ep.act_save(h, *seg)
    grad_h, b = ep.act_backward(torch.ones((n, I), dtype=torch.bfloat16, device="cuda"), q, s, *seg)
    torch.cuda.synchronize()
    return [t.cpu() for t in (a, q, s, grad_h, b)]


# widths whose last block is whole, of one lane, of eight lanes less one, and of one lane in a warp's
# second step
WIDTHS = [128, 136, 8, 120, 264, 1000, 2048]


@pytest.mark.parametrize("I", WIDTHS)
@pytest.mark.parametrize("fill", [0.0, -0.0, 1.0, 1e-40])
def test_one_nan_anywhere(ep, I, fill):
    """In each 8 columns of gate and of up values, beside others, beside zeros alone."""
    at = sorted({c for c in range(0, 2 * I, 8)} | {I - 1, 2 * I - 1})
    h = np.full((len(at), 2 * I), fill, np.float32)
    h[np.arange(len(at)), at] = NAN
    a, q, s, grad_h, b = both(ep, h)
    for r, c in enumerate(at):
        col = c % I
        assert torch.isnan(a[r, col]) and torch.isnan(b[r, col])
        # both gradients of a pair contain both values, but for du, which has no u
        assert torch.isnan(grad_h[r, col])
        assert torch.isnan(grad_h[r, I + col]) or c >= I
        # other blocks have none
        lo, hi = col // 128 * 128, min(I, col // 128 * 128 + 128)
        for t, cols in ((b, I), (grad_h, 2 * I)):
            rest = np.ones(cols, bool)
            rest[lo:hi] = False
            if cols == 2 * I:
                rest[I + lo:I + hi] = False
            assert torch.isfinite(t[r][torch.from_numpy(rest)]).all()
        # what is not zero keeps its neighbours
        if fill not in (0.0, -0.0):
            assert int(torch.isnan(b[r]).sum()) == 1
    # the codes stay a dispatch's: zeros beside zeros
    if fill == 0.0:
        assert (q == 0).all() and (s == 0).all()
        assert int(torch.signbit(s).sum()) == len(at)


@pytest.mark.parametrize("I", WIDTHS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_rows_that_are_not_finite(ep, I, value):
    """Whole rows, and one side of them: every element of the gradient that the value reaches."""
    h = np.ones((5, 2 * I), np.float32)
    h[0] = value
    h[1, :I] = value
    h[2, I:] = value
    h[3] = 0
    a, q, s, grad_h, b = both(ep, h)
    assert torch.isnan(b[:3]).all() and torch.isnan(grad_h[0]).all()
    assert torch.isnan(grad_h[1]).all() and torch.isnan(grad_h[2, :I]).all()
    # zeros stay zeros, with a scale of +0
    assert (b[3] == 0).all() and (grad_h[3] == 0).all() and (s[3].view(torch.int32) == 0).all()
    assert torch.isfinite(b[4]).all() and torch.isfinite(grad_h[4]).all()
    assert not torch.isfinite(s[0]).any()


def test_zeros_of_either_sign_are_zeros(ep):
    h = np.zeros((2, 272), np.float32)
    h[1] = -0.0
    a, q, s, grad_h, b = both(ep, h)
    assert (s.view(torch.int32) == 0).all() and (q == 0).all()
    assert (grad_h == 0).all() and (b == 0).all() and (a == 0).all()
