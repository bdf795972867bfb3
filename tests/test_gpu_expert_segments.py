"""Segments whose starts and ends are any 32-bit values: an expert without rows is one, however far
its end lies below its start."""

import pytest
import torch

pytestmark = pytest.mark.gpu

LOW, HIGH, MARK = -(2**31), 2**31 - 1, 77.0


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


# rows 5 to 9 of ten are one expert's
@pytest.mark.parametrize("start,end", [
    ([5, 5, 10], [LOW, 9, LOW + 3]), ([HIGH, 5, LOW], [LOW, 9, LOW]), ([HIGH, 5, 9], [HIGH, 9, -1]),
    ([1, 5, 7], [-HIGH, 9, LOW + 6])])
def test_ends_far_below_their_starts(ep, start, end):
    gen = torch.Generator(device="cuda").manual_seed(5)

    def new(*shape):
        return torch.randn(shape, device="cuda", generator=gen).bfloat16()

    x, w, dy, h, da = new(10, 64), new(3, 72, 64), new(10, 72), new(10, 144), new(10, 72)
    cfg = ep.ExpertConfig(3, 64, 72)

    def run(start, end):
        seg = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, end)] + [4]
        mark = lambda n, t=torch.bfloat16: torch.full((10, n), MARK, dtype=t, device="cuda")  # noqa: E731
        out = ep.expert_mm(cfg, x, w, *seg, out=mark(72))
        gx, gw = ep.expert_mm_backward(cfg, dy, *seg, w=w, x=x, grad_x=mark(64))
        _, g32 = ep.expert_mm_backward(cfg, dy, *seg, x=x, grad_w_dtype=torch.float32)
        a, q, s = ep.act_save(h, *seg, a=mark(72), h_q=mark(144, torch.uint8),
                              h_scale=mark(2, torch.float32))
        dh, b = ep.act_backward(da, q, s, *seg, grad_h=mark(144), a=mark(72))
        return out, gx, gw, g32, a, q, s, dh, b

    got, want = run(start, end), run([0, 5, 9], [0, 9, 9])
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(got, want))
    assert (got[0][:5] == MARK).all() and (got[0][9:] == MARK).all()
    assert (got[2][0] == 0).all() and (got[2][2] == 0).all()
