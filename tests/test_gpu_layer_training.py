"""A whole MoE layer's training step: router, FP8 dispatch, experts' products, activation with its
8-bit checkpoint, combine, and all gradients, against autograd in 64 bits."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    spec = importlib.util.spec_from_file_location(
        "moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("sizes", [
    dict(tokens=1, hidden=256, inner=128, experts=16, topk=2),
    dict(tokens=37, hidden=512, inner=384, experts=32, topk=4),
    dict(tokens=300, hidden=1024, inner=264, experts=8, topk=2),
    dict(tokens=700, hidden=256, inner=512, experts=60, topk=6),
], ids=str)
def test_against_autograd(layer, sizes):
    got = layer.run_training(steps=1, **sizes)
    # E4M3 rounds each value by up to 2^-4 of it, uniformly: 2^-4 / sqrt(3) in the norm
    step = 2.0 ** -4 / 3 ** 0.5
    # gate and up carry the rows' rounding (silu' <= 1.1), y their product's
    assert got["y_error"] < 2 * 1.1 * step + 2 * 2.0 ** -8
    assert got["loss_error"] < 1e-5
    # grad_logits: the gates' gradient is y's product with dy, of the size of the rounding where
    # terms of either sign cancel: norms over experts' rows keep y's bound
    assert got["grad_logits_error"] < 2 * 2.2 * step
    # grad_h takes the rows' rounding and the checkpoint's through gate and up, the weights'
    # gradients the rows' or the activation's once more
    assert got["grad_x_error"] < 2 * 2.2 * step
    assert got["grad_up_error"] < (2 * 2.2 + 1) * step
    assert got["grad_down_error"] < 2 * 2.2 * step


def test_step_from_a_graph(layer):
    """Recorded once and replayed on new inputs: the bits of an eager step."""
    ep = layer.ep
    cfg = ep.Config(24, 256, 2, 16, 1, 8, use_fp8_dispatch=True)
    e, layout, router = layer.TrainedExperts(16, 256, 128), ep.Layout(cfg), ep.RouterConfig(16, 2)
    gen = torch.Generator(device="cuda").manual_seed(4)

    def inputs():
        return [torch.randn(s, device="cuda", generator=gen).to(t) for s, t in (
            ((24, 256), torch.bfloat16), ((24, 16), torch.float32), ((24, 256), torch.bfloat16))]

    grad_loss = torch.tensor([0.01, 0.001], device="cuda")
    held = inputs()

    def step(a):
        return layer.training_step(cfg, router, e, a[0], a[1], a[2], grad_loss, layout)

    step(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for _ in range(3):
        new = inputs()
        for t, n in zip(held, new):
            t.copy_(n)
        graph.replay()
        got = [t.clone() for t in out]
        want = step(new)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert ep.check_error(layout) == ep.EP_OK
