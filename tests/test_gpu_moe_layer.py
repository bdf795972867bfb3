"""The MoE layer example end to end: router gate, dispatch, experts' 4-bit
products and combine; and the router's training step."""

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
    dict(tokens=128, hidden=1024, inner=256, experts=8, topk=2),
    dict(tokens=64, hidden=7168, inner=256, experts=64, topk=8),
], ids=str)
def test_layer_against_plain_torch(layer, sizes):
    got = layer.run(steps=2, **sizes)
    # E4M3 rounds each input by up to 2^-4 of its value, uniformly: 2^-4 /
    # sqrt(3) in the norm, twice that through the product of gate and up
    # (silu' <= 1.1), besides bf16 rounding of the middle rows and of y
    assert got["decode_error"] < 2 * 1.1 * 2.0 ** -4 / 3 ** 0.5 + 2 * 2.0 ** -8
    # y: fp32 sums of positive multiples of x, one bf16 rounding
    assert got["training_y_error"] < 2.0 ** -8
    assert got["training_loss_error"] < 1e-5
    # grad_x: one bf16 rounding of each of K rows, one of their sum
    assert got["training_grad_x_error"] < 2.0 ** -7
    # the gate gradients are fp32 sums of `hidden` products of either sign,
    # whose magnitudes add up to about sqrt(hidden) times the sum
    assert got["training_grad_logits_error"] < sizes["hidden"] ** 1.5 * 2.0 ** -24 + 1e-4


def test_decode_step_from_a_graph(layer):
    """The whole decode step is recorded once and replayed on new inputs."""
    m = layer.MoELayer(16, 256, 128, 32, 4, 4, 2)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def inputs():
        return (torch.randn((16, 256), device="cuda", generator=gen).bfloat16(),
                torch.randn((16, 32), device="cuda", generator=gen))

    x, logits = inputs()
    bias = torch.zeros(32, device="cuda")
    m.decode_step(x, logits, bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.decode_step(x, logits, bias)
    for _ in range(3):
        a, b = inputs()
        x.copy_(a)
        logits.copy_(b)
        graph.replay()
        got = [t.clone() for t in out]
        want = m.decode_step(a, b, bias)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
