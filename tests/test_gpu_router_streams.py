"""The router's calls on a stream that is given and not the current one, eager
and under capture."""

import pytest
import torch

from test_gpu_router import ep  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_forked_branch_of_a_capture_and_eager_calls_beside_its_replays(ep):  # noqa: F811
    cfg = ep.RouterConfig(256, 8)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn((3000, 256), device="cuda", generator=gen) for _ in range(2))
    want_x, want_y = ep.route_balance(cfg, x), ep.route_balance(cfg, y)
    out_x, out_y = (tuple(torch.empty_like(t) for t in want_x) for _ in range(2))
    size = ep.ep_route_workspace_bytes(cfg.c(), 1)
    branch, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    branch.wait_stream(torch.cuda.current_stream())
    ep.route_balance(cfg, y, out=out_y, stream=branch)      # keeps memory for that stream
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        branch.wait_stream(torch.cuda.current_stream())
        ep.route_balance(cfg, x, out=out_x, stream=branch)
        other = torch.empty(size, dtype=torch.uint8, device="cuda")
        for _ in range(8):      # beside the branch
            other.fill_(255)
        torch.cuda.current_stream().wait_stream(branch)
    torch.cuda.synchronize()
    for _ in range(50):
        for t in (*out_x, *out_y):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        ep.route_balance(cfg, y, out=out_y, stream=branch)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out_x, want_x))
        assert all(torch.equal(a, b) for a, b in zip(out_y, want_y))


def test_outputs_of_a_given_stream(ep):  # noqa: F811
    """Made by the calls themselves, read on the current stream after it."""
    cfg = ep.RouterConfig(64, 6, "sigmoid")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((2000, 64), device="cuda", generator=gen)
    want = ep.route_balance(cfg, x)
    grad = ep.route_backward(cfg, x, want[0], want[1])
    side = torch.cuda.Stream()
    for _ in range(20):
        torch.empty(1 << 22, device="cuda").fill_(7.0)      # freed while in flight
        side.wait_stream(torch.cuda.current_stream())
        got = ep.route_balance(cfg, x, stream=side)
        g = ep.route_backward(cfg, x, *ep.route(cfg, x, stream=side), stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(g, grad)
    with pytest.raises(ep.EpError):
        ep.route(cfg, x.cpu(), stream=side)
