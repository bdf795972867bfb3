"""The router's calls from several host threads at once, each on a stream of
its own."""

import threading

import pytest
import torch

from test_gpu_router import ep  # noqa: F401

pytestmark = pytest.mark.gpu


def test_threads_with_different_numbers_of_experts(ep):  # noqa: F811
    """Kernels that all of 513 to 2048 experts share, with shared memory that
    goes by the number of experts: no call lowers another's limit."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    jobs = []
    for E in (2048, 1200, 2048, 1900):
        x = torch.randn((64, E), device="cuda", generator=gen)
        cfg = ep.RouterConfig(E, 4, num_groups=4, topk_groups=3)
        out = ep.route_balance(cfg, x)
        jobs.append((cfg, x, tuple(torch.empty_like(t) for t in out), out, torch.cuda.Stream()))
    gws = [torch.randn((64, 4), device="cuda", generator=gen) for _ in jobs]
    grads = [ep.route_backward(c, x, want[0], g) for (c, x, _, want, _), g in zip(jobs, gws)]
    torch.cuda.synchronize()
    said, begin = [], threading.Barrier(len(jobs))

    def work(cfg, x, out, want, stream, gw, grad):
        try:
            begin.wait(60)
            with torch.cuda.stream(stream):
                got = torch.empty_like(grad)
                for _ in range(400):
                    ep.route_balance(cfg, x, out=out)
                    ep.route(cfg, x, topk_idx=out[0], topk_weights=out[1])
                    ep.route_backward(cfg, x, out[0], gw, grad_logits=got)
                stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip((*out, got), (*want, grad))):
                said.append("other outputs")
        except Exception as e:
            said.append(repr(e))

    threads = [threading.Thread(target=work, args=(*j, g, d)) for j, g, d in zip(jobs, gws, grads)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not said, said[0]
