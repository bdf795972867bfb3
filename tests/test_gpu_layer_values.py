"""The MoE layer's training step against 64-bit arithmetic that rounds where the library does: to
E4M3 with a scale for each 128 columns where rows and the activation's input are kept in 8 bits, to
bf16 where a call returns bf16.  What is left are sums in 32 bits, so that a wrong scale of a few
blocks shows."""

import importlib.util
import os

import pytest
import torch

import expert_ref as ref

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


NAMES = "y", "loss", "grad_x", "grad_logits", "grad_up", "grad_down"


def bf(t):
    return t.float().bfloat16().double()


def kept(t):
    """What E4M3 and a scale for each 128 columns keep of bf16 rows."""
    q, scale = ref.quantise(t.float())
    return ref.values(q, scale).double()


def reference(K, up, down, x, logits, dy, grad_loss):
    """(y, loss, grad_x, grad_logits, grad_up, grad_down), all on the CPU."""
    up, down, dy = up.double(), down.double(), dy.double()
    l = logits.double().requires_grad_(True)
    T, E = l.shape
    p = torch.softmax(l, 1)
    s, idx = p.topk(K, 1)
    w = s / s.sum(1, keepdim=True)
    share = torch.bincount(idx.flatten(), minlength=E).double() * E / (K * T)
    loss = torch.stack([(share * p.mean(0)).sum(), torch.logsumexp(l, 1).square().mean()])
    xq, wd = kept(x), w.detach()
    y, grad_x, grad_w = (torch.zeros(s, dtype=torch.float64) for s in (x.shape, x.shape, w.shape))
    grad_up, grad_down = torch.zeros_like(up), torch.zeros_like(down)
    for e in idx.unique().tolist():
        t, k = (idx == e).nonzero(as_tuple=True)
        h = bf(xq[t] @ up[e].T)
        gate, value = h.chunk(2, 1)
        out = bf(bf(torch.nn.functional.silu(gate) * value) @ down[e].T)
        y.index_add_(0, t, out * wd[t, k, None])
        grad_out = bf(dy[t] * wd[t, k, None])
        grad_w[t, k] = (dy[t] * out).sum(1)
        grad_a = bf(grad_out @ down[e])
        gate, value = kept(gate.contiguous()), kept(value.contiguous())
        c = torch.sigmoid(gate)
        grad_h = bf(torch.cat([grad_a * value * c * (1 + gate * (1 - c)), grad_a * gate * c], 1))
        grad_down[e] = bf(grad_out.T @ bf(gate * c * value))
        grad_up[e] = bf(grad_h.T @ bf(xq[t]))
        grad_x.index_add_(0, t, bf(grad_h @ up[e]))
    ((w * grad_w).sum() + (loss * grad_loss.double()).sum()).backward()
    return bf(y), loss.detach(), bf(grad_x), l.grad, grad_up, grad_down


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [
    (1, 256, 128, 16, 2), (37, 512, 384, 32, 4), (300, 1024, 264, 8, 2), (200, 256, 520, 60, 6)])
def test_step_against_rounded_arithmetic(layer, tokens, hidden, inner, experts, topk):
    """Where a value lies next to a border of its rounding, what the sums are off by takes it to the
    other side: by a step of bf16 (2^-7), and where that meets a border of E4M3 (one step of bf16 in
    2^4 does) by a step of that (2^-3).  E4M3 rows enter the first product to 1.4 * 2^-12 at worst,
    2^-13 in the norm of a sum: one value of h in 2^5 goes over in bf16 and one in 2^9 in E4M3; in
    the norm 2^-7 / 2^2.5 and 2^-3 / 2^4.5.  y takes the first, twice through gate and up: 2^-8.5
    with the later roundings' (less, their products are of bf16 rows); gradients take the second,
    through gate and up: 2^-7.  Bounds of twice that."""
    ep = layer.ep
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn((tokens, hidden), device="cuda", generator=gen).bfloat16()
             for _ in range(2))
    logits = torch.randn((tokens, experts), device="cuda", generator=gen)
    grad_loss = torch.tensor([0.01, 0.001], device="cuda")
    cfg = ep.Config(tokens, hidden, topk, experts, 1, use_fp8_dispatch=True)
    e = layer.TrainedExperts(experts, hidden, inner)
    got = layer.training_step(cfg, ep.RouterConfig(experts, topk), e, x, logits, dy, grad_loss)
    want = reference(topk, *(t.cpu() for t in (e.up, e.down, x, logits, dy, grad_loss)))
    bounds = dict(dict.fromkeys(("grad_x", "grad_logits", "grad_up", "grad_down"), 2.0 ** -6),
                  y=2.0 ** -7, loss=1e-5)
    off = {n: float((g.cpu().double() - r).norm() / r.norm())
           for n, g, r in zip(NAMES, got, want)}
    assert all(off[n] <= b for n, b in bounds.items()), off
    # rows of the gradients by themselves: a wrong scale of one block of one row
    for n, g, r in zip(("y", "grad_x"), (got[0], got[2]), (want[0], want[2])):
        rows = (g.cpu().double() - r).norm(dim=1) / r.norm(dim=1)
        assert float(rows.max()) <= 4 * bounds[n], (n, float(rows.max()))
