"""One MoE layer through the library: what runs before, between and after dispatch and combine.

``decode_step``: router gate -> layout and FP8 dispatch -> experts with 4-bit weights (gate and
up with the gated activation, then down) -> combine.  ``router_training_step``: router gate with
the balance loss -> dispatch and combine -> gradients of both back to the router's logits.
``training_step``: the whole layer with bf16 experts, forward and backward; the rows of the FP8
dispatch and the activation's input are kept in 8 bits for the weights' gradients.

    python examples/moe_layer.py [--tokens 128] [--hidden 7168] [--inner 2048] [--experts 256]
                                 [--topk 8] [--steps 50] [--train]

runs the first two on random weights, compares them with plain torch and prints the time of a step;
with --train it times the third.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_get_layout_gb300 as ep  # noqa: E402


class Experts:
    """Gate-up and down matrices of E experts, quantised to 4 bits by groups of 128 inputs."""

    def __init__(self, num_experts, hidden, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.up_cfg = ep.W4Config(num_experts, hidden, 2 * inner, x_fp8=True, gated=True)
        self.down_cfg = ep.W4Config(num_experts, inner, hidden)
        self.up = self._matrix(self.up_cfg, gen)
        self.down = self._matrix(self.down_cfg, gen)

    @staticmethod
    def _matrix(cfg, gen):
        shape = (cfg.num_experts, cfg.out_features, cfg.in_features // 2)
        codes = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)
        groups = shape[:2] + (cfg.in_features // cfg.group_size,)
        scales = 0.5 + torch.rand(groups, device="cuda", generator=gen)
        scales = (scales * 0.2 / cfg.in_features ** 0.5).bfloat16()
        return {"codes": codes, "scales": scales, "packed": ep.w4_pack(cfg, codes, scales)}

    @staticmethod
    def dense(m, e):
        """W of one expert in fp32."""
        c = m["codes"][e]
        q = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() - 8
        return q * m["scales"][e].float().repeat_interleave(128, -1)


class MoELayer:
    """The layer's configuration and the buffers that a serving loop keeps."""

    def __init__(self, max_tokens, hidden, inner, num_experts, topk, num_groups=1, topk_groups=1):
        self.router = ep.RouterConfig(num_experts, topk, "sigmoid", num_groups, topk_groups,
                                      route_scale=2.5)
        self.cfg = ep.Config(max_tokens, hidden, topk, num_experts, 1, expert_alignment=8,
                             use_fp8_dispatch=True)
        self.experts = Experts(num_experts, hidden, inner)
        self.layout = ep.Layout(self.cfg)
        cap = self.cfg.capacity
        self.recv_x = torch.empty((cap, hidden), dtype=torch.uint8, device="cuda")
        self.recv_scale = torch.empty((cap, hidden // 128), device="cuda")
        self.mid = torch.empty((cap, inner), dtype=torch.bfloat16, device="cuda")
        self.rows = torch.empty((cap, hidden), dtype=torch.bfloat16, device="cuda")

    def decode_step(self, x, logits, bias):
        """x: bf16 [T, H]; logits: the router product's [T, E]; returns y, idx, weights."""
        idx, w = ep.route(self.router, logits, bias)
        ep.layout_and_dispatch(self.cfg, idx, x, layout=self.layout, recv_x=self.recv_x,
                               recv_scale=self.recv_scale)
        start, end = self.layout.expert_start, self.layout.expert_end
        n = idx.numel()
        e = self.experts
        ep.expert_w4(e.up_cfg, self.recv_x, *e.up["packed"][:2], start, end, n,
                     x_scale=self.recv_scale, out=self.mid)
        ep.expert_w4(e.down_cfg, self.mid, *e.down["packed"][:2], start, end, n, out=self.rows)
        return ep.combine(self.cfg, self.layout, self.rows, w), idx, w

    def reference(self, x, idx, w):
        """y of the same tokens in fp32 from the unpacked weights and unquantised rows."""
        y = torch.zeros(x.shape, device="cuda")
        for e in idx.unique().tolist():
            t, k = (idx == e).nonzero(as_tuple=True)
            h = x[t].float() @ Experts.dense(self.experts.up, e).T
            gate, up = h.chunk(2, -1)
            h = torch.nn.functional.silu(gate) * up @ Experts.dense(self.experts.down, e).T
            y.index_add_(0, t, h * w[t, k, None])
        return y


def router_training_step(cfg, router, x, logits, factors, dy, grad_loss, seq_start=None,
                         layout=None):
    """Stand-in experts that multiply their rows by factors [E] (powers of two): returns (y,
    loss, grad_x, grad_logits) for the gradient dy of y and the coefficients grad_loss of the
    balance and z losses."""
    idx, w, count, _, tokens, loss = ep.route_balance(router, logits, seq_start=seq_start)
    layout = ep.get_layout(cfg, idx, layout)
    rows, _, _ = ep.dispatch(cfg, layout, x)
    token, k = layout.src_info.clamp(min=0).long().unbind(1)      # of each row
    row_factor = factors[idx[token.clamp(max=len(x) - 1), k.clamp(max=idx.shape[1] - 1)]][:, None]
    rows = rows * row_factor
    y = ep.combine(cfg, layout, rows, w)
    grad_rows, grad_w = ep.combine_backward(cfg, layout, dy, w, rows)
    grad_x, _ = ep.dispatch_backward(cfg, layout, grad_rows * row_factor)
    grad_logits = ep.route_backward(router, logits, idx, grad_w, None, seq_start, count, tokens,
                                    grad_loss)
    return y, loss, grad_x, grad_logits


def training_reference(K, x, logits, factors, dy, grad_loss):
    """The same by autograd in fp64, one sequence, softmax scores with renormalised weights."""
    l = logits.double().requires_grad_(True)
    xs = x.double().requires_grad_(True)
    T, E = l.shape
    p = torch.softmax(l, 1)
    s, idx = p.topk(K, 1)
    w = s / s.sum(1, keepdim=True)
    y = xs * (w * factors.double()[idx]).sum(1, keepdim=True)
    share = torch.bincount(idx.flatten(), minlength=E).double() * E / (K * T)
    loss = torch.stack([(share * p.mean(0)).sum(), torch.logsumexp(l, 1).square().mean()])
    ((y * dy.double()).sum() + (loss * grad_loss.double()).sum()).backward()
    return y.detach(), loss.detach(), xs.grad, l.grad


class TrainedExperts:
    """Gate-up and down matrices of E experts in bf16."""

    def __init__(self, num_experts, hidden, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.up_cfg = ep.ExpertConfig(num_experts, hidden, 2 * inner, x_fp8=True)
        self.down_cfg = ep.ExpertConfig(num_experts, inner, hidden)
        self.up, self.down = (
            torch.empty((num_experts, n, h), dtype=torch.bfloat16, device="cuda").normal_(
                0, h ** -0.5, generator=gen) for n, h in ((2 * inner, hidden), (hidden, inner)))


def training_step(cfg, router, experts, x, logits, dy, grad_loss, layout=None):
    """The layer's forward and backward pass for the gradient dy of y and the coefficients grad_loss
    of the balance and z losses (cfg: FP8 dispatch).  Returns (y, loss, grad_x, grad_logits,
    grad_up, grad_down)."""
    e = experts
    idx, w, count, _, tokens, loss = ep.route_balance(router, logits)
    layout = ep.get_layout(cfg, idx, layout)
    seg = layout.expert_start, layout.expert_end, idx.numel()
    rows, scale, _ = ep.dispatch(cfg, layout, x)
    h = ep.expert_mm(e.up_cfg, rows, e.up, *seg, x_scale=scale, err=layout.err)
    a, h_q, h_scale = ep.act_save(h, *seg)
    out = ep.expert_mm(e.down_cfg, a, e.down, *seg, err=layout.err)
    y = ep.combine(cfg, layout, out, w)
    del h, a       # rows, scale, h_q and h_scale are what the backward pass keeps, and out
    grad_out, grad_w = ep.combine_backward(cfg, layout, dy, w, out)
    grad_a, _ = ep.expert_mm_backward(e.down_cfg, grad_out, *seg, w=e.down, err=layout.err)
    grad_h, a = ep.act_backward(grad_a, h_q, h_scale, *seg)
    _, grad_down = ep.expert_mm_backward(e.down_cfg, grad_out, *seg, x=a, err=layout.err)
    grad_rows, grad_up = ep.expert_mm_backward(e.up_cfg, grad_h, *seg, w=e.up, x=rows,
                                               x_scale=scale, err=layout.err)
    grad_x, _ = ep.dispatch_backward(cfg, layout, grad_rows)
    grad_logits = ep.route_backward(router, logits, idx, grad_w, None, None, count, tokens,
                                    grad_loss)
    return y, loss, grad_x, grad_logits, grad_up, grad_down


def layer_reference(K, experts, x, logits, dy, grad_loss):
    """The same by autograd in fp64 from unquantised rows and activations."""
    l = logits.double().requires_grad_(True)
    xs = x.double().requires_grad_(True)
    up, down = (m.double().requires_grad_(True) for m in (experts.up, experts.down))
    T, E = l.shape
    p = torch.softmax(l, 1)
    s, idx = p.topk(K, 1)
    w = s / s.sum(1, keepdim=True)
    y = torch.zeros_like(xs)
    for e in idx.unique().tolist():
        t, k = (idx == e).nonzero(as_tuple=True)
        gate, value = (xs[t] @ up[e].T).chunk(2, -1)
        out = torch.nn.functional.silu(gate) * value @ down[e].T
        y = y.index_add(0, t, out * w[t, k, None])
    share = torch.bincount(idx.flatten(), minlength=E).double() * E / (K * T)
    loss = torch.stack([(share * p.mean(0)).sum(), torch.logsumexp(l, 1).square().mean()])
    ((y * dy.double()).sum() + (loss * grad_loss.double()).sum()).backward()
    return y.detach(), loss.detach(), xs.grad, l.grad, up.grad, down.grad


def _clock(step, steps):
    for _ in range(5):
        step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(steps):
        step()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps * 1e3


def run(tokens=128, hidden=7168, inner=2048, experts=256, topk=8, steps=50):
    """Both steps; returns their times and errors (norm of the difference over the norm)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, hidden), device="cuda", generator=gen).bfloat16()
    logits = torch.randn((tokens, experts), device="cuda", generator=gen)
    bias = 0.01 * torch.randn(experts, device="cuda", generator=gen)
    groups = 4 if experts % 4 == 0 and experts >= 8 * topk else 1
    layer = MoELayer(tokens, hidden, inner, experts, topk, groups, max(1, groups // 2))
    y, idx, w = layer.decode_step(x, logits, bias)
    want = layer.reference(x, idx, w)
    out = {"decode_error": float((y.float() - want).norm() / want.norm()),
           "decode_us": _clock(lambda: layer.decode_step(x, logits, bias), steps)}
    cfg = ep.Config(tokens, hidden, topk, experts, 1, expert_alignment=8)
    router = ep.RouterConfig(experts, topk)
    dy = torch.randn((tokens, hidden), device="cuda", generator=gen).bfloat16()
    grad_loss = torch.tensor([0.01, 0.001], device="cuda")
    factors = 2.0 ** (torch.arange(experts, device="cuda") % 3 - 1).bfloat16()
    a = cfg, router, x, logits, factors, dy, grad_loss
    got = router_training_step(*a)
    ref = training_reference(topk, x, logits, factors, dy, grad_loss)
    for name, g, r in zip(("y", "loss", "grad_x", "grad_logits"), got, ref):
        out["training_%s_error" % name] = float((g.double() - r).norm() / r.norm())
    layout = ep.Layout(cfg)
    out["training_us"] = _clock(lambda: router_training_step(*a, layout=layout), steps)
    return out


def run_training(tokens=4096, hidden=7168, inner=2048, experts=256, topk=8, steps=10, check=True):
    """The whole layer's training step; returns its time and, with `check`, its errors (norm of the
    difference over the norm; the fp64 reference is for small layers)."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn((tokens, hidden), device="cuda", generator=gen).bfloat16()
             for _ in range(2))
    logits = torch.randn((tokens, experts), device="cuda", generator=gen)
    grad_loss = torch.tensor([0.01, 0.001], device="cuda")
    cfg = ep.Config(tokens, hidden, topk, experts, 1, use_fp8_dispatch=True)
    e = TrainedExperts(experts, hidden, inner)
    a = cfg, ep.RouterConfig(experts, topk), e, x, logits, dy, grad_loss
    layout = ep.Layout(cfg)
    got, out = training_step(*a, layout=layout), {}
    assert ep.check_error(layout) == ep.EP_OK
    if check:
        want = layer_reference(topk, e, x, logits, dy, grad_loss)
        names = "y", "loss", "grad_x", "grad_logits", "grad_up", "grad_down"
        for name, g, r in zip(names, got, want):
            out[name + "_error"] = float((g.double() - r).norm() / r.norm())
    del got
    out["us"] = _clock(lambda: training_step(*a, layout=layout), steps)
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 128), ("hidden", 7168), ("inner", 2048), ("experts", 256),
                          ("topk", 8), ("steps", 50)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--train", action="store_true", help="the bf16 layer's training step, timed")
    args = vars(ap.parse_args())
    train = args.pop("train")
    for k, v in (run_training(check=False, **args) if train else run(**args)).items():
        print("%-28s %.6g" % (k, v))
