"""Performance cases of the experts' own part of an MoE layer, between dispatch and combine: products
grouped by expert (``product``) and their gradients (``backward``), and the gated activation between
them with its input kept in 8 bits (``save``) and its gradient from there (``restore``).

``run`` computes a case in plain torch (32-bit, ``own`` false) or through the library's own entry
points (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import functools
import math

import torch

own = False

BLOCK = 128     # columns that share a scale
E4M3_MAX = 448.0


def listed():
    """The cases.  T tokens to K of E experts each; H columns in, N out (gate and up together where
    the activation is gated)."""
    mm = {"fp8": False, "gated": False, "fp32": False, "align": 128, "zipf": 0.0}
    act = {"align": 128, "zipf": 0.0}
    return [
        # one token of one request through its experts' gate and up matrices: latency
        dict(mm, name="product 1 token", op="product", T=1, E=256, K=8, H=7168, N=4096, gated=True,
             align=8),
        # a decode step's batch from an FP8 dispatch: the layer's weights pass once
        dict(mm, name="product 128 tokens fp8", op="product", T=128, E=256, K=8, H=7168, N=4096,
             fp8=True, gated=True, align=8),
        # odd ragged sizes, rows without padding, skewed routing
        dict(mm, name="product odd skewed", op="product", T=999, E=60, K=4, H=1408, N=1000, align=1,
             zipf=1.2),
        # a long prompt's chunk, down product
        dict(mm, name="product 4096 tokens", op="product", T=4096, E=256, K=8, H=2048, N=7168),
        # a shared expert over a training batch: one dense product
        dict(mm, name="product dense 16384", op="product", T=16384, E=1, K=1, H=7168, N=4096),
        # gradients of a small step with odd sizes, the weights' in 32 bits
        dict(mm, name="backward odd", op="backward", T=200, E=60, K=4, H=1408, N=1000, align=1,
             zipf=1.2, fp32=True),
        # gradients of a skewed batch whose rows an FP8 dispatch kept in 8 bits
        dict(mm, name="backward 8192 fp8 skewed", op="backward", T=8192, E=64, K=6, H=4096, N=2816,
             fp8=True, zipf=1.2),
        # gradients of a training micro-batch's gate and up matrices
        dict(mm, name="backward 4096 tokens", op="backward", T=4096, E=256, K=8, H=7168, N=4096),
        # the activation of a few tokens: latency
        dict(act, name="save 16 tokens", op="save", T=16, E=256, K=8, N=4096, align=8),
        # the activation of a training micro-batch
        dict(act, name="save 4096 tokens", op="save", T=4096, E=256, K=8, N=4096),
        # its gradient at odd sizes (a last block of 104 columns)
        dict(act, name="restore odd", op="restore", T=999, E=60, K=4, N=2000, align=1, zipf=1.2),
        # and at the micro-batch's
        dict(act, name="restore 4096 tokens", op="restore", T=4096, E=256, K=8, N=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "backward", "backward", "save", "restore"])
    E = rng.choice([1, 4, 8, 32, 60, 64, 128])
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    zipf = rng.choice([0.0, 0.0, 1.2])
    align = rng.choice([1, 8, 16, 128])
    N = 8 * _log(rng, 8, 896)
    if op in ("save", "restore"):
        T = min(_log(rng, 1, 20000), int(1.2e8 / (K * N)) + 1)
        return {"op": op, "T": T, "E": E, "K": K, "N": 16 * (N // 16), "align": align,
                "zipf": zipf}
    fp8 = rng.random() < 0.4
    step = 128 if fp8 else 8
    H = step * max(1, min(_log(rng, 64, 7168), int(5e9 / (E * N))) // step)
    gated = op == "product" and rng.random() < 0.4
    if gated:
        N = 32 * max(1, N // 32)
    T = min(_log(rng, 1, 20000), int(1.6e12 / (2.0 * K * N * H)) + 1)
    return {"op": op, "T": T, "E": E, "K": K, "H": H, "N": N, "fp8": fp8, "gated": gated,
            "fp32": op == "backward" and rng.random() < 0.4, "align": align, "zipf": zipf}


# ---- inputs -----------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)


def _normal(gen, scale, *shape):
    """Normal values in bf16, made in that type: the weights of a large layer are many."""
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=gen)


def _segments(case, gen):
    """The rows of each expert as a layout gives them: T tokens, each to K experts, some more
    popular than others, segments aligned."""
    T, E, K = case["T"], case["E"], case["K"]
    pull = -case["zipf"] * torch.log(1.0 + torch.randperm(E, device="cuda", generator=gen))
    score = pull - torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen)))
    idx = score.sort(dim=1, descending=True).indices[:, :K]
    count = torch.bincount(idx.reshape(-1), minlength=E)
    room = -(-count // case["align"]) * case["align"]
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), room.cumsum(0)])
    return {"case": case, "start": start.to(torch.int32),
            "end": (start[:-1] + count).to(torch.int32),
            # the host's copy of the counts, as a synchronising layout call returns it
            "active": count.nonzero()[:, 0], "most": int(count.max()),
            "cap": T * K + E * (case["align"] - 1)}


def _quantised(x):
    """(E4M3 bits, scales) of rows in blocks of 128 columns, the last one maybe short."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    blk = torch.zeros(rows, blocks * BLOCK, device=x.device)
    blk[:, :cols] = x
    blk = blk.view(rows, blocks, BLOCK)
    scale = blk.abs().amax(2) / E4M3_MAX
    q = blk / torch.where(scale == 0, 1, scale)[:, :, None]
    q = q.view(rows, blocks * BLOCK)[:, :cols].to(torch.float8_e4m3fn)
    return q.view(torch.uint8).contiguous(), scale


def prepare(case, seed):
    gen = _generator(seed)
    s = _segments(case, gen)
    cap, N = s["cap"], case["N"]
    if case["op"] in ("save", "restore"):
        # gate and up values as a product leaves them
        h = _normal(gen, 1.0, cap, N)
        s["a"] = torch.zeros(cap, N // 2, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "save":
            s["h"] = h
            s["q"] = torch.zeros(cap, N, dtype=torch.uint8, device="cuda")
            s["scale"] = torch.zeros(cap, 2 * -(-N // 2 // BLOCK), device="cuda")
            return s
        g, u = _quantised(h[:, : N // 2].float()), _quantised(h[:, N // 2:].float())
        s["q"], s["scale"] = torch.cat([g[0], u[0]], 1), torch.cat([g[1], u[1]], 1)
        s["grad_a"] = _normal(gen, 1e-3, cap, N // 2)
        s["grad_h"] = torch.zeros(cap, N, dtype=torch.bfloat16, device="cuda")
        return s
    E, H = case["E"], case["H"]
    s["w"] = _normal(gen, 1 / math.sqrt(H), E, N, H)
    s["x"], s["x_scale"] = _normal(gen, 1.0, cap, H), None
    if case["fp8"]:
        s["x"], s["x_scale"] = _quantised(s["x"].float())
    if case["op"] == "product":
        width = N // 2 if case["gated"] else N
        s["out"] = torch.zeros(cap, width, dtype=torch.bfloat16, device="cuda")
    else:
        s["grad_out"] = _normal(gen, 1e-3, cap, N)
        s["grad_x"] = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        s["grad_w"] = torch.zeros(E, N, H, dtype=kind, device="cuda")
    return s


# ---- plain forms ---------------------------------------------------------------

def _rows(s):
    """Rows of every expert in use, side by side [experts, most], and which of them are there."""
    e = s["active"]
    rows = s["start"][e][:, None] + torch.arange(s["most"], device=e.device)
    have = rows < s["end"][e][:, None]
    return e, torch.where(have, rows, 0), have


def _values(q, scale, dtype):
    """What E4M3 bits with a scale for each 128 columns stand for."""
    spread = scale.to(dtype).repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]
    return q.view(torch.float8_e4m3fn).float().to(dtype) * spread


def _inputs(s, rows, dtype):
    if s["x_scale"] is None:
        return s["x"][rows].to(dtype)
    return _values(s["x"][rows], s["x_scale"][rows], dtype)


def _gated(y):
    gate, up = y.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_product(s):
    e, rows, have = _rows(s)
    y = torch.bmm(_inputs(s, rows, torch.float32), s["w"][e].float().transpose(1, 2))
    if s["case"]["gated"]:
        y = _gated(y)
    out = torch.zeros_like(s["out"])
    out[rows[have]] = y[have].bfloat16()
    return {"out": out}


def _plain_backward(s):
    e, rows, have = _rows(s)
    dy = torch.where(have[:, :, None], s["grad_out"][rows].float(), 0)
    dx = torch.bmm(dy, s["w"][e].float())
    grad_x, grad_w = torch.zeros_like(s["grad_x"]), torch.zeros_like(s["grad_w"])
    grad_x[rows[have]] = dx[have].bfloat16()
    del dx
    x = torch.where(have[:, :, None], _inputs(s, rows, torch.float32), 0)
    grad_w[e] = torch.bmm(dy.transpose(1, 2), x).to(grad_w.dtype)
    return {"grad_x": grad_x, "grad_w": grad_w}


def _plain_save(s):
    _, rows, have = _rows(s)
    r = rows[have]
    h = s["h"][r].float()
    a, q, scale = torch.zeros_like(s["a"]), torch.zeros_like(s["q"]), torch.zeros_like(s["scale"])
    a[r] = _gated(h).bfloat16()
    gate, up = h.chunk(2, -1)
    g, u = _quantised(gate), _quantised(up)
    q[r], scale[r] = torch.cat([g[0], u[0]], 1), torch.cat([g[1], u[1]], 1)
    return {"a": a, "q": q.view(torch.float8_e4m3fn), "scale": scale}


def _halves(s, rows, dtype):
    """Gate and up values that a checkpoint stands for."""
    (gq, uq), (gs, us) = s["q"][rows].chunk(2, -1), s["scale"][rows].chunk(2, -1)
    return _values(gq.contiguous(), gs, dtype), _values(uq.contiguous(), us, dtype)


def _plain_restore(s):
    _, rows, have = _rows(s)
    r = rows[have]
    gate, up = _halves(s, r, torch.float32)
    da = s["grad_a"][r].float()
    c = 1 / (1 + torch.exp(-gate))
    grad_h, a = torch.zeros_like(s["grad_h"]), torch.zeros_like(s["a"])
    dg, du = da * up * c * (1 + gate * (1 - c)), da * gate * c
    grad_h[r] = torch.cat([dg, du], 1).bfloat16()
    a[r] = (gate * c * up).bfloat16()
    return {"grad_h": grad_h, "a": a}


# ---- the library's entry points ---------------------------------------------------

@functools.lru_cache(maxsize=None)
def _config(E, H, N, fp8, gated):
    import combine_get_layout_gb300 as ep

    return ep, ep.ExpertConfig(E, H, N, x_fp8=fp8, gated=gated)


def _own(s):
    c = s["case"]
    seg = s["start"], s["end"], c["T"] * c["K"]
    if c["op"] in ("product", "backward"):
        ep, cfg = _config(c["E"], c["H"], c["N"], c["fp8"], c["gated"])
        if c["op"] == "product":
            return {"out": ep.expert_mm(cfg, s["x"], s["w"], *seg, x_scale=s["x_scale"],
                                        out=s["out"])}
        grad_x, grad_w = ep.expert_mm_backward(
            cfg, s["grad_out"], *seg, w=s["w"], x=s["x"], x_scale=s["x_scale"],
            grad_x=s["grad_x"], grad_w=s["grad_w"])
        return {"grad_x": grad_x, "grad_w": grad_w}
    import combine_get_layout_gb300 as ep

    if c["op"] == "save":
        a, q, scale = ep.act_save(s["h"], *seg, a=s["a"], h_q=s["q"], h_scale=s["scale"])
        return {"a": a, "q": q.view(torch.float8_e4m3fn), "scale": scale}
    grad_h, a = ep.act_backward(s["grad_a"], s["q"], s["scale"], *seg, grad_h=s["grad_h"], a=s["a"])
    return {"grad_h": grad_h, "a": a}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "product":
        return _plain_product(state)
    if op == "backward":
        return _plain_backward(state)
    return _plain_save(state) if op == "save" else _plain_restore(state)


# ---- cost and definition -----------------------------------------------------------

def work(case):
    T, E, K, N = case["T"], case["E"], case["K"], case["N"]
    R = T * K
    half, scales = N // 2, 2 * -(-N // 2 // BLOCK) * 4
    if case["op"] == "save":
        return {"bytes": R * (2 * N + 2 * half + N + scales) + 8 * E, "flops": 6.0 * R * N}
    if case["op"] == "restore":
        return {"bytes": R * (2 * half + N + scales + 2 * N + 2 * half) + 8 * E,
                "flops": 8.0 * R * N}
    H = case["H"]
    # experts that at least one of T tokens reaches (on average, uniform routing)
    active = E * (1 - (1 - K / E) ** T)
    row = H + H // BLOCK * 4 if case["fp8"] else 2 * H
    if case["op"] == "product":
        return {"bytes": active * N * H * 2 + R * (row + 2 * (half if case["gated"] else N)) + 8 * E,
                "flops": 2.0 * R * N * H}
    return {"bytes": active * N * H * 2 + E * N * H * (4 if case["fp32"] else 2)
            + R * (row + 2 * N + 2 * H) + 8 * E, "flops": 4.0 * R * N * H}


def _by_definition(s, lo, hi, e):
    """One expert's outputs in 64 bits: {name: value} of its rows lo..hi or of its weights."""
    case, rows = s["case"], torch.arange(lo, hi, device="cuda")
    if case["op"] == "product":
        y = _inputs(s, rows, torch.float64) @ s["w"][e].double().T
        if case["gated"]:
            gate, up = y.chunk(2, 1)
            y = torch.nn.functional.silu(gate) * up
        return {"out": y}
    if case["op"] == "backward":
        dy = s["grad_out"][rows].double()
        return {"grad_x": dy @ s["w"][e].double(), "grad_w": dy.T @ _inputs(s, rows, torch.float64)}
    if case["op"] == "save":
        h = s["h"][rows].double()
        half = h.shape[1] // 2
        parts = [b for side in h.split(half, 1) for b in side.split(BLOCK, 1)]
        scale = torch.stack([b.abs().amax(1) for b in parts], 1) / E4M3_MAX
        return {"a": torch.nn.functional.silu(h[:, :half]) * h[:, half:], "scale": scale}
    gate, up = (v.requires_grad_(True) for v in _halves(s, rows, torch.float64))
    a = torch.nn.functional.silu(gate) * up
    grads = torch.autograd.grad(a, (gate, up), s["grad_a"][rows].double())
    return {"grad_h": torch.cat(grads, 1), "a": a.detach()}


def exact(case, seed):
    s = prepare(case, seed)
    names = {"product": ["out"], "backward": ["grad_x", "grad_w"], "save": ["a", "scale"],
             "restore": ["grad_h", "a"]}[case["op"]]
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    for e in s["active"].tolist():
        lo, hi = int(s["start"][e]), int(s["end"][e])
        for name, v in _by_definition(s, lo, hi, e).items():
            if name == "grad_w":
                out[name][e] = v
            else:
                out[name][lo:hi] = v
    if case["op"] == "save":
        return {"a": out["a"], "q": None, "scale": out["scale"]}   # codes: the scale's last bit
    return out
