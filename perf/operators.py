"""Performance cases of the MoE layer's operators beside dispatch and combine: the router gate
(``route``), the gate with its balance loss (``balance``), its gradient (``backward``) and the
experts' products with 4-bit weights (``w4``).

``run`` computes a case in plain torch (32-bit, ``own`` false) or through the library's own entry
points (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import functools
import math

import torch

own = False

# Rounds of redrawing tokens whose choice would hang on the last bits of a sigmoid.
REDRAWS = 8
# Least distance of two choice scores that decide an order (about 30 roundings of a score near 1).
CLEAR = 4e-6


def listed():
    """The cases.  T tokens, E experts, K selections a token; H and N as in the layer's products."""
    gate = {"bf16": False, "groups": 1, "kept": 1, "renorm": True, "scale": 1.0,
            "seqs": 1, "padded": 0.0, "dead": 0, "ld": 0}
    sig = dict(gate, score="sigmoid", groups=8, kept=4, scale=2.5)
    soft = dict(gate, score="softmax")
    w4 = {"groups": 128, "fp8": False, "gated": False, "zeros": False, "align": 8, "zipf": 0.0}
    return [
        # one token of one request: the router of a decode step, latency alone
        dict(sig, name="route 1 token", op="route", T=1, E=256, K=8),
        # a decode step's batch
        dict(sig, name="route 128 tokens", op="route", T=128, E=256, K=8),
        # a long prompt's chunk, logits as a bf16 product leaves them (full of ties)
        dict(soft, name="route 16384 bf16", op="route", T=16384, E=256, K=8, bf16=True),
        # a training micro-batch as one sequence
        dict(soft, name="balance 4096", op="balance", T=4096, E=256, K=8),
        # packed ragged sequences with padding tokens and two experts out of service
        dict(soft, name="balance 8191 ragged", op="balance", T=8191, E=64, K=6, renorm=False,
             seqs=37, padded=0.05, dead=2, ld=72),
        # the largest training batch of the sweep, sigmoid scores with a choice bias
        dict(sig, name="balance 16384", op="balance", T=16384, E=256, K=8, seqs=4),
        # gradients of the two training shapes
        dict(soft, name="backward 4096", op="backward", T=4096, E=256, K=8),
        dict(sig, name="backward 16384 bf16", op="backward", T=16384, E=256, K=8, bf16=True,
             seqs=4, padded=0.02),
        # one row through one matrix: a shared expert's down product, latency
        dict(w4, name="w4 1 row dense", op="w4", T=1, E=1, K=1, H=2048, N=7168),
        # one token's 8 of 256 experts, gate and up with the gated activation, FP8 rows
        dict(w4, name="w4 1 token fp8", op="w4", T=1, E=256, K=8, H=7168, N=4096, fp8=True,
             gated=True),
        # ragged sizes, small groups with zero points, skewed routing
        dict(w4, name="w4 odd skewed", op="w4", T=37, E=60, K=4, H=1408, N=1000, groups=32,
             zeros=True, zipf=1.2, align=1),
        # a decode step's batch: the whole layer's weights pass once
        dict(w4, name="w4 128 tokens fp8", op="w4", T=128, E=256, K=8, H=7168, N=4096, fp8=True,
             gated=True),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n == 24 * 128)


def draw(rng):
    if rng.random() < 0.55:
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 256, 384, 512])
        sigmoid = rng.random() < 0.5
        groups = rng.choice([1, 4]) if E >= 16 and E % 4 == 0 else 1
        kept = rng.choice([2, 3]) if groups == 4 else 1
        op = rng.choice(["route", "balance", "backward"])
        T = _log(rng, 1, 20000)
        return {"op": op, "score": "sigmoid" if sigmoid else "softmax", "T": T, "E": E,
                "K": rng.choice([1, 2, 4, 6, 8]), "bf16": rng.random() < 0.4, "groups": groups,
                "kept": kept, "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "seqs": min(T, _log(rng, 1, 64)) if op != "route" else 1,
                "padded": rng.choice([0.0, 0.03, 0.3]), "dead": rng.choice([0, 0, 1]),
                "ld": rng.choice([0, 0, E + 8])}
    E = rng.choice([1, 4, 8, 32, 60, 64, 128])
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    g = rng.choice([32, 64, 128])
    fp8 = rng.random() < 0.4
    step = 128 if fp8 else g
    H = step * max(1, _log(rng, 256, 7168) // step)
    H += step * (H // 128 == 24)
    gated = rng.random() < 0.5
    N = _log(rng, 64, 7168)
    N += N % 2 + 128 * (N // 128 == 24)
    T = min(_log(rng, 1, 256), max(1, 32 * E // K), max(1, int(3e10 / (K * N * H))))
    return {"op": "w4", "T": T, "E": E, "K": K, "H": H, "N": N, "groups": g, "fp8": fp8,
            "gated": gated, "zeros": rng.random() < 0.3, "align": rng.choice([1, 8, 16]),
            "zipf": rng.choice([0.0, 0.0, 1.2])}


# ---- inputs -----------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)


def _logits(case, gen):
    """Router logits: a token's own spread on top of an expert's popularity."""
    T, E = case["T"], case["E"]
    popular = 0.4 * torch.randn(E, device="cuda", generator=gen)

    def some():
        x = 1.5 * torch.randn(T, E, device="cuda", generator=gen) + popular
        if case["dead"]:
            x[:, : case["dead"]] = -math.inf
        return x.bfloat16() if case["bf16"] else x

    x, bias = some(), None
    if case["score"] == "sigmoid":
        # the balancing bias, moved by steps of 1e-3 against an expert's load
        bias = (torch.randn(E, device="cuda", generator=gen) * 40).round() * 1e-3
        for _ in range(REDRAWS):
            x = torch.where(_clear(case, x, bias)[:, None], x, some())
    return x, bias


def _clear(case, x, bias):
    """Tokens whose order of choice stands by more than CLEAR, in 64 bits: the others' whole
    numbers would depend on how a sigmoid is rounded."""
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    c = 1 / (1 + torch.exp(-x.double())) + bias.double()
    c = torch.where(torch.isinf(x), -9.0, c)
    ok = torch.ones(T, dtype=torch.bool, device=x.device)
    if G > 1:
        per = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        order = per.sort(dim=1, descending=True)
        ok &= order.values[:, case["kept"] - 1] - order.values[:, case["kept"]] > CLEAR
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order.indices[:, : case["kept"]], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -9.0)
    top = c.sort(dim=1, descending=True).values[:, : K + 1]
    far = (top[:, :-1] - top[:, 1:] > CLEAR) | (top[:, :-1] < -5)
    return ok & far.all(1)


def _router_state(case, seed):
    gen = _generator(seed)
    T, E, K, B = case["T"], case["E"], case["K"], case["seqs"]
    x, bias = _logits(case, gen)
    if case["ld"]:  # a slice of a wider product
        wide = torch.zeros(T, case["ld"], dtype=x.dtype, device="cuda")
        wide[:, :E] = x
        x = wide[:, :E]
    s = {"case": case, "logits": x, "bias": bias, "mask": None, "seq_start": None}
    if case["padded"]:
        s["mask"] = (torch.rand(T, device="cuda", generator=gen) >= case["padded"]).to(torch.uint8)
    if B > 1:
        cuts = torch.randint(0, T + 1, (B - 1,), device="cuda", generator=gen).sort().values
        ends = torch.tensor([0, T], device="cuda")
        s["seq_start"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    s["topk_idx"] = torch.zeros(T, K, dtype=torch.int64, device="cuda")
    s["topk_weights"] = torch.zeros(T, K, device="cuda")
    if case["op"] == "balance":
        s["expert_count"] = torch.zeros(B, E, dtype=torch.int32, device="cuda")
        s["expert_prob"] = torch.zeros(B, E, device="cuda")
        s["seq_tokens"] = torch.zeros(B + 2, dtype=torch.int32, device="cuda")
        s["loss"] = torch.zeros(2, device="cuda")
    if case["op"] == "backward":
        # what the forward pass left, the gates' gradient from the combine's backward (of a
        # mean over tokens), and the losses' coefficients
        f = _plain_route(s, True)
        s["topk_idx"], s["expert_count"], s["seq_tokens"] = f["idx"], f["count"], f["tokens"]
        s["grad_w"] = torch.randn(T, K, device="cuda", generator=gen) / T
        s["grad_loss"] = torch.tensor([0.01, 0.001], device="cuda")
        if case["score"] == "sigmoid":
            s["grad_loss"][1] = 0
        s["grad_logits"] = torch.zeros(T, E, dtype=x.dtype, device="cuda")
    return s


def _tiles(case):
    """Packed tiles of 64 weight rows, and blocks of 128 inputs."""
    rows = 32 if case["gated"] else 64
    outs = case["N"] // 2 if case["gated"] else case["N"]
    return -(-outs // rows), -(-case["H"] // 128)


def _w4_state(case, seed):
    gen = _generator(seed)
    T, E, K, H, g = case["T"], case["E"], case["K"], case["H"], case["groups"]
    tiles, blocks = _tiles(case)
    # routing of T tokens, each to K experts, some more popular than others
    pull = -case["zipf"] * torch.log(1.0 + torch.randperm(E, device="cuda", generator=gen))
    score = pull - torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen)))
    idx = score.sort(dim=1, descending=True).indices[:, :K]
    count = torch.zeros(E, dtype=torch.int64, device="cuda")
    count += (idx.reshape(-1, 1) == torch.arange(E, device="cuda")).sum(0)
    room = -(-count // case["align"]) * case["align"]
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), room.cumsum(0)])
    cap = T * K + E * (case["align"] - 1)
    # packed codes: bell-shaped (two small uniforms), as rounding normal weights gives them
    size = (E, tiles, blocks, 8, 32, 4)
    a = torch.randint(-2**31, 2**31 - 1, size, dtype=torch.int32, device="cuda", generator=gen)
    b = torch.randint(-2**31, 2**31 - 1, size, dtype=torch.int32, device="cuda", generator=gen)
    codes = (a & 0x77777777) + (b & 0x77777777) + 0x01010101
    del a, b
    scales = torch.rand(E, tiles, blocks * 128 // g, 64, device="cuda", generator=gen)
    scales = ((0.5 + scales) / (3.0 * math.sqrt(H))).bfloat16()
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(6, 11, scales.shape, dtype=torch.uint8, device="cuda", generator=gen)
    x, x_scale = torch.randn(cap, H, device="cuda", generator=gen), None
    if case["fp8"]:
        blk = x.view(cap, H // 128, 128)
        x_scale = blk.abs().amax(2) / 448
        x = (blk / x_scale[:, :, None]).reshape(cap, H).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = x.bfloat16()
    outs = case["N"] // 2 if case["gated"] else case["N"]
    return {"case": case, "x": x, "x_scale": x_scale, "codes": codes, "scales": scales,
            "zeros": zeros, "start": start.to(torch.int32),
            "end": (start[:-1] + count).to(torch.int32),
            "out": torch.zeros(cap, outs, dtype=torch.bfloat16, device="cuda"),
            # the host's copy of the counts, as a synchronising layout call returns it
            "active": count.nonzero()[:, 0], "most": int(count.max())}


def prepare(case, seed):
    return _w4_state(case, seed) if case["op"] == "w4" else _router_state(case, seed)


# ---- plain forms ---------------------------------------------------------------

def _plain_scores(s):
    """(logits, scores, normalised scores, log sum exp) of every expert, in 32 bits."""
    x = s["logits"].float()
    if s["case"]["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-x))
        return x, p, p / p.sum(1, keepdim=True), torch.zeros_like(x[:, 0])
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(1, keepdim=True)
    return x, e / z, e / z, (top + torch.log(z))[:, 0]


def _plain_tokens(s):
    """(valid [T], one-hot sequence of each valid token [B, T])."""
    T, B, dev = s["case"]["T"], s["case"]["seqs"], s["logits"].device
    valid = torch.ones(T, dtype=torch.bool, device=dev) if s["mask"] is None else s["mask"] != 0
    if s["seq_start"] is None:
        return valid, valid[None, :].float()
    t = torch.arange(T, device=dev)
    inside = (t >= s["seq_start"][:B, None]) & (t < s["seq_start"][1:, None])
    return valid, (inside & valid).float()


def _plain_route(s, stats):
    case = s["case"]
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    x, p, q, lse = _plain_scores(s)
    valid, member = _plain_tokens(s)
    dead = torch.isinf(x)
    choice = x if s["bias"] is None else torch.where(dead, -math.inf, p + s["bias"])
    if G > 1:
        per = choice.view(T, G, E // G).sort(dim=2, descending=True).values
        if s["bias"] is None:
            per = per[:, :, 0]
        else:
            per = torch.where(torch.isinf(per), 0, per)[:, :, :2].sum(2)
        best = per.sort(dim=1, descending=True, stable=True).indices[:, : case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter(1, best, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, -math.inf)
    order = choice.sort(dim=1, descending=True, stable=True)
    taken = torch.isfinite(order.values[:, :K]) & valid[:, None]
    idx = order.indices[:, :K]
    w = torch.where(taken, p.gather(1, idx), 0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1, total)
    out = {"idx": torch.where(taken, idx, -1), "w": w * case["scale"]}
    if not stats:
        return out
    chosen = torch.zeros(T, E, device=x.device).scatter(1, idx, taken.float())
    n = member.sum(1)
    some = torch.where(n == 0, 1, n)
    count, prob = member @ chosen, (member @ q) / some[:, None]
    full = (n > 0).sum()
    f = count * (E / K) / some[:, None]
    loss = (f * prob).sum() / torch.where(full == 0, 1, full)
    z = (lse * lse * valid).sum() / torch.where(n.sum() == 0, 1, n.sum())
    tokens = torch.cat([n, n.sum()[None], full[None]])
    return dict(out, count=count.to(torch.int32), prob=prob, tokens=tokens.to(torch.int32),
                loss=torch.stack([loss, z]))


def _plain_backward(s):
    case = s["case"]
    E, K, B = case["E"], case["K"], case["seqs"]
    x, p, q, lse = _plain_scores(s)
    valid, member = _plain_tokens(s)
    n = s["seq_tokens"].float()
    some = torch.where(n == 0, 1, n)
    # the balance loss by the normalised scores, the z loss by lse
    each = s["grad_loss"][0] * s["expert_count"] * (E / K) / (some[:B, None] ** 2 * some[B + 1])
    dq = member.T @ each
    dlse = s["grad_loss"][1] * 2 * lse / some[B]
    # the gate weights by the chosen scores
    taken, idx = s["topk_idx"] >= 0, s["topk_idx"].clamp(min=0)
    dw = torch.where(taken, s["grad_w"], 0) * case["scale"]
    if case["renorm"]:
        pk = torch.where(taken, p.gather(1, idx), 0)
        total = pk.sum(1, keepdim=True)
        total = torch.where(total == 0, 1, total)
        dw = torch.where(taken, (dw - (dw * pk).sum(1, keepdim=True) / total) / total, 0)
    dp = torch.zeros_like(x).scatter_add(1, idx, dw)
    if case["score"] == "sigmoid":
        dp = dp + (dq - (dq * q).sum(1, keepdim=True)) / p.sum(1, keepdim=True)
        dx = dp * p * (1 - p)
    else:
        dp = dp + dq
        dx = p * (dp - (dp * p).sum(1, keepdim=True) + dlse[:, None])
    return {"grad": torch.where(valid[:, None], dx, 0).to(s["logits"].dtype)}


def _weights(s, e, dtype):
    """The weight rows of experts `e` [len(e), 64 * tiles, 128 * blocks], in packed row order.

    Word (piece, lane, i) of a tile and block holds 8 inputs of row 8 * (lane / 4) + piece:
    inputs 32 i + 8 (lane % 4) + 2 j and + 1 in its 4-bit fields j and j + 4."""
    tiles, blocks = _tiles(s["case"])
    b = s["codes"][e].view(torch.uint8).view(len(e), tiles, blocks, 8, 8, 4, 4, 4)
    f = torch.stack([b & 15, b >> 4], -1).view(len(e), tiles, blocks, 8, 8, 4, 4, 2, 4)
    f = f.permute(0, 1, 4, 3, 2, 6, 5, 8, 7).reshape(len(e), tiles * 64, blocks * 128)

    def spread(v):
        return v.transpose(2, 3).reshape(len(e), tiles * 64, -1, 1)

    w = f.to(dtype).view(len(e), tiles * 64, -1, s["case"]["groups"])
    w -= 8 if s["zeros"] is None else spread(s["zeros"][e]).to(dtype)
    w *= spread(s["scales"][e]).to(dtype)
    return w.view(len(e), tiles * 64, blocks * 128)[:, :, : s["case"]["H"]]


def _inputs(s, dtype):
    if s["x_scale"] is None:
        return s["x"].to(dtype)
    x = s["x"].view(torch.float8_e4m3fn).float().to(dtype).view(len(s["x"]), -1, 128)
    return (x * s["x_scale"].to(dtype)[:, :, None]).view(len(s["x"]), -1)


def _outputs(s, y):
    """Packed output rows (last dimension) -> the product's, through the gated activation."""
    case = s["case"]
    if case["gated"]:
        y = y.view(*y.shape[:-1], -1, 2, 4)
        gate, up = y[..., 0, :], y[..., 1, :]
        y = (gate / (1 + torch.exp(-gate)) * up).flatten(-2)
        return y[..., : case["N"] // 2]
    return y[..., : case["N"]]


def _plain_w4(s):
    e = s["active"]
    rows = s["start"][e][:, None] + torch.arange(s["most"], device=e.device)
    have = rows < s["end"][e][:, None]
    x = _inputs(s, torch.float32)[torch.where(have, rows, 0)]
    y = _outputs(s, torch.bmm(x, _weights(s, e, torch.float32).transpose(1, 2)))
    out = torch.zeros_like(s["out"])
    out[rows[have]] = y[have].bfloat16()
    return {"out": out}


# ---- the library's entry points ---------------------------------------------------

@functools.lru_cache(maxsize=None)
def _router(E, K, score, groups, kept, renorm, scale):
    import combine_get_layout_gb300 as ep

    return ep, ep.RouterConfig(num_experts=E, num_topk=K, score=score, num_groups=groups,
                               topk_groups=kept, renormalize=renorm, route_scale=scale)


@functools.lru_cache(maxsize=None)
def _product(E, H, N, group, fp8, gated, zeros):
    import combine_get_layout_gb300 as ep

    return ep, ep.W4Config(num_experts=E, in_features=H, out_features=N, group_size=group,
                           x_fp8=fp8, gated=gated, has_zeros=zeros)


def _own(s):
    c = s["case"]
    if c["op"] == "w4":
        ep, cfg = _product(c["E"], c["H"], c["N"], c["groups"], c["fp8"], c["gated"], c["zeros"])
        return {"out": ep.expert_w4(cfg, s["x"], s["codes"], s["scales"], s["start"], s["end"],
                                    c["T"] * c["K"], zeros=s["zeros"], x_scale=s["x_scale"],
                                    out=s["out"])}
    ep, cfg = _router(c["E"], c["K"], c["score"], c["groups"], c["kept"], c["renorm"], c["scale"])
    if c["op"] == "route":
        idx, w = ep.route(cfg, s["logits"], s["bias"], s["mask"], topk_idx=s["topk_idx"],
                          topk_weights=s["topk_weights"])
        return {"idx": idx, "w": w}
    if c["op"] == "balance":
        idx, w, count, prob, tokens, loss = ep.route_balance(
            cfg, s["logits"], s["bias"], s["mask"], s["seq_start"],
            out=(s["topk_idx"], s["topk_weights"], s["expert_count"], s["expert_prob"],
                 s["seq_tokens"], s["loss"]))
        return {"idx": idx, "w": w, "count": count, "prob": prob, "tokens": tokens, "loss": loss}
    return {"grad": ep.route_backward(
        cfg, s["logits"], s["topk_idx"], s["grad_w"], s["mask"], s["seq_start"],
        s["expert_count"], s["seq_tokens"], s["grad_loss"], grad_logits=s["grad_logits"])}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "w4":
        return _plain_w4(state)
    if op == "backward":
        return _plain_backward(state)
    return _plain_route(state, op == "balance")


# ---- cost and definition -----------------------------------------------------------

def work(case):
    T, E, K = case["T"], case["E"], case["K"]
    if case["op"] == "w4":
        H, N, g = case["H"], case["N"], case["groups"]
        # experts that at least one of T tokens reaches (on average, uniform routing)
        active = E * (1 - (1 - K / E) ** T)
        matrix = N * H // 2 + N * H // g * (3 if case["zeros"] else 2)
        row = H + H // 128 * 4 if case["fp8"] else 2 * H
        outs = N // 2 if case["gated"] else N
        return {"bytes": active * matrix + T * K * (row + 2 * outs) + 8 * E,
                "flops": 2.0 * T * K * N * H}
    word, B = 2 if case["bf16"] else 4, case["seqs"]
    mask = T if case["padded"] else 0
    if case["op"] == "route":
        return {"bytes": T * E * word + T * K * 12 + mask, "flops": 6.0 * T * E}
    if case["op"] == "balance":
        return {"bytes": T * E * word + T * K * 12 + mask + B * E * 8, "flops": 8.0 * T * E}
    return {"bytes": 2 * T * E * word + T * K * 12 + mask + B * E * 4, "flops": 12.0 * T * E}


def _exact_loss(s, x, idx):
    """Gate weights and losses in 64 bits as a function of the logits x, for given choices."""
    case = s["case"]
    T, E, K, B = case["T"], case["E"], case["K"], case["seqs"]
    dev = x.device
    valid = torch.ones(T, device=dev).bool() if s["mask"] is None else s["mask"].bool()
    lse = torch.logsumexp(x, 1)
    if case["score"] == "sigmoid":
        score = torch.sigmoid(x)
        share = score / score.sum(1, keepdim=True)
        z = torch.zeros((), dtype=torch.float64, device=dev)
    else:
        score = share = torch.softmax(x, 1)
        z = lse[valid].square().sum() / max(1, int(valid.sum()))
    taken = idx >= 0
    w = score.gather(1, idx.clamp(min=0)) * taken
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    starts = [0, T] if s["seq_start"] is None else s["seq_start"].tolist()
    terms, probs = [], []
    for b in range(B):
        t = torch.arange(starts[b], starts[b + 1], device=dev)
        t = t[valid[t]]
        mean = share[t].sum(0) / max(1, len(t))
        probs.append(mean)
        if len(t):
            load = torch.bincount(idx[t][taken[t]], minlength=E).double() * E / (K * len(t))
            terms.append((load * mean).sum())
    balance = torch.stack(terms).mean() if terms else z * 0
    return w * case["scale"], torch.stack(probs), torch.stack([balance, z])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        x, out = _inputs(s, torch.float64), torch.zeros_like(s["out"], dtype=torch.float64)
        for e in s["active"].tolist():
            lo, hi = int(s["start"][e]), int(s["end"][e])
            w = _weights(s, torch.tensor([e], device="cuda"), torch.float64)[0]
            out[lo:hi] = _outputs(s, x[lo:hi] @ w.T)
        return {"out": out}
    # The choice as the definition orders it: near ties of sigmoids were redrawn, so 32 and 64
    # bits choose alike, and equal bf16 logits go to the lowest index in both.
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    x = s["logits"].double()
    if case["op"] == "backward":
        idx = s["topk_idx"]
    else:
        c = x.clone() if s["bias"] is None else torch.sigmoid(x) + s["bias"].double()
        c[torch.isinf(x)] = -math.inf
        if G > 1:
            per = c.view(T, G, -1).topk(1 if s["bias"] is None else min(2, E // G), 2).values
            per = per.masked_fill(torch.isinf(per), 0).sum(2)
            rank = (-per).argsort(dim=1, stable=True).argsort(1)
            c[(rank >= case["kept"]).repeat_interleave(E // G, 1)] = -math.inf
        idx = (-c).argsort(dim=1, stable=True)[:, :K]
        idx = idx.masked_fill(torch.isinf(c.gather(1, idx)), -1)
        if s["mask"] is not None:
            idx = idx.masked_fill(s["mask"][:, None] == 0, -1)
    if case["op"] == "backward":
        x.requires_grad_(True)
        w, _, loss = _exact_loss(s, x, idx)
        ((w * s["grad_w"].double()).sum() + (loss * s["grad_loss"].double()).sum()).backward()
        grad = torch.nan_to_num(x.grad)  # experts out of service: 0 * inf
        return {"grad": grad}
    w, prob, loss = _exact_loss(s, x, idx)
    if case["op"] == "route":
        return {"idx": None, "w": w}
    return {"idx": None, "w": w, "count": None, "prob": prob, "tokens": None, "loss": loss}
