"""The router gate, its losses and its gradient on the GPU against plain
64-bit forms (layer_ref.py)."""

import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def make(T, E, K, score="softmax", bf16=False, groups=1, kept=1, renorm=True, scale=1.0, ld=0,
         masked=0.0, dead=0, bias=True, seed=0):
    """A case's inputs.  A token's logits are distinct multiples of 1/32 in
    shuffled order (bf16 holds them), so that sigmoids are far apart; the bias
    is a multiple of 1/1024."""
    rng = np.random.default_rng(seed)
    l = np.stack([rng.permutation(E) for _ in range(max(T, 1))])[:T].reshape(T, E)
    l = (l - E // 2) / 32.0 if E <= 256 else (l - E // 2) / 256.0
    l = np.maximum(l, -10.0)
    if bf16:
        l = torch.from_numpy(l).bfloat16().double().numpy()
    if dead:
        l[:, rng.permutation(E)[:dead]] = -INF
    c = dict(K=K, score=score, groups=groups, kept=kept, renorm=renorm, scale=scale)
    c["bias"] = (rng.integers(-40, 41, E) / 1024.0 if score == "sigmoid" and bias else None)
    c["mask"] = rng.random(T) >= masked if masked else None
    dt = torch.bfloat16 if bf16 else torch.float32
    wide = torch.full((T, max(ld, E)), 7.0, dtype=dt, device="cuda")
    wide[:, :E] = torch.from_numpy(l).to(dt)
    return l, c, wide[:, :E]


def config(ep, E, c):
    return ep.RouterConfig(E, c["K"], c["score"], c["groups"], c["kept"], c["renorm"], c["scale"])


def dev(a, dtype=None):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a), dtype=dtype).cuda()


def rtol(E, l):
    """Roundings of a score in fp32: of the exponent (its size times one), of
    the exponential, of a sum of E terms in E / 32 + 5 steps, of two quotients
    and a product; and of a sum over the chosen."""
    span = 2 * min(20.0, float(np.abs(l[np.isfinite(l)]).max(initial=0.0)))
    return ref.EPS * (2 * span + 2 * (E / 32 + 5) + 24)


CASES = [
    dict(T=1, E=1, K=1), dict(T=3, E=7, K=7, renorm=False), dict(T=5, E=8, K=2, scale=2.5),
    dict(T=33, E=60, K=4, ld=61), dict(T=64, E=64, K=6, masked=0.3, dead=2),
    dict(T=17, E=64, K=32), dict(T=40, E=96, K=8, bf16=True, ld=97),
    dict(T=129, E=256, K=8), dict(T=130, E=256, K=8, bf16=True, groups=8, kept=3),
    dict(T=31, E=256, K=1, ld=260), dict(T=9, E=130, K=8), dict(T=9, E=132, K=3, ld=133),
    dict(T=6, E=384, K=6, dead=380, groups=3, kept=2), dict(T=4, E=512, K=8, bf16=True),
    dict(T=3, E=1000, K=16), dict(T=3, E=2048, K=32, bf16=True), dict(T=2, E=2047, K=32),
    dict(T=65, E=256, K=8, score="sigmoid", groups=8, kept=4, scale=2.5, masked=0.1),
    dict(T=65, E=256, K=8, score="sigmoid", bias=False, renorm=False, bf16=True),
    dict(T=12, E=60, K=6, score="sigmoid", groups=4, kept=2, dead=3),
    dict(T=12, E=32, K=3, score="sigmoid", groups=32, kept=5),
    dict(T=5, E=2048, K=8, score="sigmoid", groups=16, kept=2),
    dict(T=5, E=160, K=6, score="sigmoid", groups=8, kept=3, bf16=True, ld=168),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_route(ep, case):
    l, c, x = make(**case)
    bias, mask = dev(c["bias"], torch.float32), dev(c["mask"])
    want, w = ref.route(l, **c)
    idx, got = ep.route(config(ep, case["E"], c), x, bias, mask)
    assert np.array_equal(idx.cpu().numpy(), want)
    np.testing.assert_allclose(got.cpu().numpy(), w, rtol=rtol(case["E"], l), atol=0)


@pytest.mark.parametrize("E,K,bf16", [(256, 8, False), (64, 32, True), (60, 60 // 2, False),
                                      (512, 32, False)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_scores_go_to_the_lower_index(ep, E, K, bf16, score):
    """All equal; a few values; -0 beside +0; ties of groups."""
    rng = np.random.default_rng(4)
    l = np.concatenate([np.zeros((2, E)), rng.integers(0, 3, (20, E)) * 1.0,
                        np.where(rng.random((4, E)) < 0.5, -0.0, 0.0)])
    x = torch.from_numpy(l).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    for groups, kept in ((1, 1), (4, 3)):
        c = dict(K=min(K, E // groups * kept), score=score, groups=groups, kept=kept, bias=None)
        want, _ = ref.route(l + 0.0, **c)
        idx, _ = ep.route(ep.RouterConfig(E, c["K"], score, groups, kept), x)
        assert np.array_equal(idx.cpu().numpy(), want)


def test_extreme_logits(ep):
    """Infinities, NaN, rows with nothing to choose, the type's largest and
    lowest values."""
    E, K = 256, 4
    big = float(np.finfo(np.float32).max)
    l = np.tile(np.linspace(-4, 4, E), (7, 1))
    l[0] = -INF
    l[1, 5:] = -INF
    l[1, 2] = -INF
    l[2, 9] = np.nan
    l[3, 9] = INF
    l[4] = -big
    l[5, 100] = big
    l[6, :] = -INF
    l[6, 31] = 3.0
    x = torch.from_numpy(l).float().cuda()
    cfg = ep.RouterConfig(E, K, renormalize=True)
    idx, w, count, prob, tokens, loss = (t.cpu().numpy() for t in ep.route_balance(cfg, x))
    want, _ = ref.route(l, K)
    assert np.array_equal(idx, want)
    assert (idx[0] == -1).all() and (w[0] == 0).all()
    assert list(idx[1]) == [4, 3, 1, 0] and np.isfinite(w[1]).all()
    assert 9 not in idx[2] and np.isnan(w[2]).all()       # a NaN row says so
    assert idx[3, 0] == 9 and np.isnan(w[3]).any()
    assert list(idx[4]) == [0, 1, 2, 3]
    np.testing.assert_array_equal(w[4], np.full(K, 0.25, np.float32))
    assert idx[5, 0] == 100 and w[5, 0] == 1 and (w[5, 1:] == 0).all()
    assert list(idx[6]) == [31, -1, -1, -1] and list(w[6]) == [1, 0, 0, 0]
    assert np.isnan(loss).all() and tokens[0] == 7
    assert count.sum() == (idx >= 0).sum()
    # the finite rows alone: finite losses and gradients, zeros where out of service
    y = x[[0, 1, 4, 6]].contiguous()
    idx, w, count, prob, tokens, loss = ep.route_balance(cfg, y)
    assert torch.isfinite(prob).all() and torch.isfinite(loss[0])
    g = ep.route_backward(cfg, y, idx, torch.ones_like(w), None, None, count, tokens,
                          torch.tensor([1.0, 0.0], device="cuda"))
    assert torch.isfinite(g).all()
    assert (g[torch.isneginf(y)] == 0).all() and (g[0] == 0).all()


def starts_of(T, B, seed=3):
    rng = np.random.default_rng(seed)
    return np.concatenate([[0], np.sort(rng.integers(0, T + 1, B - 1)), [T]]).astype(np.int32)


BALANCE = [
    dict(T=1, E=8, K=2, B=1), dict(T=5, E=8, K=2, B=9), dict(T=300, E=64, K=6, B=1, masked=0.2),
    dict(T=300, E=60, K=4, B=11, masked=0.5, ld=64), dict(T=2000, E=16, K=2, B=1),
    dict(T=257, E=256, K=8, B=3, bf16=True), dict(T=100, E=256, K=8, B=100, score="sigmoid",
                                                  groups=8, kept=4, scale=2.5),
    dict(T=40, E=2048, K=32, B=2), dict(T=64, E=130, K=6, B=2, score="sigmoid", dead=4),
    dict(T=7, E=32, K=3, B=1, masked=1.1),
    dict(T=200, E=8, K=2, B=33), dict(T=150, E=8, K=1, B=65), dict(T=90, E=16, K=2, B=1057),
    dict(T=6000, E=24, K=2, B=97, masked=0.02),
]


@pytest.mark.parametrize("case", BALANCE, ids=str)
def test_balance_and_backward(ep, case):
    case = dict(case)
    B = case.pop("B")
    l, c, x = make(**case)
    T, E, K = case["T"], case["E"], case["K"]
    cfg, mask, bias = config(ep, E, c), dev(c["mask"]), dev(c["bias"], torch.float32)
    starts = starts_of(T, B) if B > 1 else np.array([0, T], np.int32)
    seq = dev(starts) if B > 1 else None
    idx, w, count, prob, tokens, loss = ep.route_balance(cfg, x, bias, mask, seq)
    want, ww = ref.route(l, **c)
    rt = rtol(E, l)
    assert np.array_equal(idx.cpu().numpy(), want)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=rt, atol=0)
    rc, rp, rn, rl = ref.balance(l, want, c["score"], c["mask"], starts)
    assert np.array_equal(count.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rn)
    # sums of at most T positive terms
    np.testing.assert_allclose(prob.cpu().numpy(), rp, rtol=rt + ref.EPS * (T + 8), atol=0)
    np.testing.assert_allclose(loss.cpu().numpy(), rl, rtol=2 * rt + ref.EPS * (2 * T + E + B),
                               atol=0)
    # the same inputs give the same bits
    again = ep.route_balance(cfg, x, bias, mask, seq)
    assert all(torch.equal(a, b) for a, b in zip(again, (idx, w, count, prob, tokens, loss)))

    rng = np.random.default_rng(8)
    gw = (rng.standard_normal((T, K)) / T).astype(np.float32)
    gl = np.array([0.5, 0.01 if c["score"] == "softmax" else 0.0], np.float32)
    a = (l, want, gw.astype(np.float64), gl.astype(np.float64), c["score"], c["renorm"],
         c["scale"], c["mask"], starts, rc)
    rg, size = ref.backward(*a)
    g = ep.route_backward(cfg, x, idx, dev(gw), mask, seq, count, tokens, dev(gl))
    g64 = g.double().cpu().numpy()
    tol = 4 * (rt + 16 * ref.EPS) * size + (2.0 ** -8 * abs(rg) if case.get("bf16") else 0)
    assert g.dtype == x.dtype and (abs(g64 - rg) <= tol + 1e-38).all()
    # differences of the 64-bit objective along random directions; the
    # third-order term of a central difference is h^2 = 1e-8 of the values
    for _ in range(2):
        d = np.where(np.isfinite(l), rng.standard_normal((T, E)), 0.0)
        h = 1e-4
        up, down = (ref.objective(l + sgn * h * d, *a[1:]) for sgn in (1, -1))
        slope = (up - down) / (2 * h)
        near = (abs(d) * tol).sum() + 1e-6 * (abs(d) ** 3 * size).sum() + 1e-11 * abs(up) / h
        assert abs((g64 * d).sum() - slope) <= near + 1e-30
    # the terms one at a time: they add up
    only_w = ep.route_backward(cfg, x, idx, dev(gw), mask).double().cpu().numpy()
    only_l = ep.route_backward(cfg, x, None, None, mask, seq, count, tokens,
                               dev(gl)).double().cpu().numpy()
    assert (abs(only_w + only_l - g64) <= 2 * tol + 2.0 ** -7 * bool(case.get("bf16")) *
            (abs(only_w) + abs(only_l)) + 1e-38).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_single_renormalised_choice_weighs_one(ep, score):
    """w = s / s is 1 to the bit, and passes no gradient on."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    for E in (1, 8, 60, 256, 1000):
        cfg = ep.RouterConfig(E, 1, score, route_scale=2.5)
        x = 3 * torch.randn((6000, E), device="cuda", generator=gen)
        idx, w = ep.route(cfg, x)
        assert (w == 2.5).all()
        g = ep.route_backward(cfg, x, idx, torch.randn(w.shape, device="cuda", generator=gen))
        assert (g == 0).all()


def test_no_tokens(ep):
    cfg = ep.RouterConfig(16, 2)
    x = torch.empty((0, 16), device="cuda")
    idx, w = ep.route(cfg, x)
    assert idx.shape == (0, 2)
    for seq in (None, torch.zeros(4, dtype=torch.int32, device="cuda")):
        out = ep.route_balance(cfg, x, seq_start=seq)
        assert all((t == 0).all() for t in out[2:])
        g = ep.route_backward(cfg, x, out[0], out[1], None, seq, out[2], out[4], out[5])
        assert g.shape == (0, 16)


def test_workspace_need_not_be_clean_and_columns_past_E_stay(ep):
    l, c, x = make(500, 60, 4, masked=0.2, ld=64)
    cfg, mask, seq = config(ep, 60, c), dev(c["mask"]), dev(starts_of(500, 7))
    want = ep.route_balance(cfg, x, None, mask, seq)
    size = ep.ep_route_workspace_bytes(cfg.c(), 7)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    got = ep.route_balance(cfg, x, None, mask, seq, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (ws[size:] == 255).all()
    wide = torch.full((500, 68), 5.0, device="cuda")
    ep.route_backward(cfg, x, want[0], want[1], mask, grad_logits=wide[:, :60])
    assert (wide[:, 60:] == 5.0).all()
    assert (wide[~mask][:, :60] == 0).all()


def test_another_stream_and_a_graph(ep):
    l, c, x = make(200, 256, 8, masked=0.1)
    cfg, mask = config(ep, 256, c), dev(c["mask"])
    want = [t.clone() for t in ep.route_balance(cfg, x, None, mask)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.zeros_like(x)
    out = tuple(torch.empty_like(t) for t in want)
    ws = torch.empty(ep.ep_route_workspace_bytes(cfg.c(), 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y.copy_(x)
        ep.route_balance(cfg, y, None, mask, out=out, workspace=ws)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.route_balance(cfg, y, None, mask, out=out, workspace=ws)
        g = ep.route_backward(cfg, y, out[0], out[1], mask, None, out[2], out[4], out[5])
    y.copy_(x.flip(0).contiguous())
    ref_out = ep.route_balance(cfg, y, None, mask)
    ref_g = ep.route_backward(cfg, y, ref_out[0], ref_out[1], mask, None, ref_out[2], ref_out[4],
                              ref_out[5])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref_out)) and torch.equal(g, ref_g)


def test_torch_layer_refuses(ep):
    cfg = ep.RouterConfig(16, 2)
    x = torch.zeros((4, 16), device="cuda")
    bad = [
        lambda: ep.route(cfg, x.double()),
        lambda: ep.route(cfg, x[:, :15]),
        lambda: ep.route(cfg, x.T.contiguous().T),
        lambda: ep.route(cfg, x.cpu()), lambda: ep.route(cfg, x.to_sparse()),
        lambda: ep.route(cfg, x, topk_idx=torch.zeros((4, 2), dtype=torch.int64,
                                                      device="cuda").to_sparse()),
        lambda: ep.route(cfg, x.to("meta")),
        lambda: ep.route(cfg, x, torch.zeros(16, device="cuda")),             # bias: sigmoid only
        lambda: ep.route(ep.RouterConfig(16, 2, "sigmoid"), x, torch.zeros(15, device="cuda")),
        lambda: ep.route(cfg, x, None, torch.ones(3, dtype=torch.uint8, device="cuda")),
        lambda: ep.route(cfg, x, topk_idx=torch.zeros((4, 2), dtype=torch.int32, device="cuda")),
        lambda: ep.route(cfg, torch.zeros(65, device="cuda")[1:].view(4, 16)),  # misaligned
        lambda: ep.route_balance(cfg, x, workspace=torch.empty(16, dtype=torch.uint8,
                                                               device="cuda")),
        lambda: ep.route_backward(cfg, x, None, torch.zeros((4, 2), device="cuda")),
        lambda: ep.route_backward(cfg, x, grad_loss=torch.zeros(2, device="cuda")),
        lambda: ep.route_backward(cfg, x, grad_logits=x.bfloat16()),
    ]
    for call in bad:
        with pytest.raises(ep.EpError) as e:
            call()
        assert e.value.status == ep.EP_ERR_INVALID_ARG


def test_calls_on_two_streams_keep_apart(ep):
    """Each stream has its own scratch memory, and a larger call after a
    smaller one gets more of it."""
    cfg = ep.RouterConfig(512, 4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn((3000 + 500 * i, 512), device="cuda", generator=gen) for i in range(2)]
    seq = [torch.linspace(0, len(x), 2000 * i + 2, device="cuda").to(torch.int32)
           for i, x in enumerate(xs)]
    want = [ep.route_balance(cfg, x, seq_start=s) for x, s in zip(xs, seq)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for x, s, st in zip(xs, seq, streams):
            with torch.cuda.stream(st):
                got.append(ep.route_balance(cfg, x, seq_start=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
