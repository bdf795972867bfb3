"""The router gate on values at the ends of their types: weights of finite
logits are finite, with and without statistics; a bias that is not a number."""

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_router import ep  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")
# (tokens, experts): a warp a token with and without vectors and padding, and
# several tokens a warp
SIZES = [(6, 256), (6, 200), (6, 45), (6, 600), (5000, 60), (5000, 128)]


@pytest.mark.parametrize("T,E", SIZES)
@pytest.mark.parametrize("bf16", [False, True])
def test_huge_finite_logits_beside_minus_infinity(ep, T, E, bf16):  # noqa: F811
    """Sums of a few of a row's logits overflow; their softmax does not."""
    big = 3.0e38
    l = np.zeros((T, E))
    l[:, ::3] = -INF
    l[0::3, [1, 2, 4, 5]] = big
    l[1::3, 1:] = -big
    l[2::3] = np.where(np.isinf(l[2::3]), -INF, big)
    dt = torch.bfloat16 if bf16 else torch.float32
    x = torch.from_numpy(l).to(dt).cuda()
    cfg = ep.RouterConfig(E, 4)
    idx, w = ep.route(cfg, x)
    full = x[:6].double().cpu().numpy()
    want, ww = ref.route(full, 4)
    assert np.array_equal(idx[:6].cpu().numpy(), want)
    # shares of equal or vanishing scores: a quotient of small whole numbers
    np.testing.assert_allclose(w[:6].cpu().numpy(), ww, rtol=4 * ref.EPS, atol=0)
    assert torch.equal(w[:3].repeat(-(-T // 3), 1)[:T], w)
    assert torch.equal(idx[:3].repeat(-(-T // 3), 1)[:T], idx)
    got = ep.route_balance(cfg, x)
    assert torch.equal(got[0], idx) and torch.equal(got[1], w)


@pytest.mark.parametrize("T,E", SIZES)
def test_nan_and_plus_infinity_still_show(ep, T, E):  # noqa: F811
    l = np.zeros((T, E))
    l[0::3, E - 1] = np.nan
    l[1::3, 7] = INF
    l[1::3, 8] = -INF
    x = torch.from_numpy(l).float().cuda()
    idx, w = ep.route(ep.RouterConfig(E, 4), x)
    assert torch.isnan(w[0::3]).all() and torch.isnan(w[1::3]).all()
    assert (w[2::3] == 0.25).all()
    assert (idx[0::3] != E - 1).all() and (idx[1::3, 0] == 7).all()


@pytest.mark.parametrize("T,E,groups,kept,K", [
    (40, 256, 8, 3, 8), (40, 60, 4, 2, 4), (40, 160, 8, 3, 6), (40, 64, 32, 5, 4),
    (5000, 64, 8, 3, 4), (5000, 60, 4, 2, 4), (5000, 128, 16, 4, 8), (40, 256, 1, 1, 8),
])
def test_an_expert_whose_bias_is_nan_is_out_of_the_choice(ep, T, E, groups, kept, K):  # noqa: F811
    """As with a bias of -inf: neither chosen nor counted for its group."""
    rng = np.random.default_rng(6)
    l = np.stack([rng.permutation(E) for _ in range(40)]) / 32.0 - 4.0
    bias = rng.integers(-40, 41, E) / 1024.0
    out = rng.permutation(E)[:E // 2]
    bias[out] = np.nan
    kill = np.where(np.isnan(bias), -INF, bias)
    x = torch.from_numpy(np.tile(l, (T // 40, 1))).float().cuda()
    cfg = ep.RouterConfig(E, K, "sigmoid", groups, kept)
    idx, w = ep.route(cfg, x, torch.from_numpy(bias).float().cuda())
    want, ww = ref.route(l, K, "sigmoid", kill, groups, kept)
    assert np.array_equal(idx[:40].cpu().numpy(), want) and not np.isin(want, out).any()
    # a score of at most 2^-1 to 1 and a sum of K: E / 32 + 5 steps cover both
    rt = ref.EPS * (2 * (E / 32 + 5) + 40)
    np.testing.assert_allclose(w[:40].cpu().numpy(), ww, rtol=rt)
    assert torch.equal(idx, idx[:40].repeat(T // 40, 1))
    idx2, w2 = ep.route(cfg, x, torch.from_numpy(kill).float().cuda())
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    got = ep.route_balance(cfg, x, torch.from_numpy(bias).float().cuda())
    assert torch.equal(got[0], idx)
    np.testing.assert_allclose(got[1][:40].cpu().numpy(), ww, rtol=rt)


@pytest.mark.parametrize("T,E", [(40, 256), (40, 60), (6000, 60), (6000, 128), (40, 1000)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bad", [INF, np.nan])
def test_masked_tokens_get_no_gradient_whatever_comes_in(ep, T, E, score, bad):  # noqa: F811
    """Coefficients and gate gradients that are not finite, NaN in masked rows."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, E), device="cuda", generator=gen)
    mask = torch.rand(T, device="cuda", generator=gen) > 0.4
    x[~mask] = float("nan")
    cfg = ep.RouterConfig(E, 4, score)
    idx, w, count, _, tokens, _ = ep.route_balance(cfg, x, None, mask)
    gl = torch.tensor([bad, bad], device="cuda")
    gw = torch.where(mask[:, None], torch.randn((T, 4), device="cuda", generator=gen), bad)
    g = ep.route_backward(cfg, x, idx, gw, mask, None, count, tokens, gl)
    assert (g[~mask] == 0).all() and torch.isnan(g[mask]).any(1).all()
    gl.zero_()
    g = ep.route_backward(cfg, x, idx, gw, mask, None, count, tokens, gl)
    assert (g[~mask] == 0).all() and torch.isfinite(g).all()
