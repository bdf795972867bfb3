"""Scores far from a row's maximum keep the accuracy of 32-bit exponentials:
the error does not grow with the exponent."""

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_router import dev, ep  # noqa: F401

pytestmark = pytest.mark.gpu

# (tokens, experts): a warp a token without and with vectors, over 512
# experts, several tokens a warp
SIZES = [(64, 32), (64, 256), (16, 1000), (5000, 64), (5000, 128)]


def exponential(d):
    """Roundings of exp(d) as a power of two: 2^-22 of the exponential, 1 / 20
    for each of |d| from ln 2 as one number (2.8e-9 of the exponent), and
    two to put what rounds off the exponent back."""
    return 4 + np.abs(d) / 20 + 2


def logits(T, E, low, high, seed=0):
    """Multiples of 1/8, so that differences are exact; the highest in every row."""
    rng = np.random.default_rng(seed)
    l = rng.integers(low * 8, high * 8 + 1, (T, E)) / 8.0
    l[np.arange(T), rng.integers(0, E, T)] = high
    return l


def probs(ep, l, score):  # noqa: F811
    """Every token's scores over their sum, each token a sequence of its own."""
    T, E = l.shape
    x = torch.from_numpy(l).float().cuda()
    cfg = ep.RouterConfig(E, 1, score)
    seq = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    return ep.route_balance(cfg, x, seq_start=seq)[3].double().cpu().numpy()


@pytest.mark.parametrize("T,E", SIZES)
def test_softmax(ep, T, E):  # noqa: F811
    l = logits(T, E, -80, 0)
    p = np.exp(l) / np.exp(l).sum(1, keepdims=True)
    # the score, the sum of the scores (its terms near the maximum), its
    # reciprocal (2), the product and the division by one token
    tol = ref.EPS * (exponential(l) + exponential(2) + E / 32 + 5 + 4)
    assert (abs(probs(ep, l, "softmax") - p) <= tol * p).all()
    # gate weights: the same with a true quotient
    K = min(E, 8)
    cfg = ep.RouterConfig(E, K, renormalize=False)
    far = np.where(l == 0, 0, l - 40).clip(-80)
    q = np.exp(far) / np.exp(far).sum(1, keepdims=True)
    idx, w = (t.cpu().numpy() for t in ep.route(cfg, torch.from_numpy(far).float().cuda()))
    want = np.take_along_axis(q, idx, 1)
    tol = ref.EPS * (exponential(far) + exponential(2) + E / 32 + 5 + 4)
    assert (abs(w - want) <= np.take_along_axis(tol, idx, 1) * want).all()


@pytest.mark.parametrize("T,E", SIZES)
@pytest.mark.parametrize("high", [-60, -5, 20])
def test_sigmoid(ep, T, E, high):  # noqa: F811
    l = logits(T, E, -80, high, 1)
    s = 1 / (1 + np.exp(-l))
    # the exponential, one more, its reciprocal (2); the sum of the scores;
    # its reciprocal (2), the product and the division by one token
    one = exponential(l) + 3
    tol = ref.EPS * (one + one.max(1, where=l >= high - 2, initial=0)[:, None] + E / 32 + 5 + 4)
    p = s / s.sum(1, keepdims=True)
    assert (abs(probs(ep, l, "sigmoid") - p) <= tol * p).all()
    # gate weights that are not renormalised are the scores themselves
    K = min(E, 8)
    cfg = ep.RouterConfig(E, K, "sigmoid", renormalize=False)
    low = l - l.max(1, keepdims=True) + max(high - 40, -70)
    low = np.maximum(low, -80.0)
    idx, w = (t.cpu().numpy() for t in ep.route(cfg, torch.from_numpy(low).float().cuda()))
    want = np.take_along_axis(1 / (1 + np.exp(-low)), idx, 1)
    tol = ref.EPS * (np.take_along_axis(exponential(low), idx, 1) + 6)
    assert (abs(w - want) <= tol * want).all()


@pytest.mark.parametrize("T,E", SIZES)
@pytest.mark.parametrize("score,high", [("softmax", 0), ("sigmoid", -40)])
def test_gradient(ep, T, E, score, high):  # noqa: F811
    """Of the balance loss, whose terms keep their sizes."""
    l = logits(T, E, -80, high, 2)
    x = torch.from_numpy(l).float().cuda()
    cfg = ep.RouterConfig(E, min(E, 4), score)
    idx, w, count, _, tokens, _ = ep.route_balance(cfg, x)
    gl = torch.tensor([1.0, 0.0], device="cuda")
    g = ep.route_backward(cfg, x, None, None, None, None, count, tokens, gl)
    none = np.full((T, cfg.num_topk), -1)
    starts = np.array([0, T])
    want, size = ref.backward(l, none, np.zeros(none.shape), np.array([1.0, 0.0]), score, True,
                              1.0, None, starts, count.cpu().numpy())
    # the expert's own score, the weighted mean of the counts (a sum over the
    # experts, twice), and some ten products and differences
    one = exponential(l) + 3
    tol = ref.EPS * (one + 2 * exponential(high) + 2 * (E / 32 + 5) + 12)
    assert (abs(g.double().cpu().numpy() - want) <= tol * size + 1e-38).all()


def test_ends_of_the_range(ep):  # noqa: F811
    """Infinities, values past the exponent's range and NaN."""
    inf = float("inf")
    x = torch.tensor([[-inf, -1e30, -200.0, 0.0, 200.0, 1e30, inf, -87.0]], device="cuda")
    idx, w = ep.route(ep.RouterConfig(8, 7, "sigmoid", renormalize=False), x)
    assert sorted(idx[0].tolist()) == [1, 2, 3, 4, 5, 6, 7]
    by = dict(zip(idx[0].tolist(), w[0].tolist()))
    assert by[1] == by[2] == 0 and by[3] == 0.5 and by[4] == by[5] == by[6] == 1
    assert abs(by[7] / np.exp(-87.0) - 1) < 1e-5
    x[0, 2] = float("nan")
    idx, w = ep.route(ep.RouterConfig(8, 7, "sigmoid", renormalize=False), x)
    assert 2 not in idx[0].tolist() and not torch.isnan(w).any()
    y = torch.tensor([[-inf, -1e30, -200.0, 0.0, -1e38, -80.0, -inf, -1.0]], device="cuda")
    idx, w = ep.route(ep.RouterConfig(8, 8, renormalize=False), y)
    assert idx[0].tolist() == [3, 7, 5, 2, 1, 4, -1, -1]
    assert (w[0, :3] > 0).all() and (w[0, 3:] == 0).all()
