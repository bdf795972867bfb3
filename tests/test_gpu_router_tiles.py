"""The router gate, its losses and gradient where a warp routes several tokens
(over 32 tokens an SM, up to 128 experts), with groups, ties, a bias and many
choices, against the plain 64-bit forms of layer_ref.py."""

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_router import config, dev, ep, make, rtol, starts_of  # noqa: F401

pytestmark = pytest.mark.gpu

# Least distance of choice scores that are not equal: 16 roundings of a score
# and its bias, of magnitude under 2.
CLEAR = 16 * 2 * ref.EPS


def choice_scores(l, c):
    """[T, E] choice scores in 64 bits, as layer_ref.choose orders them."""
    s = l if c["score"] == "softmax" else 1 / (1 + np.exp(-l))
    return np.where(np.isneginf(l), -np.inf, s + (0.0 if c["bias"] is None else c["bias"]))


def clear(l, c):
    """Tokens none of whose orders hangs on a rounding: choice scores, and
    groups by their two best, are the same or over CLEAR apart.  Softmax
    compares logits as they are."""
    if c["score"] == "softmax":
        return np.ones(len(l), bool)

    def wide(v, parts):
        order = np.argsort(-v, axis=1, kind="stable")
        gap = np.diff(np.take_along_axis(v, order, 1), axis=1)
        parts = np.take_along_axis(parts, order[:, :, None], 1)
        same = (parts[:, 1:] == parts[:, :-1]).all(2)
        return (same | (abs(gap) > CLEAR)).all(1)

    v = choice_scores(l, c)
    v = np.where(np.isneginf(v), -9.0 - np.arange(v.shape[1]), v)
    ok = wide(v, v[:, :, None])
    if c["kept"] < c["groups"]:
        per = -np.sort(-v.reshape(len(l), c["groups"], -1), axis=2)[:, :, :2]
        per = np.where(per > -9, per, 0)
        ok &= wide(per.sum(2), per)
    return ok


def inputs(T, E, tied, **case):
    """make()'s, every `tied`-th token with equal logits and its neighbour
    with few values; tokens that are not clear repeat one that is.  (Equal
    scores by a bias make groups of equal sums of other parts: few are clear.)"""
    l, c, x = make(T, E, **case)
    rng = np.random.default_rng(11)
    finite = np.isfinite(l)
    l[::tied] = np.where(finite[::tied], 0.25, l[::tied])
    l[1::tied] = np.where(finite[1::tied], rng.integers(0, 3, l[1::tied].shape) * 0.5, l[1::tied])
    ok = clear(l, c)
    assert ok.mean() > 0.9
    l[~ok] = l[np.flatnonzero(ok)[2]]
    x.copy_(torch.from_numpy(l))
    return l, c, x


def both(**case):
    return [dict(case, score=s) for s in ("softmax", "sigmoid")]


CASES = [
    *both(T=5000, E=60, K=4, groups=4, kept=2, tied=7, B=3),
    *both(T=16384, E=96, K=8, groups=4, kept=3, tied=5, B=5, scale=2.5),
    *both(T=16384, E=16, K=4, groups=8, kept=4, tied=3, B=1),
    *both(T=6001, E=64, K=8, groups=8, kept=4, tied=7, B=97, bf16=True, masked=0.05,
          bias=False),
    *both(T=5000, E=128, K=10, groups=16, kept=5, tied=7, B=4, ld=136, bias=False),
    *both(T=5001, E=100, K=6, tied=4, B=2, dead=3, renorm=False),
    *both(T=4900, E=120, K=9, groups=3, kept=2, tied=7, B=2, dead=5),
    *both(T=9000, E=32, K=8, tied=2, B=1, bf16=True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_several_tokens_a_warp(ep, case):  # noqa: F811
    case = dict(case)
    B, T, E = case.pop("B"), case["T"], case["E"]
    l, c, x = inputs(**case)
    cfg, mask, bias = config(ep, E, c), dev(c["mask"]), dev(c["bias"], torch.float32)
    starts = starts_of(T, B) if B > 1 else np.array([0, T], np.int32)
    seq = dev(starts) if B > 1 else None
    want, ww = ref.route(l, **c)
    rt = rtol(E, l)
    idx, w = ep.route(cfg, x, bias, mask)
    assert np.array_equal(idx.cpu().numpy(), want)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=rt, atol=0)
    got = ep.route_balance(cfg, x, bias, mask, seq)
    assert torch.equal(got[0], idx)
    np.testing.assert_allclose(got[1].cpu().numpy(), ww, rtol=rt, atol=0)
    rc, rp, rn, rl = ref.balance(l, want, c["score"], c["mask"], starts)
    count, prob, tokens, loss = (t.cpu().numpy() for t in got[2:])
    assert np.array_equal(count, rc) and np.array_equal(tokens, rn)
    # sums of at most T positive terms
    np.testing.assert_allclose(prob, rp, rtol=rt + ref.EPS * (T + 8), atol=0)
    np.testing.assert_allclose(loss, rl, rtol=2 * rt + ref.EPS * (2 * T + E + B), atol=0)
    for _ in range(30):
        again = ep.route_balance(cfg, x, bias, mask, seq)
        assert all(torch.equal(a, b) for a, b in zip(again, got))

    rng = np.random.default_rng(8)
    gw = (rng.standard_normal((T, c["K"])) / T).astype(np.float32)
    gl = np.array([0.5, 0.01 if c["score"] == "softmax" else 0.0], np.float32)
    rg, size = ref.backward(l, want, gw.astype(np.float64), gl.astype(np.float64), c["score"],
                            c["renorm"], c["scale"], c["mask"], starts, rc)
    g = ep.route_backward(cfg, x, idx, dev(gw), mask, seq, got[2], got[4], dev(gl))
    tol = 4 * (rt + 16 * ref.EPS) * size + (2.0 ** -8 * abs(rg) if case.get("bf16") else 0)
    assert (abs(g.double().cpu().numpy() - rg) <= tol + 1e-38).all()
