"""Host-side checks of the router's and the 4-bit products' entry points that
need no GPU: struct layouts, sizes, argument validation.  No call here
reaches a kernel (bad arguments only, with fake addresses that nothing
dereferences)."""

import ctypes

import numpy as np
import pytest

import layer_ref as ref


@pytest.fixture(scope="module")
def ep():
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


A = 0x10000   # an aligned address
M = 0x10008   # a misaligned one


def test_struct_layouts(ep):
    assert ctypes.sizeof(ep.EpRouterConfig) == 32 and ctypes.sizeof(ep.EpW4Config) == 28


def router(ep, **kw):
    base = dict(num_experts=64, num_topk=4, score=0, num_groups=4, topk_groups=2, renormalize=1,
                logits_bf16=0, route_scale=1.0)
    base.update(kw)
    return ep.EpRouterConfig(*base.values())


@pytest.mark.parametrize("bad", [
    dict(num_experts=0), dict(num_experts=2049), dict(num_topk=0), dict(num_topk=33),
    dict(score=2), dict(num_groups=3), dict(num_groups=0), dict(num_groups=64),
    dict(topk_groups=0), dict(topk_groups=5), dict(renormalize=2), dict(logits_bf16=-1),
    dict(num_experts=8, num_topk=5), dict(route_scale=float("nan")),
])
def test_router_configs_rejected(ep, bad):
    c = router(ep, **bad)
    assert ep.ep_route_workspace_bytes(c, 1) == -1
    E = max(1, c.num_experts)
    assert ep.ep_route(c, 1, A, E, None, None, A, A, None) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_route_balance(c, 1, A, E, None, None, 1, None, A, A, A, A, A, A, A,
                               None) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_route_backward(c, 1, A, E, None, A, A, 1, None, None, None, None, A, E,
                                None) == ep.EP_ERR_INVALID_ARG


def test_router_arguments_rejected(ep):
    c = router(ep)
    good = [c, 2, A, 64, None, None, A, A, None]
    for at, v in ((1, -1), (1, (1 << 30) + 1), (2, None), (2, M), (3, 63), (4, A), (4, M), (5, M), (6, None), (6, M),
                  (7, None), (7, M)):
        a = list(good)
        a[at] = v
        assert ep.ep_route(*a) == ep.EP_ERR_INVALID_ARG, (at, v)
    good = [c, 2, A, 64, None, None, 2, A, A, A, A, A, A, A, A, None]
    for at, v in ((1, -1), (3, 60), (6, 0), (6, (1 << 20) + 1), (7, None), (7, M), (8, None),
                  (9, M), (10, None), (11, None), (12, M), (13, None), (14, None), (14, M)):
        a = list(good)
        a[at] = v
        assert ep.ep_route_balance(*a) == ep.EP_ERR_INVALID_ARG, (at, v)
    good = [c, 2, A, 64, None, A, A, 2, A, A, A, A, A, 64, None]
    for at, v in ((1, -1), (1, (1 << 30) + 1), (2, M), (3, 63), (4, M), (5, None), (6, M), (7, 0), (8, None),
                  (9, None), (10, None), (11, None), (11, M), (12, None), (13, 63)):
        a = list(good)
        a[at] = v
        assert ep.ep_route_backward(*a) == ep.EP_ERR_INVALID_ARG, (at, v)
    # no tokens: nothing to launch, nothing to check but the shapes
    assert ep.ep_route(c, 0, None, 64, None, None, None, None, None) == ep.EP_OK
    assert ep.ep_route_backward(c, 0, None, 64, None, None, None, 1, None, None, None, None, None,
                                64, None) == ep.EP_OK


def test_workspace_grows_with_sequences(ep):
    c = router(ep)
    sizes = [ep.ep_route_workspace_bytes(c, b) for b in (1, 2, 1000, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 16 == 0 for s in sizes)
    assert ep.ep_route_workspace_bytes(c, 0) == -1
    assert ep.ep_route_workspace_bytes(c, (1 << 20) + 1) == -1


def test_w4_sizes(ep):
    c = ep.EpW4Config(3, 160, 70, 32, 0, 0, 1)       # 2 tiles of 64 rows, 2 blocks of 128
    assert ep.ep_w4_codes_bytes(c) == 3 * 2 * 2 * 4096
    assert ep.ep_w4_scales_bytes(c) == 3 * 2 * 8 * 64 * 2
    assert ep.ep_w4_zeros_bytes(c) == 3 * 2 * 8 * 64
    c = ep.EpW4Config(3, 256, 70, 128, 1, 1, 0)      # 35 outputs: 2 tiles of 32
    assert ep.ep_w4_codes_bytes(c) == 3 * 2 * 2 * 4096
    assert ep.ep_w4_zeros_bytes(c) == 0


@pytest.mark.parametrize("bad", [
    (0, 128, 64, 128, 0, 0, 0), (2049, 128, 64, 128, 0, 0, 0), (1, 0, 64, 128, 0, 0, 0),
    (1, 100, 64, 32, 0, 0, 0), (1, 128, 0, 128, 0, 0, 0), (1, 128, 63, 128, 0, 1, 0),
    (1, 160, 64, 32, 1, 0, 0), (1, 128, 64, 48, 0, 0, 0), (1, 128, 64, 128, 2, 0, 0),
    (1, 128, 64, 128, 0, 2, 0), (1, 128, 64, 128, 0, 0, 2), (1, 2**20 + 128, 64, 128, 0, 0, 0),
    (1, 128, 2**20 + 1, 128, 0, 0, 0),
])
def test_w4_configs_rejected(ep, bad):
    c = ep.EpW4Config(*bad)
    assert ep.ep_w4_codes_bytes(c) == ep.ep_w4_scales_bytes(c) == ep.ep_w4_zeros_bytes(c) == -1
    assert ep.ep_w4_pack(c, A, A, None, A, A, None, None) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_expert_w4(c, 1, 1, A, None, A, A, None, A, A, A, None) == ep.EP_ERR_INVALID_ARG


def test_w4_arguments_rejected(ep):
    c = ep.EpW4Config(2, 128, 64, 64, 0, 0, 0)
    good = [c, 4, 4, A, None, A, A, None, A, A, A, None]
    for at, v in ((1, -1), (2, -1), (3, None), (3, M), (4, A), (5, None), (6, M), (7, A),
                  (8, None), (9, M), (10, None), (10, M)):
        a = list(good)
        a[at] = v
        assert ep.ep_expert_w4(*a) == ep.EP_ERR_INVALID_ARG, (at, v)
    assert ep.ep_expert_w4(c, 0, 0, None, None, A, A, None, A, A, None, None) == ep.EP_OK
    fp8z = ep.EpW4Config(2, 128, 64, 64, 1, 0, 1)
    good = [fp8z, 4, 4, A, A, A, A, A, A, A, A, None]
    for at, v in ((4, None), (4, M), (7, None), (7, M)):
        a = list(good)
        a[at] = v
        assert ep.ep_expert_w4(*a) == ep.EP_ERR_INVALID_ARG, (at, v)
    for a in ([c, A, A, A, A, A, None], [c, A, A, None, A, A, A], [c, None, A, None, A, A, None],
              [c, A, M, None, A, A, None], [fp8z, A, A, None, A, A, A],
              [fp8z, A, A, A, A, A, None]):
        assert ep.ep_w4_pack(*a, None) == ep.EP_ERR_INVALID_ARG


def test_reference_gradient_against_differences():
    """The plain gradient the GPU tests compare with, against differences of
    the plain objective."""
    rng = np.random.default_rng(0)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            T, E, K = 6, 9, 3
            l = rng.standard_normal((T, E))
            l[1, 4] = -np.inf
            mask, starts = np.array([1, 1, 0, 1, 1, 1], bool), np.array([0, 3, 3, 6])
            idx, _ = ref.route(l, K, score, None, 3, 2, renorm, 2.5, mask)
            count, *_ = ref.balance(l, idx, score, mask, starts)
            gl = np.array([0.7, 0.3 if score == "softmax" else 0.0])
            a = (idx, rng.standard_normal((T, K)), gl, score, renorm, 2.5, mask, starts, count)
            g, _ = ref.backward(l, *a)
            for t in range(T):
                for e in range(E):
                    if np.isinf(l[t, e]):
                        assert g[t, e] == 0
                        continue
                    d = np.zeros_like(l)
                    d[t, e] = 1e-5
                    slope = (ref.objective(l + d, *a) - ref.objective(l - d, *a)) / 2e-5
                    assert abs(slope - g[t, e]) < 1e-8


def test_compiled_calls_refuse_before_they_call(ep):
    """Tensors on the CPU, of the wrong kind or count: no kernel is reached."""
    import torch

    cfg = ep.RouterConfig(8, 2)
    x = torch.zeros((3, 8))
    w4 = ep.W4Config(1, 128, 64)
    codes, scales = torch.zeros((1, 1, 1, 8, 32, 4), dtype=torch.int32), torch.zeros((1, 1, 1, 64))
    seg = torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: ep.route(cfg, x), lambda: ep.route_balance(cfg, x),
        lambda: ep.route_backward(cfg, x),
        lambda: ep.expert_w4(w4, torch.zeros((1, 128), dtype=torch.bfloat16), codes,
                             scales.bfloat16(), seg, seg, 1),
    ]
    for call in bad:
        with pytest.raises(ep.EpError) as e:
            call()
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    assert ep._calls.route(cfg._at, "logits", None, None, None, None, None) == -1
    with pytest.raises(TypeError):
        ep._calls.route(cfg._at, x)
    with pytest.raises(TypeError):
        ep._calls.route("config", x, None, None, None, None, None)
    with pytest.raises(ep.EpError):
        ep.RouterConfig(8, 2, score="tanh")
