"""Host-side checks of the experts' bf16 products and of the gated activation that need no GPU:
struct layouts, argument validation, refusals of the torch layer, streams of the outputs; and the
plain gradients that the GPU tests compare with, against differences.  No call here reaches a
kernel."""

import copy
import ctypes
import pickle
import types

import numpy as np
import pytest
import torch

import expert_ref as ref
from test_layer_devices import Elsewhere
from test_layer_streams import Fake, Streams

A = 0x10000   # an aligned address
M = 0x10008   # a misaligned one


@pytest.fixture(scope="module")
def ep():
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def test_struct_layout(ep):
    assert ctypes.sizeof(ep.EpExpertConfig) == 20


BAD = [
    (0, 64, 64, 0, 0), (2049, 64, 64, 0, 0), (1, 0, 64, 0, 0), (1, 60, 64, 0, 0), (1, 64, 0, 0, 0),
    (1, 64, 4, 0, 0), (1, 64, 68, 0, 0), (1, 64, 64, 1, 0), (1, 64, 48, 0, 1), (1, 64, 64, 2, 0),
    (1, 64, 64, 0, 2), (1, 2**20 + 8, 64, 0, 0), (1, 64, 2**20 + 8, 0, 0), (1, 2**20, 2**18, 0, 0),
    (1, -64, 64, 0, 0),
]


@pytest.mark.parametrize("bad", BAD)
def test_configs_rejected(ep, bad):
    c = ep.EpExpertConfig(*bad)
    assert ep.ep_expert_mm(c, 1, 1, A, None, A, A, A, A, None, None) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_expert_mm_backward(c, 1, 1, A, A, A, None, A, A, A, A, 0, None,
                                    None) == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ep.EpError) as e:
        ep.ExpertConfig(*bad[:3], x_fp8=bad[3], gated=bad[4])
    assert e.value.status == ep.EP_ERR_INVALID_ARG


def test_edges_accepted(ep):
    for ok in ((1, 8, 8, 0, 0), (2048, 2**20, 8, 0, 0), (1, 128, 32, 1, 1), (1, 2**19, 2**18, 0, 0)):
        c = ep.EpExpertConfig(*ok)
        assert ep.ep_expert_mm(c, 0, 0, None, None, A, A, A, None, None, None) == ep.EP_OK
    with pytest.raises(ep.EpError):
        ep.ExpertConfig(2**32 + 1, 64, 64)


def vary(f, ep, good, bad):
    for at, v in bad:
        a = list(good)
        a[at] = v
        assert f(*a) == ep.EP_ERR_INVALID_ARG, (at, v)


def test_product_arguments_rejected(ep):
    c, q = ep.EpExpertConfig(2, 128, 64, 0, 0), ep.EpExpertConfig(2, 128, 64, 1, 0)
    vary(ep.ep_expert_mm, ep, [c, 4, 4, A, None, A, A, A, A, None, None],
         [(0, None), (1, -1), (2, -1), (3, None), (3, M), (4, A), (5, None), (5, M), (6, None),
          (6, M), (7, None), (7, M), (8, None), (8, M), (9, M)])
    vary(ep.ep_expert_mm, ep, [q, 4, 4, A, A, A, A, A, A, None, None], [(4, None), (4, M)])
    vary(ep.ep_selftest_expert_timeout, ep, [c, 4, 4, A, None, A, A, A, A, A, None],
         [(0, None), (1, 0), (2, 0)] + [(i, v) for i in (3, 5, 6, 7, 8, 9) for v in (None, M)]
         + [(4, A)])
    assert ep.ep_expert_mm(c, 0, 5, None, None, A, A, A, None, None, None) == ep.EP_OK
    assert ep.ep_expert_mm(c, 5, 0, A, None, A, A, A, A, None, None) == ep.EP_OK


def test_gradient_arguments_rejected(ep):
    c, q = ep.EpExpertConfig(2, 128, 64, 0, 0), ep.EpExpertConfig(2, 128, 64, 1, 0)
    g = ep.EpExpertConfig(2, 128, 64, 0, 1)
    good = [c, 4, 4, A, A, A, None, A, A, A, A, 0, None, None]
    vary(ep.ep_expert_mm_backward, ep, good,
         [(0, None), (0, g), (1, -1), (2, -1), (3, None), (3, M), (4, None), (4, M), (5, None),
          (5, M), (6, A), (7, None), (7, M), (8, None), (8, M), (9, M), (10, M), (11, -1), (11, 3),
          (12, M)])
    vary(ep.ep_expert_mm_backward, ep, [q, 4, 4, A, A, A, A, A, A, A, A, 1, None, None],
         [(6, None), (6, M)])
    vary(ep.ep_expert_mm_backward, ep, [c, 4, 4, A, A, A, None, A, A, None, A, 0, None, None],
         [(10, None)])
    # nothing to compute and nothing to clear
    assert ep.ep_expert_mm_backward(c, 0, 0, None, A, None, None, A, A, A, None, 0, None,
                                    None) == ep.EP_OK
    assert ep.ep_expert_mm_backward(c, 0, 0, None, None, None, None, A, A, None, A, 2, None,
                                    None) == ep.EP_OK


def test_activation_arguments_rejected(ep):
    vary(ep.ep_act_save, ep, [2, 64, 4, 4, A, A, A, A, A, A, None],
         [(0, 0), (0, 2049), (1, 0), (1, 60), (1, 2**19 + 8), (2, -1), (3, -1)]
         + [(i, v) for i in range(4, 10) for v in (None, M)])
    vary(ep.ep_act_backward, ep, [2, 64, 4, 4, A, A, A, A, A, A, A, None],
         [(0, 0), (0, 2049), (1, 0), (1, 60), (1, 2**19 + 8), (2, -1), (3, -1), (10, M)]
         + [(i, v) for i in range(4, 10) for v in (None, M)])
    assert ep.ep_act_save(2, 64, 0, 4, None, A, A, None, None, None, None) == ep.EP_OK
    assert ep.ep_act_backward(2, 64, 4, 0, A, A, A, A, A, A, None, None) == ep.EP_OK


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_a_copied_config_has_its_own_struct(ep, how):
    c = ep.ExpertConfig(60, 256, 64, True, True)
    d = how(c)
    assert d == c and hash(d) == hash(c) and d.out_width == 32
    assert d._at == ctypes.addressof(d._c) != c._at
    assert ctypes.string_at(d._at, 20) == bytes(c.c())


f32, i32, bf16, u8 = torch.float32, torch.int32, torch.bfloat16, torch.uint8
SEG = dict(expert_start=((3,), i32), expert_end=((2,), i32))
ARGS = {
    "expert_mm": dict(x=((4, 128), u8), w=((2, 64, 128), bf16), x_scale=((4, 1), f32),
                      out=((4, 64), bf16), err=((4,), i32), **SEG),
    "expert_mm_backward": dict(grad_out=((4, 64), bf16), w=((2, 64, 128), bf16),
                               x=((4, 128), u8), x_scale=((4, 1), f32), grad_x=((4, 128), bf16),
                               grad_w=((2, 64, 128), f32), err=((4,), i32), **SEG),
    "act_save": dict(h=((4, 128), bf16), a=((4, 64), bf16), h_q=((4, 128), u8),
                     h_scale=((4, 2), f32), **SEG),
    "act_backward": dict(grad_a=((4, 64), bf16), h_q=((4, 128), u8), h_scale=((4, 2), f32),
                         grad_h=((4, 128), bf16), a=((4, 64), bf16), **SEG),
}
CASES = [(n, a) for n, args in ARGS.items() for a in [None, *args]]


def call(ep, name, a):
    cfg = (ep.ExpertConfig(2, 128, 64, x_fp8=True),) if name.startswith("expert") else ()
    return getattr(ep, name)(*cfg, **a, num_rows=0)


def refused(ep, name, a):
    with pytest.raises(ep.EpError) as e:
        call(ep, name, a)
    assert e.value.status == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ARGS)
def test_tensors_of_no_gpu_or_another(ep, name):
    refused(ep, name, {k: torch.zeros(s, dtype=t) for k, (s, t) in ARGS[name].items()})
    refused(ep, name, {k: Elsewhere(s, t, "cuda:7") for k, (s, t) in ARGS[name].items()})


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg", CASES)
def test_one_tensor_that_does_not_fit(ep, name, arg):
    """Of another GPU, another type, one element more, or strided."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    good = {k: torch.zeros(s, dtype=t, device="cuda") for k, (s, t) in ARGS[name].items()}
    if arg is None:
        call(ep, name, good)
        return
    shape, dtype = ARGS[name][arg]
    bad = [Elsewhere(shape, dtype, "cuda:7"),
           torch.zeros(shape, dtype=torch.float16, device="cuda"), "no tensor"]
    if arg not in SEG and arg != "err":
        bad += [torch.zeros(shape[:-1] + (shape[-1] + 8,), dtype=dtype, device="cuda"),
                torch.zeros((2,) + shape[::-1], dtype=dtype, device="cuda")[0].T
                if len(shape) == 2 and shape[1] > 1 else torch.zeros(3, dtype=dtype, device="cuda")]
    for t in bad:
        if t == "no tensor" and arg in ("x", "grad_out", "h", "grad_a"):
            continue      # their shape is asked for first
        refused(ep, name, dict(good, **{arg: t}))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_gradients_that_do_not_belong_together(ep):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    good = {k: torch.zeros(s, dtype=t, device="cuda") for k, (s, t) in ARGS["expert_mm_backward"].items()}
    for change in (dict(w=None), dict(x=None), dict(w=None, x=None, grad_x=None, grad_w=None),
                   dict(grad_w=good["grad_w"].bfloat16(), accumulate=True),
                   dict(x=None, grad_w=None, accumulate=True), dict(x_scale=None),
                   dict(grad_w=None, accumulate=True),
                   dict(grad_w=None, grad_w_dtype=torch.float16)):
        refused(ep, "expert_mm_backward", dict(good, **change))
    bf = ep.ExpertConfig(2, 128, 64)
    with pytest.raises(ep.EpError):      # scales of rows that have none
        ep.expert_mm(bf, torch.zeros((4, 128), dtype=bf16, device="cuda"), good["w"],
                     good["expert_start"], good["expert_end"], 4, x_scale=good["x_scale"])
    for rows in (-1, 2**31, -2**40):
        with pytest.raises(ep.EpError):
            ep.act_save(torch.zeros((4, 128), dtype=bf16, device="cuda"), good["expert_start"],
                        good["expert_end"], rows)


@pytest.mark.parametrize("name", ["expert_mm", "expert_mm_backward", "act_save", "act_backward"])
def test_outputs_are_made_for_the_stream_that_writes_them(ep, monkeypatch, name):
    streams, recorded = Streams(monkeypatch), []
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.append((t, s.cuda_stream)), raising=False)
    monkeypatch.setattr(ep, "_calls", types.SimpleNamespace(
        **{n: lambda *a: 0 for n in ("expert_mm", "expert_mm_backward", "act_save",
                                     "act_backward")}))
    cfg = ep.ExpertConfig(2, 128, 64)
    rows, wide, w = Fake((4, 128), bf16), Fake((4, 64), bf16), Fake((2, 64, 128), bf16)
    many, run = {
        "expert_mm": (1, lambda s: (ep.expert_mm(cfg, rows, w, None, None, 4, stream=s),)),
        "expert_mm_backward": (2, lambda s: ep.expert_mm_backward(cfg, wide, None, None, 4, w=w,
                                                                 x=rows, stream=s)),
        "act_save": (3, lambda s: ep.act_save(rows, None, None, 4, stream=s)),
        "act_backward": (2, lambda s: ep.act_backward(wide, rows, rows, None, None, 4, stream=s)),
    }[name]
    for stream, made_on in ((streams.stream(2), 2), (streams.stream(1), 1), (None, 1)):
        streams.made.clear()
        recorded.clear()
        out = run(stream)
        assert len(out) == many and [s for s, _, _ in streams.made] == [made_on] * many
        assert all(any(t is o for _, _, t in streams.made) for o in out)
        assert len(recorded) == (many if made_on == 2 else 0) and all(s == 1 for _, s in recorded)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w, dy = (rng.standard_normal(s) for s in ((5, 6), (4, 6), (5, 4)))
    value = lambda x, w: (x @ w.T * dy).sum()  # noqa: E731
    for got, at in ((ref.by_rows(dy, w)[0], 0), (ref.by_weights(dy, x, True)[0], 1)):
        for i in np.ndindex(got.shape):
            hi, lo = [x.copy(), w.copy()], [x.copy(), w.copy()]
            hi[at][i] += 1e-5
            lo[at][i] -= 1e-5
            assert abs((value(*hi) - value(*lo)) / 2e-5 - got[i]) < 1e-8
    h, da = 3 * rng.standard_normal((3, 8)), rng.standard_normal((3, 4))
    got = ref.activation_backward(da, h)[0]
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = 1e-5
        slope = ((ref.activation(h + d)[0] - ref.activation(h - d)[0]) * da).sum() / 2e-5
        assert abs(slope - got[i]) < 1e-8
