"""Tensors of two GPUs, or of another than the current one, are refused before
anything is launched.  The other GPU's tensors have a device and a shape but no
memory, so that one GPU is enough, or none."""

import pytest
import torch

f32, i32, i64, bf16, u8 = (torch.float32, torch.int32, torch.int64, torch.bfloat16, torch.uint8)


class Elsewhere(torch.Tensor):
    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


@pytest.fixture(scope="module")
def ep():
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


T, E, K, B = 8, 16, 2, 2
ARGS = {
    "route": dict(logits=((T, E), f32), bias=((E,), f32), token_mask=((T,), u8),
                  topk_idx=((T, K), i64), topk_weights=((T, K), f32)),
    "route_balance": dict(logits=((T, E), f32), bias=((E,), f32), token_mask=((T,), u8),
                          seq_start=((B + 1,), i32), topk_idx=((T, K), i64),
                          topk_weights=((T, K), f32), count=((B, E), i32), prob=((B, E), f32),
                          tokens=((B + 2,), i32), loss=((2,), f32), workspace=((1 << 20,), u8)),
    "route_backward": dict(logits=((T, E), f32), topk_idx=((T, K), i64), grad_w=((T, K), f32),
                           token_mask=((T,), u8), seq_start=((B + 1,), i32),
                           expert_count=((B, E), i32), seq_tokens=((B + 2,), i32),
                           grad_loss=((2,), f32), grad_logits=((T, E), f32)),
    "expert_w4": dict(x=((4, 128), u8), codes=((2, 1, 1, 8, 32, 4), i32),
                      scales=((2, 1, 1, 64), bf16), expert_start=((2,), i32),
                      expert_end=((2,), i32), zeros=((2, 1, 1, 64), u8), x_scale=((4, 1), f32),
                      out=((4, 64), bf16)),
    "w4_pack": dict(codes=((2, 64, 64), u8), scales=((2, 64, 1), bf16), zeros=((2, 64, 1), u8)),
}
CASES = [(name, arg) for name, args in ARGS.items() for arg in [None, *args]]


def call(ep, name, a):
    if name == "route_balance":
        out = tuple(a.pop(k) for k in ("topk_idx", "topk_weights", "count", "prob", "tokens",
                                       "loss"))
        return ep.route_balance(ep.RouterConfig(E, K, "sigmoid"), out=out, **a)
    if name in ("expert_w4", "w4_pack"):
        cfg = ep.W4Config(2, 128, 64, x_fp8=True, has_zeros=True)
        return getattr(ep, name)(cfg, **a, **({"num_rows": 0} if name == "expert_w4" else {}))
    return getattr(ep, name)(ep.RouterConfig(E, K, "sigmoid"), **a)


def refused(ep, name, a):
    with pytest.raises(ep.EpError) as e:
        call(ep, name, a)
    assert e.value.status == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ARGS)
def test_no_tensor_on_the_current_gpu(ep, name):
    refused(ep, name, {k: Elsewhere(s, t, "cuda:7") for k, (s, t) in ARGS[name].items()})


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg", CASES)
def test_one_tensor_on_another_gpu(ep, name, arg):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a = {k: torch.zeros(s, dtype=t, device="cuda") for k, (s, t) in ARGS[name].items()}
    if arg is None:
        call(ep, name, a)
        return
    a[arg] = Elsewhere(*ARGS[name][arg], "cuda:7")
    refused(ep, name, a)
    torch.cuda.synchronize()


def test_scratch_memory_is_not_made_for_another_gpu(ep):
    x, args = Elsewhere((T, E), f32, "cuda:7"), ARGS["route_balance"]
    out = tuple(Elsewhere(*args[k], "cuda:7")
                for k in ("topk_idx", "topk_weights", "count", "prob", "tokens", "loss"))
    with pytest.raises(ep.EpError):
        ep.route_balance(ep.RouterConfig(E, K), x,
                         seq_start=Elsewhere((B + 1,), i32, "cuda:7"), out=out)
