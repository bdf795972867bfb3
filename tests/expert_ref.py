"""Plain 64-bit forms of the experts' products and of the gated activation with its 8-bit
checkpoint, expert by expert from the definitions in include/ep.h, with bounds of the errors that
fp32 sums and one rounding may make."""

import numpy as np
import torch

EPS = 2.0 ** -24      # one fp32 rounding
BF16 = 2.0 ** -8      # one bf16 rounding


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def segments(counts, align):
    """(start [E + 1], end [E]) of rows laid out by expert."""
    start = np.concatenate([[0], np.cumsum([-(-c // align) * align for c in counts])])
    return start.astype(np.int32), (start[:-1] + np.array(counts)).astype(np.int32)


def values(q, scale):
    """What E4M3 bits and a scale for each 128 columns stand for, in fp32 as the library forms
    them."""
    f = q.view(torch.float8_e4m3fn).float()
    return f * scale.repeat_interleave(128, 1)[:, : f.shape[1]]


def quantise(x):
    """(E4M3 bits, scales) of fp32 rows [n, cols]: IEEE quotients, nearest even."""
    n, cols = x.shape
    blocks = -(-cols // 128)
    b = torch.zeros(n, blocks * 128)
    b[:, :cols] = x
    b = b.view(n, blocks, 128)
    scale = b.abs().amax(2) / 448.0
    q = torch.where(scale[:, :, None] == 0, 0.0, b / scale[:, :, None])
    q = q.reshape(n, -1)[:, :cols].clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).contiguous(), scale


def product(x, w):
    """(x w^T, a bound of its error before the last rounding): the tensor cores add 16 products
    and the sum so far at a time, each a rounding of two bits fewer than fp32's."""
    y = x @ w.T
    return y, 4 * EPS * (x.shape[1] / 16 + 8) * (abs(x) @ abs(w).T)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def forward(x, w, gated, fp8=False):
    """(y, bound) of one expert's rows, the last rounding to bf16 included.  E4M3 rows enter in
    two bf16 parts whose sum is off by up to 2^-12 of the value: the second, at most 2^-4 of
    it, is rounded twice to 8 bits (of the scale's rest, and of the product)."""
    y, d = product(x, w)
    if fp8:
        d = 2 * d + EPS * abs(y) + 2.0 ** -12 * (abs(x) @ abs(w).T)
    if gated:
        half = w.shape[0] // 2
        (g, u), (dg, du) = (y[:, :half], y[:, half:]), (d[:, :half], d[:, half:])
        a = silu(g)
        y = a * u
        # |silu'| <= 1.1; expf, the sum, the quotient and the product round too
        d = 1.1 * dg * (abs(u) + du) + abs(a) * du + 16 * EPS * (1 + abs(g)) * abs(y)
    return y, d * (1 + BF16) + BF16 * abs(y) + 1e-38


def by_rows(dy, w):
    y, d = product(dy, np.ascontiguousarray(w.T))
    return y, d * (1 + BF16) + BF16 * abs(y) + 1e-38


def by_weights(dy, x, f32, fp8=False):
    """fp8 with f32: x enters in two bf16 parts, the nearest and the rest: off
    by half a step of the second, 2^-17."""
    y, d = product(np.ascontiguousarray(dy.T), np.ascontiguousarray(x.T))
    if fp8 and f32:
        d = 2 * d + EPS * abs(y) + BF16 * BF16 / 2 * (abs(dy).T @ abs(x))
    last = EPS if f32 else BF16
    return y, d * (1 + last) + last * abs(y) + 1e-38


def activation(h):
    """(a, bound) of [g, u]."""
    half = h.shape[1] // 2
    g, u = h[:, :half], h[:, half:]
    a = silu(g) * u
    return a, 16 * EPS * (1 + abs(g)) * abs(a) + BF16 * abs(a) + 1e-38


def activation_backward(da, h):
    """(grad_h, bound) at h = [g, u]."""
    half = h.shape[1] // 2
    g, u = h[:, :half], h[:, half:]
    with np.errstate(over="ignore"):
        c = 1 / (1 + np.exp(-g))
    dg, du = da * u * c * (1 + g * (1 - c)), da * g * c
    # 1 - c and the sum cancel: their errors are of the terms, not of the result
    eg = 16 * EPS * (2 + abs(g)) * abs(da * u * c)
    eu = 16 * EPS * (1 + abs(g)) * abs(du)
    y, e = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    return y, e * (1 + BF16) + BF16 * abs(y) + 1e-38
