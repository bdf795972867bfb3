"""What the experts' products keep of their operands and sums.

Long reductions are of small whole numbers: their sums are exact in 32 bits, whatever the order, so
that the output is the exact sum's rounding, and a step left out or taken twice shows.  The bounds of
E4M3 operands are held to their definition (value * scale), by outputs in which the leading bits
cancel."""

import numpy as np
import pytest
import torch

import expert_ref as ref

HALF = 2.0 ** -8       # half a step of bf16, relative to the value


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def segments(counts, align=8):
    start, end = ref.segments(counts, align)
    return (torch.from_numpy(start).cuda(), torch.from_numpy(end).cuda(), int(sum(counts))), start


class Whole:
    """Operands of whole numbers, at most 2 in magnitude: with up to 2^20 of them in a sum, nothing
    reaches 2^24, and every partial sum is exact in fp32."""

    def __init__(self, ep, counts, H, N, fp8, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def new(*shape):
            return torch.randint(-2, 3, shape, device="cuda", generator=gen, dtype=torch.int8)

        self.counts, self.cfg = counts, ep.ExpertConfig(len(counts), H, N, x_fp8=fp8)
        self.seg, self.start = segments(counts)
        cap = max(1, int(self.start[-1]))
        x, w, dy = new(cap, H), new(len(counts), N, H), new(cap, N)
        self.w, self.dy, self.scale = w.bfloat16(), dy.bfloat16(), None
        self.x = x.bfloat16()
        self.wv, self.dyv, self.xv = w.double(), dy.double(), x.double()
        if fp8:
            # powers of two: -1, 0 or 1 as exponents of the blocks' scales
            power = torch.randint(-1, 2, (cap, H // 128), device="cuda", generator=gen)
            self.x = x.float().to(torch.float8_e4m3fn).view(torch.uint8)
            self.scale = torch.exp2(power.float())
            self.xv = self.xv * self.scale.double().repeat_interleave(128, 1)

    def rows(self, e):
        return slice(int(self.start[e]), int(self.start[e]) + self.counts[e])


LONG = [
    dict(counts=[3, 1], H=1 << 20, N=8), dict(counts=[5], H=1 << 20, N=264),
    dict(counts=[0, 5], H=128, N=1 << 20), dict(counts=[200000], H=128, N=16),
    dict(counts=[1 << 20], H=128, N=8), dict(counts=[70000, 0, 3], H=256, N=72),
    dict(counts=[1], H=7168, N=128), dict(counts=[3, 0, 1], H=2176, N=520),
    dict(counts=[0, 6500, 30], H=128, N=136), dict(counts=[5, 2], H=2048, N=4160),
    dict(counts=[40, 200], H=128, N=2120), dict(counts=[300, 700], H=8192, N=1104),
    dict(counts=[2048, 2049, 4097], H=640, N=1104), dict(counts=[16400], H=128, N=2800),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("c", LONG, ids=str)
def test_long_reductions_are_exact(ep, c, fp8):
    k = Whole(ep, fp8=fp8, **c)
    out = ep.expert_mm(k.cfg, k.x, k.w, *k.seg, x_scale=k.scale)
    kw = dict(w=k.w, x=k.x, x_scale=k.scale)
    grad_x, grad_w = ep.expert_mm_backward(k.cfg, k.dy, *k.seg, **kw)
    del kw["w"]
    _, grad_32 = ep.expert_mm_backward(k.cfg, k.dy, *k.seg, grad_w_dtype=torch.float32, **kw)
    added = torch.arange(-3, 4, device="cuda").float().repeat(grad_32.numel() // 7 + 1)
    added = added[:grad_32.numel()].view(grad_32.shape).contiguous()
    before = added.double()
    ep.expert_mm_backward(k.cfg, k.dy, *k.seg, grad_w=added, accumulate=True, **kw)
    for e in range(len(k.counts)):
        r = k.rows(e)
        y, dx, dw = k.xv[r] @ k.wv[e].T, k.dyv[r] @ k.wv[e], k.dyv[r].T @ k.xv[r]
        assert max([0.0] + [float(t.abs().max()) for t in (y, dx, dw) if t.numel()]) < 2 ** 21
        # (fp32 holds them: one rounding to bf16)
        assert torch.equal(out[r], y.float().bfloat16())
        assert torch.equal(grad_x[r], dx.float().bfloat16())
        assert torch.equal(grad_w[e], dw.float().bfloat16())
        assert torch.equal(grad_32[e], dw.float())
        assert torch.equal(added[e], (dw + before[e]).float())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1 << 14, 1 << 17, 1 << 20])
def test_sums_of_one_sign(ep, n):
    """Of positive terms the tensor cores drop, with each 16 of them, up to a last bit of the sum so
    far, which is half the whole on average: n / 16 * 2^-24 of the whole at most, beside the last
    rounding.  An fp32 gradient adds sums of 2048 rows."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    new = lambda *s: torch.rand(s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    loss = n / 16 * 2.0 ** -24
    seg, _ = segments([4])
    x, w = new(8, n), new(1, 8, n)
    y = ep.expert_mm(ep.ExpertConfig(1, n, 8), x, w, *seg)[:4].double()
    want = x[:4].double() @ w[0].double().T
    assert ((y - want).abs() <= (loss + HALF) * want).all()
    cfg = ep.ExpertConfig(1, 8, n)
    dx, _ = ep.expert_mm_backward(cfg, x, *seg, w=w.view(1, n, 8))
    want = x[:4].double() @ w.view(n, 8).double()
    assert ((dx[:4].double() - want).abs() <= (loss + HALF) * want).all()
    seg, _ = segments([n])
    x, dy = new(n, 8), new(n, 8)
    cfg, want = ep.ExpertConfig(1, 8, 8), dy.double().T @ x.double()
    _, dw = ep.expert_mm_backward(cfg, dy, *seg, x=x)
    assert ((dw[0].double() - want).abs() <= (loss + HALF) * want).all()
    _, dw = ep.expert_mm_backward(cfg, dy, *seg, x=x, grad_w_dtype=torch.float32)
    # 128 losses in each sum, and a rounding for each sum that is added
    loss = 128 * 2.0 ** -24 + n / 2048 * 2.0 ** -24
    assert ((dw[0].double() - want).abs() <= loss * want).all()


def bf16_of(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).float().numpy()


def two_parts(value, scale):
    """value * scale as the forward product takes it: the scale's nearest number of four bits and
    what is left, each times the value, in bf16."""
    first = ((scale.view(np.uint32) + np.uint32(0x80000)) & np.uint32(0xFFF00000)).view(np.float32)
    rest = bf16_of(scale - first)
    a, b = bf16_of(first * value), bf16_of(rest * value)
    return a.astype(np.float64) + b


PARTS = 1.4 * 2.0 ** -12


def test_two_parts_of_every_scale():
    """All mantissas of a scale by all of E4M3: within 1.4 * 2^-12 of the product (and not within
    2^-12: the rest of the scale is rounded, and then its product)."""
    scale = (np.arange(0, 1 << 23, dtype=np.uint32) | np.uint32(0x3F800000)).view(np.float32)
    most = 0.0
    for m in range(8, 16):
        value = np.float32(m / 8)
        v = scale.astype(np.float64) * value
        most = max(most, float((abs(two_parts(value, scale) - v) / v).max()))
    assert 1.25 * 2.0 ** -12 < most < PARTS


def rows_of_one_value(n, gen, exponents=(-20, 20)):
    """E4M3 rows [n, 256]: a finite value in column 0 with a scale of any mantissa, 1 in column 128."""
    codes = torch.randint(1, 127, (n,), generator=gen, dtype=torch.uint8)
    codes |= torch.randint(0, 2, (n,), generator=gen, dtype=torch.uint8) << 7
    q = torch.zeros(n, 256, dtype=torch.uint8)
    q[:, 0], q[:, 128] = codes, torch.ones(()).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.ones(n, 2)
    power = torch.randint(exponents[0], exponents[1], (n,), generator=gen)
    scale[:, 0] = (1 + torch.rand(n, generator=gen)) * torch.exp2(power.float())
    return q, scale


@pytest.mark.gpu
def test_bits_of_rows_in_8_bits_forward(ep):
    """Output n of row n is the row's value less its bf16: what the operand keeps beyond 8 bits."""
    n = 2048
    q, scale = rows_of_one_value(n, torch.Generator().manual_seed(1))
    scale[0, 0], q[0, 0] = 0.0330238, torch.tensor(1.125).to(torch.float8_e4m3fn).view(torch.uint8)
    v = q[:, 0].view(torch.float8_e4m3fn).double() * scale[:, 0].double()
    near = v.float().bfloat16()
    w = torch.zeros(1, n, 256, dtype=torch.bfloat16)
    w[0, :, 0], w[0, :, 128] = 1, -near
    seg, _ = segments([n])
    y = ep.expert_mm(ep.ExpertConfig(1, 256, n, x_fp8=True), q.cuda(), w.cuda(), *seg,
                     x_scale=scale.cuda())
    got, want = y.diagonal().double().cpu(), v - near.double()
    # the sums' own roundings: a few 2^-23 of the terms
    assert ((got - want).abs() <= (PARTS + 2.0 ** -20) * v.abs() + HALF * want.abs()).all()
    assert ((got - want).abs() > 2.0 ** -15 * v.abs()).any()      # (parts, not the whole scale)


@pytest.mark.gpu
def test_bits_of_rows_in_8_bits_in_a_gradient(ep):
    """Of one row and a gradient of 1: an fp32 gradient holds value * scale to 17 bits, a bf16 one
    its nearest bf16, rounded once."""
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(2)
    q[(q & 0x7F) == 0x7F] = 0
    q = q[None].repeat(40, 1).contiguous()
    gen = torch.Generator().manual_seed(2)
    scale = (1 + torch.rand(40, 4, generator=gen)) * torch.exp2(
        torch.randint(-30, 30, (40, 4), generator=gen).float())
    v = ref.values(q, scale)
    start = torch.arange(40, dtype=torch.int32).cuda()
    seg = start, start + 1, 40
    dy = torch.ones(40, 8, dtype=torch.bfloat16).cuda()
    cfg = ep.ExpertConfig(40, 512, 8, x_fp8=True)
    kw = dict(x=q.cuda(), x_scale=scale.cuda())
    _, g32 = ep.expert_mm_backward(cfg, dy, *seg, grad_w_dtype=torch.float32, **kw)
    _, g16 = ep.expert_mm_backward(cfg, dy, *seg, **kw)
    for j in range(8):
        d = (g32[:, j].cpu().double() - v.double()).abs()
        assert (d <= 2.0 ** -17 * v.double().abs()).all()
        assert torch.equal(g16[:, j].cpu(), v.bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("counts,H,N", [([700, 300], 512, 264), ([40] * 30, 256, 136)])
def test_a_bf16_gradient_of_rows_in_8_bits(ep, counts, H, N):
    """Against sums of value * scale itself.  Rounding an operand is off by at most 2^-8 of it, evenly
    spread: by 2^-8 / sqrt(3) in the root of the mean square, and so are sums over rows of such errors
    with factors of either sign, in the norm; the last rounding once more.  An fp32 gradient of the
    same rows is 17 bits near."""
    gen = torch.Generator().manual_seed(3)
    seg, start = segments(counts)
    cap = int(start[-1])
    q, scale = ref.quantise(torch.randn(cap, H, generator=gen))
    dy = torch.randn(cap, N, generator=gen).bfloat16()
    v = ref.values(q, scale).double()
    cfg, kw = ep.ExpertConfig(len(counts), H, N, x_fp8=True), dict(x=q.cuda(), x_scale=scale.cuda())
    _, g16 = ep.expert_mm_backward(cfg, dy.cuda(), *seg, **kw)
    _, g32 = ep.expert_mm_backward(cfg, dy.cuda(), *seg, grad_w_dtype=torch.float32, **kw)
    for e, n in enumerate(counts):
        r = slice(int(start[e]), int(start[e]) + n)
        want = dy[r].double().T @ v[r]
        off = float((g16[e].cpu().double() - want).norm() / want.norm())
        assert off < HALF * (2 / 3) ** 0.5
        off = float((g32[e].cpu().double() - want).norm() / want.norm())
        assert off < 2.0 ** -17 + (n / 16 + 2) * ref.EPS


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-40, -80, -104, -118, -140])
def test_small_scales(ep, power):
    """Weights as large as the scales are small, so that results are of the size of 1: a part of an
    operand keeps its bits down to 2^-133, the smallest bf16 (half a step of it: 2^-134)."""
    gen = torch.Generator().manual_seed(4)
    counts, H, N = [30, 0, 7], 256, 72
    seg, start = segments(counts)
    q, scale = ref.quantise(torch.randn(int(start[-1]), H, generator=gen) * 3)
    scale = torch.ldexp(scale, torch.tensor(power))
    w = torch.ldexp(torch.randn(3, N, H, generator=gen), torch.tensor(min(-power, 110))).bfloat16()
    out = ep.expert_mm(ep.ExpertConfig(3, H, N, x_fp8=True), q.cuda(), w.cuda(), *seg,
                       x_scale=scale.cuda())
    x = q.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128, 1)
    for e, n in enumerate(counts):
        r = slice(int(start[e]), int(start[e]) + n)
        y = x[r] @ w[e].double().T
        terms, sizes = x[r].abs() @ w[e].double().abs().T, w[e].double().abs().sum(1)
        # a scale under 2^-126 has no four bits of its own: it is the second part, of 8 bits
        parts = PARTS if power > -118 else 2 * HALF
        off = (parts + 2.0 ** -18) * terms + 2 * 2.0 ** -134 * sizes + HALF * y.abs()
        assert ((out[r].cpu().double() - y).abs() <= off * (1 + HALF)).all()
        if power > -110 and n:
            assert float(y.abs().median()) > 8 * float(off.median())
