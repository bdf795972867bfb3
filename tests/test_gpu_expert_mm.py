"""The experts' products with bf16 weights and their gradients on the GPU against plain 64-bit
forms (expert_ref.py)."""

import numpy as np
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu

MARK = 77.0      # what rows of no expert hold before and after


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


class Case:
    """Weights and rows of E experts with `counts` rows each, aligned to A; rows of no expert are
    NaN."""

    def __init__(self, ep, counts, H, N, fp8=False, gated=False, A=1, extra=0, seed=0):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.cfg = ep.ExpertConfig(E, H, N, fp8, gated)
        self.counts, self.gated, self.H, self.N = counts, gated, H, N
        self.start, self.end = ref.segments(counts, A)
        self.cap = max(1, int(self.start[-1])) + extra
        self.own = np.zeros(self.cap, bool)
        for s, e in zip(self.start, self.end):
            self.own[s:e] = True
        self.w = ref.bf16(rng.standard_normal((E, N, H)) / H ** 0.5)
        x = rng.standard_normal((self.cap, H)).astype(np.float32)
        if fp8:
            q, self.scale = ref.quantise(torch.from_numpy(x) * 3)
            q[~torch.from_numpy(self.own)] = 0x7F      # NaN
            v = ref.values(q, self.scale)
            self.xf, self.x = ref.f64(v), ref.f64(v.bfloat16())
            self.dx, self.dscale = q.cuda(), self.scale.cuda()
        else:
            x[~self.own] = np.nan
            t = ref.bf16(x)
            self.x, self.dx, self.dscale = ref.f64(t), t.cuda(), None
            self.xf = self.x
        dy = rng.standard_normal((self.cap, N)).astype(np.float32)
        dy[~self.own] = np.nan
        self.dy = ref.bf16(dy)
        self.dw, self.ddy = self.w.cuda(), self.dy.cuda()
        self.dstart = torch.from_numpy(self.start).cuda()
        self.dend = torch.from_numpy(self.end).cuda()
        self.rows = int(sum(counts))

    def out(self, width):
        return torch.full((self.cap, width), MARK, dtype=torch.bfloat16, device="cuda")

    def forward(self, ep, num_rows=None, **kw):
        kw.setdefault("out", self.out(self.cfg.out_width))
        return ep.expert_mm(self.cfg, self.dx, self.dw, self.dstart, self.dend,
                            self.rows if num_rows is None else num_rows, x_scale=self.dscale, **kw)

    def backward(self, ep, **kw):
        kw.setdefault("grad_x", self.out(self.H))
        return ep.expert_mm_backward(self.cfg, self.ddy, self.dstart, self.dend, self.rows,
                                     w=self.dw, x=self.dx, x_scale=self.dscale, **kw)

    def check_rows(self, got, form):
        got = ref.f64(got)
        assert (got[~self.own] == MARK).all()
        for e, n in enumerate(self.counts):
            if n:
                rows = slice(int(self.start[e]), int(self.end[e]))
                y, err = form(e, rows)
                assert (abs(got[rows] - y) <= err).all(), (e, abs(got[rows] - y).max())

    def check_forward(self, got):
        self.check_rows(got, lambda e, r: ref.forward(self.xf[r], ref.f64(self.w[e]), self.gated,
                                                       self.dscale is not None))

    def check_backward(self, grad_x, grad_w, before=None):
        self.check_rows(grad_x, lambda e, r: ref.by_rows(ref.f64(self.dy[r]), ref.f64(self.w[e])))
        f32 = grad_w.dtype == torch.float32
        got = ref.f64(grad_w)
        for e, n in enumerate(self.counts):
            rows = slice(int(self.start[e]), int(self.end[e]))
            y, err = ref.by_weights(ref.f64(self.dy[rows]), (self.xf if f32 else self.x)[rows], f32,
                                    self.dscale is not None)
            if before is not None:
                was = ref.f64(before[e])
                y, err = y + was, err + ref.EPS * (abs(y) + abs(was))
            assert (abs(got[e] - y) <= (err if n or before is not None else 0)).all(), e


def name_of(c):
    return str(c) if len(str(c)) < 99 else str(dict(c, counts=len(c["counts"])))


CASES = [
    dict(counts=[1], H=8, N=8), dict(counts=[1], H=64, N=128), dict(counts=[1], H=72, N=136),
    dict(counts=[3], H=96, N=72), dict(counts=[16], H=128, N=256), dict(counts=[17], H=1408, N=1000),
    dict(counts=[1, 0, 2, 0, 0, 7, 8, 9], H=384, N=96, A=8), dict(counts=[0, 0, 5], H=160, N=64),
    dict(counts=[0, 0], H=64, N=64), dict(counts=[255, 256, 257], H=136, N=264, A=16),
    dict(counts=[64, 63, 65, 128, 127, 129], H=264, N=136), dict(counts=[513], H=256, N=128, A=128),
    dict(counts=[2300, 5], H=128, N=264, A=128), dict(counts=[1] * 70, H=128, N=64),
    dict(counts=[0, 1] * 40 + [3], H=64, N=136), dict(counts=[1, 4500], H=72, N=72),
    dict(counts=[1], H=7168, N=128), dict(counts=[40, 300], H=520, N=2056),
    dict(counts=[5, 0, 33], H=128, N=64, A=128, extra=300),
    dict(counts=[1] * 33, H=64, N=8), dict(counts=[2] * 97, H=72, N=16, A=4),
    dict(counts=[3, 1], H=1 << 20, N=8), dict(counts=[0, 5], H=8, N=1 << 20),
    dict(counts=[0, 1, 0, 2] * 512, H=8, N=16),
]


@pytest.mark.parametrize("c", CASES, ids=name_of)
def test_forward(ep, c):
    case = Case(ep, **c)
    case.check_forward(case.forward(ep))


@pytest.mark.parametrize("c", CASES, ids=name_of)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward(ep, c, dtype):
    case = Case(ep, **c)
    case.check_backward(*case.backward(ep, grad_w_dtype=dtype))


FP8 = [
    dict(counts=[1], H=128, N=8), dict(counts=[33, 0, 2, 16], H=256, N=192, A=8),
    dict(counts=[255, 257, 1], H=384, N=136), dict(counts=[600], H=640, N=264, A=128),
    dict(counts=[1] * 40, H=128, N=64, A=128), dict(counts=[3, 70], H=1408, N=136),
]


@pytest.mark.parametrize("c", FP8, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_in_8_bits(ep, c, dtype):
    case = Case(ep, fp8=True, **c)
    case.check_forward(case.forward(ep))
    case.check_backward(*case.backward(ep, grad_w_dtype=dtype))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("c", [
    dict(counts=[1], H=128, N=32), dict(counts=[17, 1, 40], H=512, N=192, A=16),
    dict(counts=[0, 0, 5], H=128, N=96), dict(counts=[300, 256], H=256, N=288, A=8),
    dict(counts=[1] * 66, H=128, N=64), dict(counts=[2, 0, 9], H=1152, N=1056)], ids=str)
def test_gated(ep, c, fp8):
    case = Case(ep, fp8=fp8, gated=True, **c)
    case.check_forward(case.forward(ep))


def test_gated_rows_of_odd_width(ep):
    case = Case(ep, [9, 20], 72, 160, gated=True)
    case.check_forward(case.forward(ep))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[5, 0, 300], [0, 0]])
def test_gradient_added_to_what_is_there(ep, counts, fp8):
    H = 384 if fp8 else 136
    case = Case(ep, counts, H, 72, fp8=fp8)
    before = torch.randn(len(counts), 72, H, device="cuda")
    before[:, 0, :2] = torch.tensor([-0.0, 1e-40], device="cuda")
    grad_w = before.clone()
    grad_x, got = case.backward(ep, grad_w=grad_w, accumulate=True)
    assert got is grad_w
    for e, n in enumerate(counts):
        if n == 0:
            assert torch.equal(got[e].view(torch.int32), before[e].view(torch.int32))
    case.check_backward(grad_x, grad_w, before)


def test_one_gradient_alone(ep):
    case = Case(ep, [5, 0, 70], 72, 136)
    gx, gw = case.backward(ep)
    args = case.cfg, case.ddy, case.dstart, case.dend, case.rows
    only_x = ep.expert_mm_backward(*args, w=case.dw, grad_x=case.out(72))
    only_w = ep.expert_mm_backward(*args, x=case.dx)
    assert only_x[1] is None and torch.equal(only_x[0], gx)
    assert only_w[0] is None and torch.equal(only_w[1], gw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [128, 2176, 4224])
def test_more_rows_than_said(ep, H, fp8):
    """num_rows sizes the launch, not the work; with the longer reduction, pairs that share it take
    one tile after another."""
    case = Case(ep, [700, 3, 290], H, 392, A=8, fp8=fp8)
    case.check_forward(case.forward(ep, num_rows=1))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("c", [
    dict(counts=[1], H=7168, N=128), dict(counts=[3, 0, 1], H=2176, N=520),
    dict(counts=[40, 200], H=128, N=2120), dict(counts=[0, 6500, 30], H=128, N=136),
    dict(counts=[5, 2], H=2048, N=4160), dict(counts=[4200], H=384, N=8),
    dict(counts=[1, 8300], H=256, N=72, A=16)], ids=str)
def test_reductions_in_parts(ep, c, fp8):
    """Few tiles and a long reduction, along the inputs, the outputs or the rows."""
    case = Case(ep, fp8=fp8, **c)
    case.check_forward(case.forward(ep))
    for dtype in (torch.bfloat16, torch.float32):
        case.check_backward(*case.backward(ep, grad_w_dtype=dtype))
    first, again = case.forward(ep), case.forward(ep)
    assert torch.equal(first, again)
    if c["N"] % 32 == 0:
        gated = Case(ep, fp8=fp8, gated=True, **c)
        gated.check_forward(gated.forward(ep))


@pytest.mark.parametrize("fp8", [False, True])
def test_sum_in_parts_added_to_what_is_there(ep, fp8):
    case = Case(ep, [9000, 0], 128, 72, fp8=fp8)
    before = torch.randn(2, 72, 128, device="cuda")
    before[:, 0, :2] = torch.tensor([-0.0, 1e-40], device="cuda")
    grad_w = before.clone()
    case.check_backward(*case.backward(ep, grad_w=grad_w, accumulate=True), before)
    assert torch.equal(grad_w[1].view(torch.int32), before[1].view(torch.int32))


def test_no_rows(ep):
    case = Case(ep, [3, 2], 64, 64)
    out = case.out(64)
    assert (case.forward(ep, num_rows=0, out=out) == MARK).all()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert ep.expert_mm(case.cfg, x, case.dw, case.dstart, case.dend, 5).shape == (0, 64)
    for dtype in (torch.bfloat16, torch.float32):
        gw = torch.ones((2, 64, 64), dtype=dtype, device="cuda")
        gx, _ = ep.expert_mm_backward(case.cfg, x, case.dstart, case.dend, 5, w=case.dw, x=x,
                                      grad_w=gw)
        assert gx.shape == (0, 64) and (gw == 0).all()
    ep.expert_mm_backward(case.cfg, x, case.dstart, case.dend, 5, x=x, grad_w=gw + 1,
                          accumulate=True)
    gw = torch.ones((2, 64, 64), device="cuda")
    ep.expert_mm_backward(case.cfg, x, case.dstart, case.dend, 5, x=x, grad_w=gw, accumulate=True)
    assert (gw == 1).all()


def test_segments_are_clipped_to_the_rows_there_are(ep):
    case = Case(ep, [5, 30], 64, 72)
    a = case.forward(ep)
    case.dstart[0] = -4
    case.dend[1] = 1 << 30
    assert torch.equal(case.forward(ep), a)
    gx, gw = case.backward(ep)
    case.check_backward(gx, gw)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_what_is_not_finite_stays_in_its_row(ep, bad):
    case = Case(ep, [20, 40], 128, 136)
    good = case.forward(ep)
    gx, gw = case.backward(ep)
    case.dx[7, 5] = bad
    case.ddy[30, 9] = bad
    out = case.forward(ep)
    assert not torch.isfinite(out[7]).any()
    keep = torch.arange(case.cap, device="cuda") != 7
    assert torch.equal(out[keep], good[keep])
    bx, bw = case.backward(ep)
    keep = torch.arange(case.cap, device="cuda") != 30
    assert not torch.isfinite(bx[30]).any() and torch.equal(bx[keep], gx[keep])
    # an input's column of its expert, a gradient's row of its expert
    assert not torch.isfinite(bw[0][:, 5]).any() and not torch.isfinite(bw[1][9]).any()
    at = torch.isfinite(bw)
    assert torch.equal(bw[at], gw[at]) and int((~at).sum()) == 136 + 128


@pytest.mark.parametrize("bad", ["code", "scale", "infinite scale"])
def test_what_is_not_finite_in_8_bits_stays_in_its_row(ep, bad):
    case = Case(ep, [20, 40], 256, 136, fp8=True)
    good, (_, gw) = case.forward(ep), case.backward(ep)
    if bad == "code":
        case.dx[7, 5] = 0xFF
    else:
        case.dscale[7, 0] = np.nan if bad == "scale" else np.inf
    out, (_, bw) = case.forward(ep), case.backward(ep)
    assert not torch.isfinite(out[7]).any()
    keep = torch.arange(case.cap, device="cuda") != 7
    assert torch.equal(out[keep], good[keep]) and torch.equal(bw[1], gw[1])
    columns = [5] if bad == "code" else list(range(128))
    rest = [c for c in range(256) if c not in columns]
    assert not torch.isfinite(bw[0][:, columns]).any()
    assert torch.equal(bw[0][:, rest], gw[0][:, rest])


@pytest.mark.parametrize("scale", [300.0, 127.9, 1e-30, 1e20, -3.0, 2.0 ** -140])
def test_scales_of_any_size(ep, scale):
    case = Case(ep, [30, 0, 7], 256, 72, fp8=True)
    case.dscale *= scale
    case.xf = ref.f64(ref.values(case.dx, case.dscale))
    case.x = ref.f64(ref.values(case.dx, case.dscale).bfloat16())
    case.xf[~case.own], case.x[~case.own] = 0, 0
    case.check_forward(case.forward(ep))
    if abs(scale) > 1e-35:
        for dtype in (torch.bfloat16, torch.float32):
            case.check_backward(*case.backward(ep, grad_w_dtype=dtype))


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_again_and_on_another_stream(ep, fp8):
    case = Case(ep, [400, 0, 33, 260], 256, 520, fp8=fp8, A=8)
    first, grads = case.forward(ep), case.backward(ep)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        out = case.forward(ep, stream=stream)
        gx, gw = case.backward(ep, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(gx, grads[0]) and torch.equal(gw, grads[1])


def test_captured_and_replayed(ep):
    """A graph reads the segments and rows anew at each replay."""
    case = Case(ep, [30, 0, 99], 128, 72, extra=200)
    other = Case(ep, [0, 140, 2], 128, 72, seed=1, extra=187)
    assert case.cap == other.cap
    names = ("dx", "dw", "ddy", "dstart", "dend")
    first = {n: getattr(case, n).clone() for n in names}
    out, gx = case.out(72), case.out(128)
    gw = torch.zeros((3, 72, 128), device="cuda")

    def both():
        case.forward(ep, out=out)
        case.backward(ep, grad_x=gx, grad_w=gw)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for now in (other, case):
        for n in names:
            getattr(case, n).copy_(first[n] if now is case else getattr(now, n))
        out.fill_(MARK)
        gx.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        now.check_forward(out)
        now.check_backward(gx, gw)


def test_two_calls_at_once(ep):
    """On two streams, with outputs of their own."""
    cases = [Case(ep, [200, 57], 512, 264, seed=s) for s in (1, 2)]
    want = [c.forward(ep) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[c.forward(ep, stream=s) for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in outs:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))


def test_a_long_reduction(ep):
    """Sums over 200,000 rows stay within fp32's error of sums of 16."""
    case = Case(ep, [200000], 8, 16)
    for dtype in (torch.float32, torch.bfloat16):
        gx, gw = case.backward(ep, grad_w_dtype=dtype)
        case.check_backward(gx, gw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("c", [
    dict(counts=[2049, 0, 20000], H=128, N=72), dict(counts=[4100] * 3, H=640, N=1104),
    dict(counts=[2048, 4096, 1], H=384, N=8), dict(counts=[30001], H=256, N=64),
    dict(counts=[16400], H=128, N=2800), dict(counts=[8230, 8200], H=128, N=96)], ids=str)
def test_long_sums_in_32_bits(ep, c, fp8):
    """An fp32 gradient is off by what one sum of 2048 rows is: 128 times a dropped last bit of the
    sum so far, which is no longer than the whole in the norm (twice, for the two parts of E4M3
    rows, and half a step of their second, 2^-17), and a rounding for each of the sums added."""
    case = Case(ep, fp8=fp8, **c)
    before = torch.randn(len(c["counts"]), c["N"], c["H"], device="cuda")
    grad_w = before.clone()
    _, got = case.backward(ep, grad_w_dtype=torch.float32)
    case.backward(ep, grad_w=grad_w, accumulate=True)
    for _ in range(5):
        assert torch.equal(case.backward(ep, grad_w_dtype=torch.float32)[1], got)
    for e, n in enumerate(c["counts"]):
        rows = slice(int(case.start[e]), int(case.end[e]))
        y = ref.f64(case.dy[rows]).T @ case.xf[rows]
        norm = np.linalg.norm(y) or 1.0
        off = (129 + n / 2048) * ref.EPS * (2 if fp8 else 1) + (2.0 ** -17 if fp8 else 0)
        assert np.linalg.norm(ref.f64(got[e]) - y) <= off * norm, e
        was = ref.f64(before[e])
        off = off * norm + (2 + n / 2048) * ref.EPS * np.linalg.norm(abs(y) + abs(was))
        assert np.linalg.norm(ref.f64(grad_w[e]) - y - was) <= off, e


def test_rows_past_32_bit_offsets(ep):
    """Rows whose element offsets do not fit 32 bits."""
    H, N, cap = 4096, 8, 700000
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((cap, H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.empty((2, N, H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    start = torch.tensor([0, cap - 70], dtype=torch.int32, device="cuda")
    end = torch.tensor([3, cap], dtype=torch.int32, device="cuda")
    cfg = ep.ExpertConfig(2, H, N)
    out = ep.expert_mm(cfg, x, w, start, end, 73)
    dy = torch.empty((cap, N), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    gx, gw = ep.expert_mm_backward(cfg, dy, start, end, 73, w=w, x=x)
    for e, rows in ((0, slice(0, 3)), (1, slice(cap - 70, cap))):
        y, err = ref.forward(ref.f64(x[rows]), ref.f64(w[e]), False)
        assert (abs(ref.f64(out[rows]) - y) <= err).all()
        y, err = ref.by_rows(ref.f64(dy[rows]), ref.f64(w[e]))
        assert (abs(ref.f64(gx[rows]) - y) <= err).all()
        y, err = ref.by_weights(ref.f64(dy[rows]), ref.f64(x[rows]), False)
        assert (abs(ref.f64(gw[e]) - y) <= err).all()


@pytest.mark.parametrize("H", [1152, 4224])
@pytest.mark.parametrize("kw", [dict(), dict(gated=True), dict(fp8=True)], ids=str)
def test_waits_that_run_out_are_reported(ep, kw, H):
    """Copies that never come: the kernel ends by itself, the error word says so, and the next call
    is right."""
    case = Case(ep, [40, 3], H, 320, **kw)
    err, out = torch.zeros(4, dtype=torch.int32, device="cuda"), case.out(case.cfg.out_width)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    st = ep.ep_selftest_expert_timeout(case.cfg.c(), case.cap, case.rows, ptr(case.dx),
                                       ptr(case.dscale), ptr(case.dw), ptr(case.dstart),
                                       ptr(case.dend), ptr(out), ptr(err), stream)
    assert st == ep.EP_OK
    torch.cuda.synchronize()
    assert err[0].item() & 4 and (err[1:] == 0).all()
    err.zero_()
    case.check_forward(case.forward(ep, err=err))
    assert (err == 0).all()
