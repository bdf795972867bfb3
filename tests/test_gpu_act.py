"""The gated activation with its 8-bit checkpoint on the GPU against plain 64-bit forms
(expert_ref.py)."""

import numpy as np
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu

MARK = 77.0


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


class Case:
    def __init__(self, counts, I, A=1, extra=0, seed=0):
        rng = np.random.default_rng(seed)
        self.counts, self.I, self.blocks = counts, I, -(-I // 128)
        self.start, self.end = ref.segments(counts, A)
        self.cap = max(1, int(self.start[-1])) + extra
        self.own = np.zeros(self.cap, bool)
        for s, e in zip(self.start, self.end):
            self.own[s:e] = True
        h = rng.standard_normal((self.cap, 2 * I)) * rng.choice([0.01, 1, 8], (self.cap, 1))
        h[::7, : min(I, 128)] = 0
        h[~self.own] = np.nan
        self.h = ref.bf16(h)
        self.da = ref.bf16(rng.standard_normal((self.cap, I)))
        self.seg = (torch.from_numpy(self.start).cuda(), torch.from_numpy(self.end).cuda(),
                    int(sum(counts)))

    def outputs(self):
        new = lambda w, t, v: torch.full((self.cap, w), v, dtype=t, device="cuda")  # noqa: E731
        return (new(self.I, torch.bfloat16, MARK), new(2 * self.I, torch.uint8, 77),
                new(2 * self.blocks, torch.float32, MARK))

    def save(self, ep, **kw):
        a, q, s = self.outputs()
        return ep.act_save(self.h.cuda(), *self.seg, a=a, h_q=q, h_scale=s, **kw)

    def codes(self):
        g, u = (ref.quantise(p.contiguous()) for p in self.h.float().chunk(2, 1))
        return torch.cat([g[0], u[0]], 1), torch.cat([g[1], u[1]], 1)

    def kept(self, q, scale):
        (gq, uq), (gs, us) = q.chunk(2, 1), scale.chunk(2, 1)
        return ref.f64(torch.cat([ref.values(gq.contiguous(), gs), ref.values(uq.contiguous(), us)],
                                 1))


def name_of(c):
    return str(c) if len(str(c)) < 99 else str(dict(c, counts=len(c["counts"])))


CASES = [
    dict(counts=[1], I=8), dict(counts=[1], I=128), dict(counts=[3, 0, 2], I=136, A=8),
    dict(counts=[0, 0, 9], I=1000), dict(counts=[5, 1], I=512), dict(counts=[2, 7], I=520, A=128),
    dict(counts=[1] * 70, I=16), dict(counts=[40, 33], I=2048, A=16), dict(counts=[0, 0], I=64),
    dict(counts=[300, 0, 1], I=1408, extra=5), dict(counts=[1] * 33, I=24),
    dict(counts=[4], I=7168), dict(counts=[1, 1], I=1 << 19), dict(counts=[0, 1, 2, 0] * 512, I=16),
]


@pytest.mark.parametrize("c", CASES, ids=name_of)
def test_save(ep, c):
    case = Case(**c)
    a, q, s = case.save(ep)
    own = torch.from_numpy(case.own)
    y, err = ref.activation(ref.f64(case.h)[case.own])
    assert (abs(ref.f64(a)[case.own] - y) <= err).all()
    want_q, want_s = case.codes()
    assert torch.equal(q.cpu()[own], want_q[own]) and torch.equal(s.cpu()[own], want_s[own])
    assert (a.cpu()[~own] == MARK).all() and (q.cpu()[~own] == 77).all()
    assert (s.cpu()[~own] == MARK).all()


@pytest.mark.parametrize("c", CASES, ids=name_of)
def test_backward(ep, c):
    case = Case(**c)
    q, s = case.codes()
    dh = torch.full((case.cap, 2 * case.I), MARK, dtype=torch.bfloat16, device="cuda")
    a = torch.full((case.cap, case.I), MARK, dtype=torch.bfloat16, device="cuda")
    ep.act_backward(case.da.cuda(), q.cuda(), s.cuda(), *case.seg, grad_h=dh, a=a)
    h = case.kept(q, s)[case.own]
    y, err = ref.activation_backward(ref.f64(case.da)[case.own], h)
    assert (abs(ref.f64(dh)[case.own] - y) <= err).all()
    y, err = ref.activation(h)
    assert (abs(ref.f64(a)[case.own] - y) <= err).all()
    own = torch.from_numpy(case.own)
    assert (dh.cpu()[~own] == MARK).all() and (a.cpu()[~own] == MARK).all()
    alone, none = ep.act_backward(case.da.cuda(), q.cuda(), s.cuda(), *case.seg, want_a=False)
    assert none is None and torch.equal(alone.cpu()[own], dh.cpu()[own])


def test_values_at_the_ends(ep):
    """Blocks that hold infinities, NaN, the smallest and the largest values: what a dispatch's
    codes are for them, and an activation in each element that has one."""
    v = torch.tensor([0.0, -0.0, 1e-38, -1e-40, 3e38, -3e38, 88.0, -88.0, -200.0, 200.0, 1.0, -1.28])
    h = torch.zeros(6, 256)
    h[0, :12], h[0, 128:140] = v, 1.0
    h[1, :12], h[1, 128:140] = 1.0, v
    h[2, 3], h[3, 5], h[4, 130] = np.inf, np.nan, -np.inf
    h[5] = 1e-40
    h = h.bfloat16()
    seg = (torch.tensor([0], dtype=torch.int32, device="cuda"),
           torch.tensor([6], dtype=torch.int32, device="cuda"), 6)
    a, q, s = ep.act_save(h.cuda(), *seg)
    f = h.double()
    with np.errstate(all="ignore"):
        want = (f[:, :128] / (1 + torch.exp(-f[:, :128])) * f[:, 128:])
    fin = torch.isfinite(want) & (abs(want) < 3.3e38)
    d = abs(a.cpu().double() - want)
    # a sigmoid under 2^-126 counts as 0: the whole value may be missing there
    lost = torch.where(torch.sigmoid(f[:, :128]) < 2.0 ** -125, abs(want), 0)
    assert (d[fin] <= (2.0 ** -7 * abs(want) + lost + 1e-38)[fin]).all()
    assert torch.isnan(a[3, 5]) and torch.isfinite(a[3, :5]).all()
    cfg = ep.Config(6, 256, 1, 1, 1, 1, True)
    layout = ep.get_layout(cfg, torch.zeros((6, 1), dtype=torch.int64, device="cuda"))
    want_q, want_s, _ = ep.dispatch(cfg, layout, h.cuda())
    assert torch.equal(q, want_q[:6]) and torch.equal(s, want_s[:6])


def test_a_checkpoint_is_a_row_in_8_bits(ep):
    """Where 128 divides the width, a product takes a checkpoint as its rows."""
    case = Case([20, 0, 9], 128, A=8)
    _, q, s = case.save(ep)
    w = ref.bf16(np.random.default_rng(5).standard_normal((3, 40, 256)) / 16)
    out = ep.expert_mm(ep.ExpertConfig(3, 256, 40, x_fp8=True), q, w.cuda(), *case.seg, x_scale=s)
    x = ref.f64(ref.values(q, s))
    for e, n in enumerate(case.counts):
        rows = slice(int(case.start[e]), int(case.end[e]))
        if n:
            y, err = ref.forward(x[rows], ref.f64(w[e]), False, True)
            assert (abs(ref.f64(out[rows]) - y) <= err).all()


def test_streams_capture_and_more_rows_than_said(ep):
    case = Case([70, 0, 33], 520, A=8)
    want = case.save(ep)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = case.save(ep, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s, e, _ = case.seg
    outs, h = case.outputs(), case.h.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.act_save(h, s, e, 1, *outs)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    da = case.da.cuda()
    want = ep.act_backward(da, outs[1], outs[2], s, e, 103)
    got = [torch.zeros_like(t) for t in want]
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
        ep.act_backward(da, outs[1], outs[2], s, e, 103, *got)
    graph.replay()
    torch.cuda.synchronize()
    own = torch.from_numpy(case.own).cuda()
    assert all(torch.equal(a[own], b[own]) for a, b in zip(got, want))


def test_no_rows(ep):
    case = Case([3], 64)
    a, q, s = case.outputs()
    ep.act_save(case.h.cuda(), *case.seg[:2], 0, a, q, s)
    assert (a == MARK).all() and (q == 77).all() and (s == MARK).all()
    h = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    a, q, s = ep.act_save(h, *case.seg)
    assert a.shape == (0, 64) and q.shape == (0, 128) and s.shape == (0, 2)
    assert ep.act_backward(a, q, s, *case.seg)[0].shape == (0, 128)


@pytest.mark.parametrize("start,end", [([-5, 4], [2, 1 << 30]), ([0, 0], [6, 6])])
def test_segments_are_clipped(ep, start, end):
    """To the rows there are; rows in two segments are computed twice, alike."""
    case = Case([6], 128)
    seg = (torch.tensor(start, dtype=torch.int32, device="cuda"),
           torch.tensor(end, dtype=torch.int32, device="cuda"), 12)
    a, q, s = ep.act_save(case.h.cuda(), *seg, *case.outputs())
    b, r, t = case.save(ep)
    own = torch.zeros(6, dtype=torch.bool)
    for lo, hi in zip(start, end):
        own[max(lo, 0):hi] = True
    for got, want in ((a, b), (q, r), (s, t)):
        assert torch.equal(got.cpu()[own], want.cpu()[own])
        assert (got.cpu()[~own] == 77).all()


def test_codes_are_a_dispatchs(ep):
    """Every bf16 maximum of a block, with values of all magnitudes below it: the codes and scales
    that an FP8 dispatch gives the same rows."""
    top = torch.arange(0, 0x7F81, dtype=torch.int32, device="cuda").to(torch.int16)
    gen = torch.Generator(device="cuda").manual_seed(7)
    h = torch.randint(0, 1 << 15, (len(top), 128), device="cuda", generator=gen, dtype=torch.int32)
    h = torch.minimum(h % (top.int()[:, None] + 1), top.int()[:, None]).to(torch.int16)
    h[:, ::2] |= -(1 << 15)
    h[:, 5] = top
    h = h.view(torch.bfloat16)
    h = torch.cat([h, h.flip(0)], 1).contiguous()
    n = len(h)
    seg = (torch.tensor([0], dtype=torch.int32, device="cuda"),
           torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    _, q, s = ep.act_save(h, *seg)
    cfg = ep.Config(n, 256, 1, 1, 1, 1, True)
    layout = ep.get_layout(cfg, torch.zeros((n, 1), dtype=torch.int64, device="cuda"))
    want_q, want_s, _ = ep.dispatch(cfg, layout, h)
    assert torch.equal(s, want_s[:n])
    nan = (want_q[:n] & 0x7F) == 0x7F
    assert torch.equal((q & 0x7F) == 0x7F, nan) and torch.equal(q[~nan], want_q[:n][~nan])
