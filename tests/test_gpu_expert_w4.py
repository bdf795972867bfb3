"""The experts' products with 4-bit weights on the GPU against a plain 64-bit
form (layer_ref.py)."""

import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


class Case:
    """Weights and rows of E experts with `counts` rows each, aligned to A."""

    def __init__(self, ep, counts, H, N, group=128, fp8=False, gated=False, zeros=False, A=1,
                 seed=0):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.cfg = ep.W4Config(E, H, N, group, fp8, gated, zeros)
        self.group, self.gated, self.counts = group, gated, counts
        self.codes = rng.integers(0, 256, (E, N, H // 2)).astype(np.uint8)
        s = bf16(rng.uniform(0.5, 1.5, (E, N, H // group)) * rng.choice([-1, 1, 1]) / (4 * H ** 0.5))
        self.scales = s.double().numpy()
        self.zeros = rng.integers(0, 16, self.scales.shape).astype(np.uint8) if zeros else None
        self.packed = ep.w4_pack(self.cfg, torch.from_numpy(self.codes).cuda(), s.cuda(),
                                 None if not zeros else torch.from_numpy(self.zeros).cuda())
        self.start = np.concatenate([[0], np.cumsum([-(-c // A) * A for c in counts])])
        self.end = self.start[:-1] + np.array(counts)
        self.cap = max(1, int(self.start[-1]))
        x = rng.standard_normal((self.cap, H))
        if fp8:
            q = torch.from_numpy(x * 100).to(torch.float8_e4m3fn)
            self.x_scale = rng.uniform(0.001, 0.02, (self.cap, H // 128)).astype(np.float32)
            self.x = q.double().numpy() * np.repeat(self.x_scale.astype(np.float64), 128, 1)
            self.dx = q.view(torch.uint8).cuda()
            self.dscale = torch.from_numpy(self.x_scale).cuda()
        else:
            self.dx = bf16(x).cuda()
            self.x, self.dscale = self.dx.double().cpu().numpy(), None
        self.dstart = torch.tensor(self.start, dtype=torch.int32).cuda()
        self.dend = torch.tensor(self.end, dtype=torch.int32).cuda()

    def run(self, ep, out=None, num_rows=None, stream=None):
        c, s, z = self.packed
        n = int(sum(self.counts)) if num_rows is None else num_rows
        return ep.expert_w4(self.cfg, self.dx, c, s, self.dstart, self.dend, n, zeros=z,
                            x_scale=self.dscale, out=out, stream=stream)

    def check(self, out):
        got = out.double().cpu().numpy()
        for e, n in enumerate(self.counts):
            if n == 0:
                continue
            W = ref.w4_matrix(self.codes[e], self.scales[e],
                              None if self.zeros is None else self.zeros[e], self.group)
            rows = slice(int(self.start[e]), int(self.end[e]))
            y, err = ref.w4(self.x[rows], W, self.gated)
            # bf16 rounds by at most 2^-9 of the value
            assert (abs(got[rows] - y) <= err + 2.0 ** -8 * abs(y) + 1e-30).all(), e


CASES = [
    dict(counts=[1], H=128, N=64), dict(counts=[1], H=32, N=1, group=32),
    dict(counts=[3], H=96, N=70, group=32), dict(counts=[8], H=1408, N=1000, group=64),
    dict(counts=[9], H=256, N=130, group=128), dict(counts=[1], H=2048, N=512),
    dict(counts=[1, 0, 2, 0, 0, 7, 8, 9], H=384, N=96, group=32, zeros=True, A=8),
    dict(counts=[0, 0, 5], H=160, N=66, group=32, gated=True),
    dict(counts=[17, 1, 40], H=512, N=200, gated=True, A=16),
    dict(counts=[2, 33, 0, 16], H=256, N=192, fp8=True, A=8),
    dict(counts=[1] * 70, H=128, N=64, fp8=True, gated=True, group=64, zeros=True),
    dict(counts=[65, 100], H=256, N=64, zeros=True), dict(counts=[1, 1], H=7168, N=128, fp8=True),
    dict(counts=[4, 24], H=2080, N=72, group=32), dict(counts=[1], H=8192, N=62, gated=True),
    dict(counts=[0, 1] * 40 + [3], H=64, N=130, group=64),
    dict(counts=[5, 6], H=640, N=2050, group=128, gated=True, zeros=True),
    dict(counts=[0] * 32 + [9], H=64, N=64, group=32), dict(counts=[3] * 33, H=64, N=64, group=64),
    dict(counts=[1, 0, 0] * 352 + [2], H=32, N=32, group=32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_product(ep, case):
    k = Case(ep, **case)
    out = torch.full((k.cap, k.cfg.out_width), 77.0, dtype=torch.bfloat16, device="cuda")
    k.run(ep, out)
    k.check(out)
    used = np.zeros(k.cap, bool)
    for s, e in zip(k.start, k.end):
        used[s:e] = True
    assert (out[torch.from_numpy(~used).cuda()] == 77.0).all()      # rows of no expert
    again = torch.full_like(out, 77.0)
    k.run(ep, again, num_rows=1)                                    # the bound only sizes the launch
    assert torch.equal(out, again)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
def test_packed_layout(ep, gated, zeros):
    """Every code, scale and zero point at the place include/ep.h gives it."""
    E, N, H, g = 2, 74, 160, 32
    k = Case(ep, [1, 1], H, N, g, gated=gated, zeros=zeros)
    codes, scales, zs = (None if t is None else t.cpu() for t in k.packed)
    tiles, blocks = codes.shape[1:3]
    assert tiles == (2 if gated or N > 64 else 1) and blocks == 2
    words = codes.numpy().view(np.uint32)
    q = np.stack([k.codes & 15, k.codes >> 4], -1).reshape(E, N, H)
    half = N // 2
    for e in range(E):
        for t in range(tiles):
            for n in range(64):
                if gated:
                    o = t * 32 + n // 8 * 4 + n % 4
                    row = (half + o if n & 4 else o) if o < half else -1
                else:
                    row = t * 64 + n if t * 64 + n < N else -1
                for s in range(blocks * 128 // g):
                    have = row >= 0 and s < H // g
                    assert float(scales[e, t, s, n]) == (k.scales[e, row, s] if have else 0.0)
                    if zeros:
                        assert int(zs[e, t, s, n]) == (k.zeros[e, row, s] if have else 8)
                for h in range(blocks * 128):
                    b, i, lq, r = h // 128, h % 128 // 32, h % 32 // 8, h % 8
                    word = int(words[e, t, b, n % 8, n // 8 * 4 + lq, i])
                    field = word >> (4 * (r // 2 + 4 * (r % 2))) & 15
                    assert field == (q[e, row, h] if row >= 0 and h < H else 8)


def test_special_values_stay_in_their_row(ep):
    """A row of x that is not finite, and lowest values, leave the others be."""
    k = Case(ep, [6], 256, 96, 64)
    want = k.run(ep)
    k.dx[2, 3] = float("nan")
    k.dx[4, 200] = float("inf")
    k.dx[5] = 0
    got = k.run(ep)
    assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]])
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[4]).any()
    assert (got[5] == 0).all()


def test_segments_are_clipped_to_the_buffers(ep):
    k = Case(ep, [4, 4, 4], 128, 64)
    want = k.run(ep)
    k.dstart[0], k.dend[2] = -5, 40           # rows [0, 4) and [8, 12)
    k.dstart[1], k.dend[1] = 7, 3             # none
    out = torch.full_like(want, 9.0)
    k.run(ep, out)
    assert torch.equal(out[:4], want[:4]) and torch.equal(out[8:], want[8:])
    assert (out[4:8] == 9.0).all()


def test_offsets_past_31_bits(ep):
    """Codes, rows and outputs whose byte offsets need more than 32 bits."""
    E, H, N = 3, 32768, 65536 + 64
    cfg = ep.W4Config(E, H, N, 128)
    gen = torch.Generator(device="cuda").manual_seed(1)
    tiles, blocks = (N + 63) // 64, H // 128
    codes = torch.randint(-2**31, 2**31 - 1, (E, tiles, blocks, 8, 32, 4), dtype=torch.int32,
                          device="cuda", generator=gen)
    scales = torch.full((E, tiles, blocks, 64), 0.001, dtype=torch.bfloat16, device="cuda")
    cap = 70000
    x = torch.zeros((cap, H), dtype=torch.bfloat16, device="cuda")
    x[cap - 2:] = torch.randn((2, H), device="cuda", generator=gen).bfloat16()
    out = torch.zeros((cap, N), dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 0, cap - 2], dtype=torch.int32, device="cuda")
    end = torch.tensor([0, 0, cap], dtype=torch.int32, device="cuda")
    ep.expert_w4(cfg, x, codes, scales, start, end, 2, out=out)
    tile = codes[2, tiles - 1].cpu().numpy().view(np.uint32)      # last 64 rows, [blocks, 8, 32, 4]
    W = np.zeros((64, H))
    for p in range(8):
        for j in range(8):
            f = (tile[:, p] >> (4 * j)) & 15                      # [blocks, 32, 4]
            h = np.arange(4)[None, None] * 32 + (np.arange(32) % 4 * 8)[None, :, None] + \
                (2 * j if j < 4 else 2 * j - 7) + np.arange(blocks)[:, None, None] * 128
            n = np.broadcast_to((np.arange(32) // 4 * 8 + p)[None, :, None], h.shape)
            W[n, h] = f - 8.0
    W *= float(scales[0, 0, 0, 0])
    y, err = ref.w4(x[cap - 2:].double().cpu().numpy(), W, False)
    got = out[cap - 2:, N - 64:].double().cpu().numpy()
    assert (abs(got - y) <= err + 2.0 ** -8 * abs(y)).all()
    assert not out[:cap - 2, :64].any()


def test_another_stream_and_a_graph(ep):
    k = Case(ep, [3, 0, 9], 256, 130, 64, gated=True)
    want = k.run(ep)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = k.dx.clone()
    k.dx.zero_()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        k.dx.copy_(x)
        k.run(ep, out)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k.run(ep, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_torch_layer_refuses(ep):
    k = Case(ep, [2, 2], 256, 64)
    c, s, _ = k.packed
    a = (c, s, k.dstart, k.dend, 4)
    z = torch.zeros(s.shape, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: ep.W4Config(2, 100, 64, 32), lambda: ep.W4Config(2, 160, 64, 32, x_fp8=True),
        lambda: ep.W4Config(2, 128, 63, 32, gated=True), lambda: ep.W4Config(2, 128, 64, 16),
        lambda: ep.W4Config(0, 128, 64), lambda: ep.W4Config(2049, 128, 64),
        lambda: ep.expert_w4(k.cfg, k.dx.float(), *a),
        lambda: ep.expert_w4(k.cfg, k.dx[:, :128], *a),
        lambda: ep.expert_w4(k.cfg, k.dx, c[:1], *a[1:]),
        lambda: ep.expert_w4(k.cfg, k.dx, *a, zeros=z),
        lambda: ep.expert_w4(k.cfg, k.dx, *a, x_scale=torch.zeros((4, 2), device="cuda")),
        lambda: ep.expert_w4(k.cfg, k.dx, *a, out=torch.zeros((4, 64), device="cuda")),
        lambda: ep.expert_w4(k.cfg, k.dx, c, s, k.dstart[:1], k.dend, 4),
        lambda: ep.expert_w4(k.cfg, k.dx, c, s, k.dstart.long(), k.dend, 4),
        lambda: ep.expert_w4(k.cfg, k.dx, c, s, k.dstart, k.dend, -1),
        lambda: ep.w4_pack(k.cfg, torch.zeros((2, 64, 100), dtype=torch.uint8, device="cuda"),
                           s),
    ]
    for call in bad:
        with pytest.raises(ep.EpError) as err:
            call()
        assert err.value.status == ep.EP_ERR_INVALID_ARG
