"""Both forms of the gradient products' kernel (tiles of one CTA, of SM pairs) on the same inputs, named
by moe_gemm_backward_form so that the cost model's constants do not decide what is covered: group
lengths, rows outside every group, offsets that are no plan, rows that are not finite, every scale
byte, streams and graphs that share a workspace.  Integers whose sums are exact in fp32: outputs are
compared bit for bit."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _grad_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8

EDGES = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 191, 192, 193, 255, 256, 257, 511, 513, 0]
both = pytest.mark.parametrize("ctas", [1, 2])
formats = pytest.mark.parametrize("product,nv", [(2, False), (13, False), (2, True), (13, True)])


class _Case:
    """Groups of these lengths (gap: rows in front of the first and behind the last) with |dy| <= 2 and
    weights, NVFP4's tensor scales of 1/2, 1 or 2 included, up to 36 in steps of 1/4: sums below
    2^24 / 4."""

    def __init__(self, product, nv, lens, H=512, I=256, gap=(0, 0), seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed + H + 3 * I + len(lens))
        ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
        self.product, self.nv, rows, G = product, nv, sum(lens) + sum(gap), len(lens)
        C, F = (H, I) if product == 2 else (2 * I, H)
        self.off = torch.tensor([gap[0] + sum(lens[:i]) for i in range(G + 1)], dtype=I32, device=DEV)
        self.dy, self.w = ri(-2, 3, rows, C).to(BF), ri(0, 256, G, C, F // 2).to(U8)
        self.gs = None
        if nv:
            self.w_s = ri(1, 4, G, C, F // 16).float().to(torch.float8_e4m3fn).view(U8)
            self.gs = torch.tensor([0.5, 1.0, 2.0], device=DEV)[ri(0, 3, *((G,) if product == 2 else (G, 2)))]
        else:
            self.w_s = ri(127, 129, G, C, F // 32).to(U8)
        self.d = moe.dims(rows, H, I, G, 1, 0)
        self.dx = torch.full((rows, F), 7.0, dtype=BF, device=DEV)
        self.ws = moe.alloc_workspace(256)

    def run(self, ctas, dx=None, dy=None):
        moe.moe_gemm_backward_form(self.d, self.product, ctas, self.dy if dy is None else dy, self.off,
                                   self.w, self.w_s, self.dx if dx is None else dx, self.ws, self.gs, self.nv)
        return self

    def want(self):
        dx = ref.expert_grad(self.dy, self.off, self.w, self.w_s, *self.dx.shape, self.gs, self.nv)[0]
        return torch.where(torch.isnan(dx), 7.0, dx).to(BF)  # (rows of no group stay)

    def check(self):
        assert moe.moe_check_status(self.ws) == 0
        assert torch.equal(self.dx, self.want())


@both
@formats
@pytest.mark.parametrize("lens", [EDGES, [1], [0, 3], [16] * 40, [1] * 300, [2000], [0] * 8 + [5] + [0] * 8,
                                  [1, 0] * 512, [260, 3, 700, 1]], ids=lambda v: f"{len(v)}x{v[0]}")
def test_group_lengths(ctas, product, nv, lens):
    _Case(product, nv, lens).run(ctas).check()


@both
@formats
@pytest.mark.parametrize("H,I", [(256, 256), (1280, 768), (768, 1280)])
def test_features_and_contractions(ctas, product, nv, H, I):
    _Case(product, nv, [3, 0, 290, 17, 140, 64, 33], H, I).run(ctas).check()


@both
@pytest.mark.parametrize("product,H,I", [(2, 128, 128), (13, 128, 128), (2, 384, 640), (13, 1152, 128)])
def test_odd_multiples_of_128(ctas, product, H, I):
    _Case(product, False, EDGES, H, I).run(ctas).check()


@both
@formats
@pytest.mark.parametrize("lens,gap", [([3, 40, 0, 270], (5, 0)), ([3, 40, 0, 270], (0, 9)),
                                      ([130, 1], (130, 300)), ([0, 0, 0], (0, 12))])
def test_rows_outside_every_group(ctas, product, nv, lens, gap):
    _Case(product, nv, lens, gap=gap).run(ctas).check()


@both
@formats
def test_rows_outside_every_group_have_no_part(ctas, product, nv):
    c = _Case(product, nv, [3, 40, 0, 270], gap=(5, 9))
    want = c.want()
    c.dy[:5], c.dy[-9:] = float("nan"), float("inf")
    assert torch.equal(c.run(ctas).dx, want)


@both
@formats
@pytest.mark.parametrize("lens", [[5, -2, 6, 3], [5, 200], [-1, 5, 8]])
def test_offsets_that_are_no_plan(ctas, product, nv, lens):
    c = _Case(product, nv, [3, 3, 3, 3])
    c.off = torch.tensor([0] + lens + [0] * (4 - len(lens)), dtype=I32, device=DEV).cumsum(0).to(I32)
    c.run(ctas)
    assert moe.moe_check_status(c.ws) == moe.STATUS_BAD_PLAN
    assert torch.all(c.dx == 7.0)


@both
@formats
def test_rows_that_are_not_finite_stay_in_their_rows(ctas, product, nv):
    c = _Case(product, nv, [20, 200, 30]).run(ctas)
    bad, out = c.dy.clone(), torch.empty_like(c.dx)
    bad[3, 5], bad[100, 7], bad[249, -1] = float("nan"), float("inf"), float("nan")
    c.run(ctas, out, bad)
    rest = torch.ones(250, dtype=torch.bool, device=DEV)
    rest[[3, 100, 249]] = False
    assert torch.equal(out[rest], c.dx[rest])
    assert torch.all(torch.isnan(out[[3, 249]])) and not torch.any(torch.isfinite(out[100]))


@both
@pytest.mark.parametrize("nv", [False, True])
def test_every_scale_byte(ctas, nv):
    """One-hot rows read single weight rows back: group b has scale byte b in row b (MXFP4: weights
    below 2^-126 may count as 0, values past bf16's range are infinities, byte 255 is NaN)."""
    H, I, G = 256, 512, 256
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.randint(0, 256, (G, H, I // 2), generator=g, device=DEV).to(U8)
    w_s = torch.full((G, H, I // (16 if nv else 32)), 56 if nv else 120, dtype=U8, device=DEV)
    b = torch.arange(G, device=DEV)
    w_s[b, b] = b.to(U8)[:, None]
    dy = torch.zeros(G, H, dtype=BF, device=DEV)
    dy[b, b] = 1.0
    dx, ws = torch.empty(G, I, dtype=BF, device=DEV), moe.alloc_workspace(256)
    moe.moe_gemm_backward_form(moe.dims(G, H, I, G, 1, 0), 2, ctas, dy,
                               torch.arange(G + 1, dtype=I32, device=DEV), w, w_s, dx, ws, nvfp4=nv)
    assert moe.moe_check_status(ws) == 0
    nan = torch.zeros(G, dtype=torch.bool, device=DEV)
    nan[[127, 255] if nv else [255]] = True
    want = (ref.nvfp4 if nv else ref.mxfp4)(w[b, b][:, None], w_s[b, b][:, None])[:, 0]
    got, want = dx[~nan].double(), want[~nan].to(BF).double()
    assert torch.all(torch.isnan(dx[nan]))
    small = want.abs() < 2.0 ** -126
    assert torch.equal(got[~small], want[~small])
    assert torch.all((got - want)[small].abs() <= want[small].abs())


@both
@formats
def test_the_same_in_every_run(ctas, product, nv):
    c = _Case(product, nv, [100, 3, 600, 40], 1280, 768)
    dy = torch.randn(c.dy.shape, device=DEV).to(BF)
    a, b = (torch.empty_like(c.dx) for _ in range(2))
    c.run(ctas, a, dy)
    for _ in range(5):
        c.run(ctas, b, dy)
        assert torch.equal(a, b)


@both
@formats
def test_two_streams_and_two_graphs_with_one_workspace(ctas, product, nv):
    cases = [_Case(product, nv, [100, 200], seed=s) for s in (1, 2)]
    cases[1].ws = cases[0].ws
    streams, graphs = [[f() for _ in cases] for f in (torch.cuda.Stream, torch.cuda.CUDAGraph)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.run(ctas)
    torch.cuda.synchronize()
    for c, g in zip(cases, graphs):
        c.check()
        with torch.cuda.graph(g):
            c.run(ctas)
        c.dx.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_public_calls_reach_both_forms():
    forms = {moe.gemm_backward_ctas(moe.dims(T, 512, 256, 8, 2, 1), p) for T in (4, 4096) for p in (2, 13)}
    assert forms == {1, 2}
