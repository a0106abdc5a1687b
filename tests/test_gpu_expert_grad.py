"""Gradient products of the MXFP4 experts (moe_grouped_gemm_w2_backward / _w13_backward) against
float64: bit-exact on integers, every group length around the tiles' edges, empty groups and
rows outside every group, every scale byte, few and many features and contractions.

Tolerance on real numbers: half a step of bf16, and for each of the C / 16 steps of the tensor
cores' fp32 sum 2^-22 of the terms' magnitudes."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _grad_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8

EDGES = [1, 0, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 0, 96, 127, 128, 129, 191, 192, 193, 0, 255,
         256, 257, 300, 511, 512, 513, 0]


def _call(which, lens, H, I, seed=0, ints=True, gap=(0, 0), scales=(127, 129)):
    """Groups of these lengths (gap: rows in front of the first and behind the last).  Returns
    the inputs and the output, which starts as 7."""
    g = torch.Generator(device=DEV).manual_seed(seed + H + 3 * I + len(lens))
    rows = sum(lens) + sum(gap)
    C, F = (H, I) if which == "w2" else (2 * I, H)
    G = len(lens)
    off = torch.tensor([gap[0] + sum(lens[:i]) for i in range(G + 1)], dtype=I32, device=DEV)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
    if ints:
        # |dy| <= 2 and weights of whole or half steps up to 6 * 2: sums are multiples of 1/2
        # below 2^23 / 2, exact in fp32
        dy = ri(-2, 3, rows, C).to(BF)
        w_s = ri(*scales, G, C, F // 32).to(U8)
    else:
        dy = torch.randn(rows, C, generator=g, device=DEV).to(BF)
        w_s = ri(110, 130, G, C, F // 32).to(U8)
    w = ri(0, 256, G, C, F // 2).to(U8)
    d = moe.dims(rows, H, I, G, 1, 0)
    dx = torch.full((rows, F), 7.0, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    f = moe.moe_grouped_gemm_w2_backward if which == "w2" else moe.moe_grouped_gemm_w13_backward
    f(d, dy, off, w, w_s, dx, ws)
    assert moe.moe_check_status(ws) == 0
    return dy, off, w, w_s, dx


def _check(dy, off, w, w_s, dx, ints):
    want, size = ref.expert_grad(dy, off, w, w_s, *dx.shape)
    out = torch.isnan(want)
    assert torch.all(dx[out] == 7.0)  # rows of no group
    if ints:
        assert torch.equal(dx[~out], want[~out].to(BF))  # (exact in fp32, so one rounding)
    else:
        tol = ref.U16 * want.abs() + (dy.shape[1] / 16 + 1) * 2.0 ** -22 * size
        assert torch.all((dx.double() - want).abs()[~out] <= tol[~out])


# (on single CTAs or SM pairs by the sizes' cost; some features end in a pair's first half.  Each
# form by name: test_gpu_grad_forms.py)
@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("H,I", [(128, 128), (256, 384), (640, 128), (1152, 256), (384, 640),
                                 (4096, 1152), (1152, 2048), (2048, 2048)])
@pytest.mark.parametrize("ints", [True, False])
def test_group_lengths(which, H, I, ints):
    _check(*_call(which, EDGES, H, I, ints=ints), ints)


@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("lens", [[1], [7], [0, 3], [16] * 40, [1] * 300, [2000], [0] * 8 + [5] + [0] * 8,
                                  [1, 0] * 512, [260, 3, 700, 1]])
def test_few_and_many_groups(which, lens):
    _check(*_call(which, lens, 512, 256), True)


@pytest.mark.parametrize("which", ["w2", "w13"])
def test_layer_sizes(which):
    _check(*_call(which, [3, 0, 290, 17, 140, 64], 7168, 2048), True)
    _check(*_call(which, [3, 0, 290, 17, 140, 64], 7168, 2048, ints=False), False)


@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("H,I", [(512, 256), (2048, 1152), (1152, 1024)])
def test_scales_above_one_factors_range(which, H, I):
    """Scale bytes on both sides of 128, where a bf16 factor ends: |dy| <= 2, weights up to
    6 * 2^5 in steps of 2^-3, sums of 2304 terms below 2^20 = 2^23 steps."""
    _check(*_call(which, [40, 200, 0, 3, 129], H, I, scales=(125, 133)), True)


@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("gap", [(5, 0), (0, 9), (130, 300)])
def test_rows_outside_every_group(which, gap):
    _check(*_call(which, [3, 40, 0, 270], 256, 128, gap=gap), True)


def test_no_group_has_rows():
    _check(*_call("w2", [0, 0, 0], 256, 128, gap=(0, 12)), True)


@pytest.mark.parametrize("lens", [[5, -2, 6, 3], [5, 200], [-1, 5, 8]])
def test_offsets_that_are_no_plan(lens):
    """Decreasing offsets and ones outside the rows: the status word says so, nothing is written."""
    H, I, rows = 128, 128, 12
    d = moe.dims(rows, H, I, len(lens), 1, 0)
    off = torch.tensor([0] + lens, dtype=I32, device=DEV).cumsum(0).to(I32)
    z = lambda *s, dt: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    dx = torch.full((rows, I), 7.0, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    moe.moe_grouped_gemm_w2_backward(d, z(rows, H, dt=BF), off, z(len(lens), H, I // 2, dt=U8),
                                     z(len(lens), H, I // 32, dt=U8), dx, ws)
    assert moe.moe_check_status(ws) == moe.STATUS_BAD_PLAN
    assert torch.all(dx == 7.0)


def test_every_scale_byte_and_code():
    """One-hot rows read single weight rows back: group b has scale byte b in row b % 128.
    Weights below 2^-126 may count as zero (subnormals), values past bf16's range are
    infinities, byte 255 is NaN."""
    H, I, G = 128, 512, 256
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.randint(0, 256, (G, H, I // 2), generator=g, device=DEV).to(U8)
    w[:, :, :8] = torch.arange(8, dtype=U8, device=DEV) * 2 + (torch.arange(8, dtype=U8, device=DEV) * 2 + 1) * 16
    w_s = torch.full((G, H, I // 32), 120, dtype=U8, device=DEV)
    b = torch.arange(G, device=DEV)
    w_s[b, b % H] = b.to(U8)[:, None]
    dy = torch.zeros(G, H, dtype=BF, device=DEV)
    dy[b, b % H] = 1.0
    d = moe.dims(G, H, I, G, 1, 0)
    dx = torch.empty(G, I, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    moe.moe_grouped_gemm_w2_backward(d, dy, torch.arange(G + 1, dtype=I32, device=DEV), w, w_s, dx, ws)
    assert moe.moe_check_status(ws) == 0
    want = ref.mxfp4(w[b, b % H], w_s[b, b % H])
    assert torch.all(torch.isnan(dx[255]))
    got, want = dx[:255].double(), want[:255].to(BF).double()
    small = want.abs() < 2.0 ** -126
    assert torch.equal(got[~small], want[~small])
    assert torch.all((got - want)[small].abs() <= want[small].abs())


def test_non_finite_rows_stay_in_their_rows():
    H, I = 256, 128
    dy, off, w, w_s, dx = _call("w2", [20, 30], H, I)
    bad = dy.clone()
    bad[3, 5], bad[33, 7] = float("nan"), float("inf")
    d = moe.dims(50, H, I, 2, 1, 0)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    out = torch.empty_like(dx)
    moe.moe_grouped_gemm_w2_backward(d, bad, off, w, w_s, out, ws)
    rest = torch.ones(50, dtype=torch.bool, device=DEV)
    rest[[3, 33]] = False
    assert torch.equal(out[rest], dx[rest])
    assert torch.all(torch.isnan(out[3])) and not torch.any(torch.isfinite(out[33]))


def _call_nv(which, lens, H, I, seed=0, ints=True, gs=True):
    """_call with NVFP4 weights.  ints: scales 1, 2, 3 and tensor scales 1, 2 and 1/2: terms are
    multiples of 1/4 up to 2 * 6 * 3 * 2."""
    g = torch.Generator(device=DEV).manual_seed(seed + H + 3 * I + len(lens))
    rows, (C, F), G = sum(lens), (H, I) if which == "w2" else (2 * I, H), len(lens)
    off = torch.tensor([sum(lens[:i]) for i in range(G + 1)], dtype=I32, device=DEV)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
    w = ri(0, 256, G, C, F // 2).to(U8)
    shape = (G,) if which == "w2" else (G, 2)
    if ints:
        dy = ri(-2, 3, rows, C).to(BF)
        w_s = ri(1, 4, G, C, F // 16).float().to(torch.float8_e4m3fn).view(U8)
        t = torch.tensor([0.5, 1.0, 2.0], device=DEV)[ri(0, 3, *shape)]
    else:
        dy = torch.randn(rows, C, generator=g, device=DEV).to(BF)
        w_s = ri(1, 120, G, C, F // 16).to(U8)  # every positive E4M3 value up to 256
        t = torch.rand(*shape, generator=g, device=DEV) + 0.5
    t = t if gs else None
    d = moe.dims(rows, H, I, G, 1, 0)
    dx = torch.full((rows, F), 7.0, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    f = moe.moe_grouped_gemm_w2_backward_nvfp4 if which == "w2" \
        else moe.moe_grouped_gemm_w13_backward_nvfp4
    f(d, dy, off, w, w_s, t, dx, ws)
    assert moe.moe_check_status(ws) == 0
    want, size = ref.expert_grad(dy, off, w, w_s, rows, F, t, True)
    if ints:
        assert torch.equal(dx, want.to(BF))
    else:
        # the scale's product and the halves' sum besides
        tol = ref.U16 * want.abs() + (C / 16 + 3) * 2.0 ** -22 * size
        assert torch.all((dx.double() - want).abs() <= tol)


@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("H,I", [(256, 256), (512, 768), (1280, 256), (4096, 1280), (1280, 2048)])
@pytest.mark.parametrize("ints", [True, False])
def test_nvfp4_group_lengths(which, H, I, ints):
    _call_nv(which, EDGES, H, I, ints=ints)


@pytest.mark.parametrize("which", ["w2", "w13"])
@pytest.mark.parametrize("lens", [[1], [0, 3], [16] * 40, [1] * 300, [2000], [260, 3, 700, 1]])
@pytest.mark.parametrize("gs", [True, False])
def test_nvfp4_few_and_many_groups(which, lens, gs):
    _call_nv(which, lens, 512, 256, gs=gs)


@pytest.mark.parametrize("which", ["w2", "w13"])
def test_nvfp4_layer_sizes(which):
    _call_nv(which, [3, 0, 290, 17, 140, 64], 7168, 2048)
    _call_nv(which, [3, 0, 290, 17, 140, 64], 7168, 2048, ints=False)


def test_nvfp4_every_scale_byte():
    """One-hot rows read single weight rows back: group b has scale byte b in row b (bytes 127 and
    255 are NaN, those from 128 on negative)."""
    H, I, G = 256, 256, 256
    g = torch.Generator(device=DEV).manual_seed(6)
    w = torch.randint(0, 256, (G, H, I // 2), generator=g, device=DEV).to(U8)
    w_s = torch.full((G, H, I // 16), 56, dtype=U8, device=DEV)  # 1.0
    b = torch.arange(G, device=DEV)
    w_s[b, b] = b.to(U8)[:, None]
    dy = torch.zeros(G, H, dtype=BF, device=DEV)
    dy[b, b] = 1.0
    d = moe.dims(G, H, I, G, 1, 0)
    dx = torch.empty(G, I, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    moe.moe_grouped_gemm_w2_backward_nvfp4(d, dy, torch.arange(G + 1, dtype=I32, device=DEV), w, w_s,
                                           None, dx, ws)
    nan = torch.tensor([127, 255], device=DEV)
    assert torch.all(torch.isnan(dx[nan]))
    rest = torch.ones(G, dtype=torch.bool, device=DEV)
    rest[nan] = False
    want = ref.nvfp4(w[b, b][:, None], w_s[b, b][:, None])[:, 0].to(BF)
    assert torch.equal(dx[rest].float(), want[rest].float())


PAIRS = [(1.0, 0.375), (0.375, 1.0), (-3.0, 0.5), (0.5, -3.0), (0.0, 2.5), (2.5, 0.0), (0.0, 0.0),
         (2.0 ** -60, 1.5), (1.5, 2.0 ** -60), (3e30, 1e30), (1e-30, 3e-30)]


@pytest.mark.parametrize("H,I", [(256, 256), (1280, 2048)])
@pytest.mark.parametrize("rows", [1, 31, 128, 129, 200, 257])
def test_nvfp4_w13_halves_of_any_scales(H, I, rows):
    """Tensor scales of either order, sign and size, and none: one or two sums a tile.  Besides the
    sums' steps: the quotient, its product and that with the last scale round once each."""
    g = torch.Generator(device=DEV).manual_seed(rows + H)
    G, C, F = len(PAIRS), 2 * I, H
    off = torch.arange(G + 1, dtype=I32, device=DEV) * rows
    dy = torch.randn(G * rows, C, generator=g, device=DEV).to(BF)
    w = torch.randint(0, 256, (G, C, F // 2), generator=g, device=DEV).to(U8)
    w_s = torch.randint(1, 120, (G, C, F // 16), generator=g, device=DEV).to(U8)
    t = torch.tensor(PAIRS, device=DEV)
    dx = torch.full((G * rows, F), 7.0, dtype=BF, device=DEV)
    d = moe.dims(G * rows, H, I, G, 1, 0)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    moe.moe_grouped_gemm_w13_backward_nvfp4(d, dy, off, w, w_s, t, dx, ws)
    assert moe.moe_check_status(ws) == 0
    want, size = ref.expert_grad(dy, off, w, w_s, G * rows, F, t, True)
    tol = ref.U16 * want.abs() + (C / 16 + 3) * 2.0 ** -22 * size
    assert torch.all((dx.double() - want).abs() <= tol)


@pytest.mark.parametrize("which", ["w2", "w13"])
def test_outputs_are_the_same_in_every_run(which):
    a, b = (_call(which, [100, 3, 600, 40], 1152, 640, ints=False)[4] for _ in range(2))
    assert torch.equal(a, b)


def test_two_streams_and_two_graphs_with_one_workspace():
    """Calls that overlap share a workspace (its status word is all they write there)."""
    H, I, rows = 512, 384, 300
    g = torch.Generator(device=DEV).manual_seed(11)
    off = torch.tensor([0, 100, rows], dtype=I32, device=DEV)
    w = torch.randint(0, 256, (2, H, I // 2), generator=g, device=DEV).to(U8)
    w_s = torch.full((2, H, I // 32), 127, dtype=U8, device=DEV)
    d = moe.dims(rows, H, I, 2, 1, 0)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    dy = [torch.randint(-2, 3, (rows, H), generator=g, device=DEV).to(BF) for _ in range(2)]
    want = [ref.expert_grad(v, off, w, w_s, rows, I)[0].to(BF) for v in dy]
    dx = [torch.empty(rows, I, dtype=BF, device=DEV) for _ in range(2)]
    call = lambda i: moe.moe_grouped_gemm_w2_backward(d, dy[i], off, w, w_s, dx[i], ws)  # noqa: E731
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dx, want))
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            call(i)
    for v in dx:
        v.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dx, want))
    assert moe.moe_check_status(ws) == 0


def test_past_2_31_values():
    """dx of more than 2^31 values; the last rows against float64."""
    rows, H, I = 600000, 128, 3840
    g = torch.Generator(device=DEV).manual_seed(9)
    dy = torch.randint(-2, 3, (rows, H), generator=g, device=DEV).to(BF)
    w = torch.randint(0, 256, (2, H, I // 2), generator=g, device=DEV).to(U8)
    w_s = torch.full((2, H, I // 32), 127, dtype=U8, device=DEV)
    d = moe.dims(rows, H, I, 2, 1, 0)
    dx = torch.empty(rows, I, dtype=BF, device=DEV)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    off = torch.tensor([0, 1000, rows], dtype=I32, device=DEV)
    moe.moe_grouped_gemm_w2_backward(d, dy, off, w, w_s, dx, ws)
    assert moe.moe_check_status(ws) == 0
    for a, b, e in ((0, 1000, 0), (1000, 1300, 1), (rows - 500, rows, 1)):
        want = dy[a:b].double() @ ref.mxfp4(w[e], w_s[e])
        assert torch.equal(dx[a:b], want.to(BF))
