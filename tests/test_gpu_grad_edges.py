"""The layer's gradient where fp32's range ends: NVFP4 tensor scales that are large, infinite or
NaN, and SwiGLU's gradient where the product of its factors leaves fp32's range on the way."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _grad_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
NAN, INF = float("nan"), float("inf")


def _nvfp4(which, H, I, rows, ctas, t):
    """dx of groups of `rows` rows whose tensor scales are t, by `ctas` CTAs a tile.  dy is -2 .. 2
    steps of 2^-14 and the block scales 1, 2 or 3: the sums are exact in fp32 (multiples of 2^-15, of
    2 I <= 4096 terms up to 2^-14 * 36 below 9)."""
    g = torch.Generator(device=DEV).manual_seed(rows + H)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
    G, (C, F) = len(t), (H, I) if which == "w2" else (2 * I, H)
    off = torch.arange(G + 1, dtype=I32, device=DEV) * rows
    dy = (ri(-2, 3, G * rows, C) * 2.0 ** -14).to(BF)
    w = ri(0, 256, G, C, F // 2).to(U8)
    w_s = ri(1, 4, G, C, F // 16).float().to(torch.float8_e4m3fn).view(U8)
    dx = torch.full((G * rows, F), 7.0, dtype=BF, device=DEV)
    d = moe.dims(G * rows, H, I, G, 1, 0)
    ws = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    moe.moe_gemm_backward_form(d, 2 if which == "w2" else 13, ctas, dy, off, w, w_s, dx, ws, t, True)
    assert moe.moe_check_status(ws) == 0
    return dy, off, w, w_s, dx


def _agrees(dy, off, w, w_s, t, dx):
    """The formula's value, rounded to bf16, where it is finite: half a step, 2^-22 of the halves'
    magnitudes for each step of 16 of a half that is summed onto the multiplied other one (each
    half by itself is exact), and 2^-22 for the scales' quotient, its product and that with the
    last scale.  Else the same infinity, or NaN."""
    want, size = 0.0, 0.0
    parts = 1 if t.ndim == 1 else 2  # (the scales multiply the sums: 0 times an infinite one is NaN)
    rows, C = dx.shape[0] // len(t), dy.shape[1] // parts
    for p in range(parts):
        c = slice(p * C, (p + 1) * C)
        total, m = ref.expert_grad(dy[:, c], off, w[:, c], w_s[:, c], *dx.shape, nv=True)
        scale = t.view(len(t), parts)[:, p].double().repeat_interleave(rows)[:, None]
        want, size = want + scale * total, size + scale.abs() * m
    got, fine = dx.double(), torch.isfinite(want)
    tol = ref.U16 * want.abs() + (dy.shape[1] / 16 + 3) * 2.0 ** -22 * size
    assert torch.all((got - want).abs()[fine] <= tol[fine])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])


BIG = 2.0 ** 122
# (pairs have two sums of W13's halves a tile up to 128 rows, above that one)
SHAPES = [(256, 256, 100, 1), (256, 256, 100, 2), (256, 256, 200, 2), (1280, 2048, 200, 1),
          (1280, 2048, 200, 2)]


@pytest.mark.parametrize("H,I,rows,ctas", SHAPES)
def test_w13_tensor_scales_that_are_nan(H, I, rows, ctas):
    t = torch.tensor([(NAN, 0.0), (0.0, NAN), (NAN, 1.0), (1.0, NAN), (NAN, NAN), (NAN, INF),
                      (-INF, NAN), (1.0, 0.5)], device=DEV)
    dx = _nvfp4("w13", H, I, rows, ctas, t)[-1].view(len(t), -1)
    assert torch.all(torch.isnan(dx[:-1])) and torch.all(torch.isfinite(dx[-1]))


@pytest.mark.parametrize("H,I,rows,ctas", SHAPES)
def test_w13_tensor_scales_that_are_infinite(H, I, rows, ctas):
    t = torch.tensor([(INF, 0.5), (0.5, -INF), (-INF, 1.5), (0.375, INF), (1.0, 0.5)], device=DEV)
    dy, off, w, w_s, dx = _nvfp4("w13", H, I, rows, ctas, t)
    _agrees(dy, off, w, w_s, t, dx)


@pytest.mark.parametrize("H,I,rows,ctas", SHAPES)
def test_w13_tensor_scales_that_are_large(H, I, rows, ctas):
    t = torch.tensor([(BIG, 1.0), (1.0, -BIG), (BIG, BIG), (-BIG, 2.0 ** 100), (2.0 ** 60, BIG),
                      (2.0 ** 120, 2.0 ** 121), (1.0, 1.0)], device=DEV)
    dy, off, w, w_s, dx = _nvfp4("w13", H, I, rows, ctas, t)
    assert torch.all(torch.isfinite(dx))
    _agrees(dy, off, w, w_s, t, dx)


@pytest.mark.parametrize("H,I,rows,ctas", SHAPES)
def test_w2_tensor_scales_of_every_kind(H, I, rows, ctas):
    t = torch.tensor([BIG, -BIG, 2.0 ** 121, NAN, INF, -INF, 1.0, 0.0, 2.0 ** -100], device=DEV)
    dy, off, w, w_s, dx = _nvfp4("w2", H, I, rows, ctas, t)
    _agrees(dy, off, w, w_s, t, dx)


GATES = [0.0, 1.5, -1.2785, 20, -20, -60, 60, -80, 87, -87, 88, -88, -100, 1000, -1000, 2e38, -2e38]
ROWS = [(u, dh) for u in (3e38, -1e30, 1e20, 1.0, 1e-30) for dh in (3e38, 1e20, -1e30, 0.5, 1e-38)]


@pytest.mark.parametrize("form", ["bf16", "codes"])
def test_swiglu_factors_whose_product_is_past_fp32(form):
    """|d u| up to 1e77.  Where the formula's value fits bf16 the gradient is finite and within the
    bound of the kernel's other tests: a sigmoid below 2^-126 may count as 0, and (|g| + 16) * 2^-22
    covers the sigmoid's error and the products behind it."""
    I = 128
    gates = GATES if form == "bf16" else GATES[:-2]  # (one scale for a row's gates)
    y13 = torch.empty(len(ROWS), 2 * I, dtype=BF, device=DEV)
    y13[:, :I] = torch.tensor(gates, device=DEV).repeat(I)[:I]
    y13[:, I:] = torch.tensor([u for u, _ in ROWS], device=DEV)[:, None]
    dh = torch.tensor([d for _, d in ROWS], device=DEV).to(BF)[:, None].repeat(1, I).contiguous()
    dy = torch.empty_like(y13)
    if form == "bf16":
        moe.moe_swiglu_backward(dh, dy, y13=y13)
        y = y13.double()
    else:
        yq, ys = (torch.empty(len(ROWS), n, dtype=U8, device=DEV) for n in (2 * I, 2 * I // 128))
        moe.moe_quant_act(y13, yq, ys)
        moe.moe_swiglu_backward(dh, dy, yq=yq, ys=ys)
        y = ref.fp8_values(yq, ys)
    g, u, d = y[:, :I], y[:, I:], dh.double()
    dg, du, scale = ref.swiglu_bwd(g, u, d)
    c, tiny = (g.abs() + 16) * 2.0 ** -22, d.abs() * (1 + g.abs()) * 2.0 ** -126
    most = torch.finfo(BF).max
    for got, want, tol in ((dy[:, :I], dg, ref.U16 * dg.abs() + c * scale + u.abs() * tiny),
                           (dy[:, I:], du, (ref.U16 + c) * du.abs() + tiny)):
        tol = tol + 2.0 ** -126
        fits, past = want.abs() + tol <= most, want.abs() - tol > most * (1 + ref.U16)
        assert torch.all(torch.isfinite(got[fits].float()))
        assert torch.all((got.double() - want).abs()[fits] <= tol[fits])
        assert torch.equal(got[past].double(), torch.sign(want[past]) * INF)
