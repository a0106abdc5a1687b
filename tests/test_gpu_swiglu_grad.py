"""moe_swiglu_quant_save against the calls it joins (bit for bit) and moe_swiglu_backward
against float64: every width's end in a CTA, both forms of the input, weights and their
gradient, extreme gates.

Tolerances.  e^-g by ex2.approx of a rounded argument: relative (|g| + 4) * 2^-23; the sigmoid
adds a quotient of 2 units: with the products behind it c = (|g| + 16) * 2^-22 covers each
factor.  dg = d u (s + silu (1 - s)): c times |d u| (s + |silu|), and half a step of bf16,
2^-8 |dg|; where e^-g overflows or is above 2^126 the sigmoid is 0 for less than 2^-126, that
is |d u| (1 + |g|) 2^-126.  dw: 16 * 4 products of a thread, 5 shuffles, 16 warps: 96 * 2^-24 of
the terms' magnitudes."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _grad_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

SHAPES = [(1, 128), (7, 384), (300, 640), (33, 2048), (65, 4096), (5, 8320), (2, 16512), (9, 512),
          (1000, 256), (3, 32768)]


def _y13(rows, I, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + I)
    y = torch.randn(rows, 2 * I, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    return y.to(BF).to(DEV), g


def _save(y13):
    rows, I = y13.shape[0], y13.shape[1] // 2
    new = lambda c: torch.full((rows, c), 0x5A, dtype=U8, device=DEV)  # noqa: E731
    out = dict(hq=new(I), hs=new(I // 128), yq=new(2 * I), ys=new(2 * I // 128))
    moe.moe_swiglu_quant_save(y13, **out)
    return out


@pytest.mark.parametrize("rows,I", SHAPES)
def test_save_is_the_two_quantisations(rows, I):
    y13, _ = _y13(rows, I)
    if rows > 2:
        y13[1] = 0
        y13[2, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], dtype=BF)
        y13[2, I:I + 4] = y13[2, :4].flip(0)
    s = _save(y13)
    hq, hs, yq, ys = (torch.empty_like(s[n]) for n in ("hq", "hs", "yq", "ys"))
    moe.moe_swiglu_quant(y13, hq, hs)
    moe.moe_quant_act(y13, yq, ys)
    assert torch.equal(s["yq"], yq) and torch.equal(s["ys"], ys)
    assert torch.equal(s["hq"], hq) and torch.equal(s["hs"], hs)


def _weights(rows, k, shared, g):
    """perm_src, w, dw of the first T k of the rows."""
    T = rows // (k + shared)
    perm = torch.randperm(T * k, generator=g).to(I32).to(DEV)
    return perm, torch.rand(T, k, generator=g).to(DEV), torch.full((T, k), 7.0, device=DEV)


def _check(g, u, dh, wr, dy13, want_h=None, dw=None, perm=None, h_err=0.0):
    d = dh.double() * wr[:, None]
    dg, du, scale = ref.swiglu_bwd(g, u, d)
    I = g.shape[1]
    c = (g.abs() + 16) * 2.0 ** -22
    tiny = d.abs() * (1 + g.abs()) * 2.0 ** -126
    got = dy13.double()
    # (and the outputs' own smallest step, bf16's and fp32's subnormals)
    assert torch.all((got[:, :I] - dg).abs() <=
                     ref.U16 * dg.abs() + c * scale + (1 + u.abs()) * tiny + 2.0 ** -126)
    assert torch.all((got[:, I:] - du).abs() <= (ref.U16 + c) * du.abs() + tiny + 2.0 ** -126)
    if dw is not None:
        R = perm.numel()
        terms = dh.double()[:R] * want_h[:R]
        tol = (96 * ref.U32 * terms.abs() + h_err[:R] * dh.double()[:R].abs()).sum(1) + 2.0 ** -126
        at = dw.view(-1)[perm.long()].double()
        assert torch.all((at - terms.sum(1)).abs() <= tol)


@pytest.mark.parametrize("rows,I", SHAPES)
@pytest.mark.parametrize("form", ["codes", "codes, h", "bf16", "bf16, h", "in place"])
@pytest.mark.parametrize("weights", ["none", "w", "dw", "both"])
def test_backward(rows, I, form, weights):
    y13, gen = _y13(rows, I, 1)
    s = _save(y13)
    dh = (torch.randn(rows, I, generator=gen) * 0.3).to(BF).to(DEV)
    k, sh = (3, 1) if rows >= 4 else (1, 0)
    perm, w, dw = _weights(rows, k, sh, gen)
    if weights in ("none", "dw"):
        w = None
    if weights in ("none", "w"):
        dw = None
    if weights == "none":
        perm = None
    codes = form.startswith("codes")
    y = ref.fp8_values(s["yq"], s["ys"]) if codes else y13.double()
    g, u = y[:, :I].clone(), y[:, I:].clone()
    given = form.endswith("h")
    h = ref.fp8_values(s["hq"], s["hs"]) if given else g * ref.sigmoid(g) * u
    h_err = torch.zeros_like(g) if given else (g.abs() + 16) * 2.0 ** -22 * h.abs() + \
        (g * u).abs() * 2.0 ** -126
    wr = torch.ones(rows, dtype=torch.float64, device=DEV)
    if w is not None:
        wr[:perm.numel()] = w.double().view(-1)[perm.long()]
    dy13 = y13 if form == "in place" else torch.empty_like(y13)
    src = dict(yq=s["yq"], ys=s["ys"]) if codes else dict(y13=y13)
    if given:
        src |= dict(hq=s["hq"], hs=s["hs"])
    moe.moe_swiglu_backward(dh, dy13, perm_src=perm, w=w, dw=dw, **src)
    _check(g, u, dh, wr, dy13, h, dw, perm, h_err)


def test_extreme_gates():
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 60, -60, 87, -87, 87.5, -87.5, 88, -88, 90,
                      -90, 100, -100, 1000, -1000, 3e38, -3e38, 1.2785, -1.2785])
    I = 128
    g = v.repeat(6)[:I].to(BF).to(DEV)
    y13 = torch.empty(5, 2 * I, dtype=BF, device=DEV)
    y13[:, :I] = g
    y13[:, I:] = torch.tensor([1.0, -2.0, 0.0, 2.0 ** -100, 1e-38], device=DEV)[:, None]
    dh = torch.full((5, I), 0.5, dtype=BF, device=DEV)
    dy13 = torch.empty_like(y13)
    moe.moe_swiglu_backward(dh, dy13, y13=y13)
    y = y13.double()
    assert torch.all(torch.isfinite(dy13.float()))
    _check(y[:, :I], y[:, I:], dh, torch.ones(5, dtype=torch.float64, device=DEV), dy13)


def test_rows_without_a_slot():
    """A row whose perm_src is no slot has weight 1 and no dw; other entries are untouched."""
    rows, I = 6, 256
    y13, gen = _y13(rows, I, 2)
    dh = torch.randn(rows, I, generator=gen).to(BF).to(DEV)
    perm = torch.tensor([4, -1, 0, 5, 2 ** 31 - 1], dtype=I32, device=DEV)
    w, dw = torch.full((5,), 2.0, device=DEV), torch.full((5,), 7.0, device=DEV)
    dy, one = torch.empty_like(y13), torch.empty_like(y13)
    moe.moe_swiglu_backward(dh, dy, y13=y13, perm_src=perm, w=w, dw=dw)
    moe.moe_swiglu_backward(dh, one, y13=y13)
    two = torch.tensor([True, False, True, False, False, False], device=DEV)
    assert torch.equal(dy[~two], one[~two])
    assert torch.all((dy[two].double() - 2 * one[two].double()).abs() <=
                     2 * ref.U16 * 2 * one[two].double().abs())
    assert dw[1:4].tolist() == [7.0, 7.0, 7.0] and dw[0] != 7.0 and dw[4] != 7.0


def test_no_rows():
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    moe.moe_swiglu_quant_save(e(0, 256), e(0, 128, dt=U8), e(0, 1, dt=U8), e(0, 256, dt=U8),
                              e(0, 2, dt=U8))
    moe.moe_swiglu_backward(e(0, 128), e(0, 256), y13=e(0, 256))


def test_difference_quotients():
    """dg and du of the kernel against central differences of sum(dh silu(g) u) in float64."""
    rows, I = 3, 128
    y13, gen = _y13(rows, I, 3)
    y13.clamp_(-6, 6)
    dh = torch.randn(rows, I, generator=gen).to(BF).to(DEV)
    dy = torch.empty_like(y13)
    moe.moe_swiglu_backward(dh, dy, y13=y13)
    y, eps = y13.double(), 1e-5

    def f(v):
        return dh.double() * v[:, :I] * ref.sigmoid(v[:, :I]) * v[:, I:]
    for half in (0, 1):
        step = torch.zeros_like(y)
        step[:, half * I:(half + 1) * I] = eps
        quot = (f(y + step) - f(y - step)) / (2 * eps)
        got = dy.double()[:, half * I:(half + 1) * I]
        # difference error: eps^2 f''' / 6 and float64 rounding / eps, both below 1e-8 here
        assert torch.all((got - quot).abs() <= ref.U16 * quot.abs() + 1e-4 * dh.double().abs() + 1e-8)


def test_past_2_31_values():
    rows, I = 270000, 4096
    y13 = torch.empty(rows, 2 * I, dtype=BF, device=DEV).normal_()
    s = _save(y13)
    dh = torch.empty(rows, I, dtype=BF, device=DEV).normal_()
    perm = torch.arange(rows, dtype=I32, device=DEV).flip(0).contiguous()
    w, dw = torch.rand(rows, device=DEV), torch.empty(rows, device=DEV)
    dy13 = torch.empty_like(y13)
    moe.moe_swiglu_backward(dh, dy13, yq=s["yq"], ys=s["ys"], hq=s["hq"], hs=s["hs"], perm_src=perm,
                            w=w, dw=dw)
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device=DEV)
    small = _save(y13[at].contiguous())
    for n in s:
        assert torch.equal(s[n][at], small[n])
    y = ref.fp8_values(small["yq"], small["ys"])
    h = ref.fp8_values(small["hq"], small["hs"])
    _check(y[:, :I], y[:, I:], dh[at], w.double()[perm[at].long()], dy13[at], h,
           dw[perm[at].long()], torch.arange(5, device=DEV), torch.zeros_like(h))
