"""Residual + RMS norm (moe_add_rmsnorm) and its gradient against float64, at the widths
where a row changes hands (one warp, one CTA's registers, rows read twice), odd widths,
single rows, and more rows than the gradient has CTAs.

Tolerances: y and h carry one rounding to their type (relative 2^-8 in bf16, 2^-24 in fp32)
on an fp32 value; the sum of a row's squares has at most 64 + cols / 512 roundings on any
path to it, so rstd is within (64 + cols / 512) * 2^-24, relative (half of that from the
root, the rest for its own rounding, the division's and eps)."""

import numpy as np
import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from oracle import moe_oracle as o
from tests import _block_ref as ref
from tests._parity import bits_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
U16, U32 = ref.U16, ref.U32
BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "fp32": F32}

SHAPES = [(1, 1), (3, 8), (1, 128), (7, 7168), (5, 1000), (9, 1023), (40, 256), (1300, 512),
          (2, 2048), (2, 2049), (1, 16384), (2, 16512), (3, 20008), (640, 136)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _data(rows, cols, stream, gain, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + cols)
    x = torch.randn(rows, cols, generator=g).to(BF16).to(DEV)
    r = (torch.randn(rows, cols, generator=g) * 2).to(DT[stream]).to(DEV) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(DT[gain]).to(DEV)
    return x, r, w


def _rstd_tol(cols):
    return (64 + cols / 512) * U32


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream,gain,residual", [("bf16", "bf16", True), ("fp32", "fp32", True),
                                                  ("bf16", "fp32", False),
                                                  ("fp32", "bf16", True)])
def test_forward(rows, cols, stream, gain, residual):
    x, r, w = _data(rows, cols, stream, gain, residual=residual)
    h = torch.empty(rows, cols, dtype=DT[stream], device=DEV)
    y = torch.empty(rows, cols, dtype=BF16, device=DEV)
    rstd = torch.empty(rows, dtype=F32, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, EPS, h=h, y=y, rstd=rstd)
    a64, r64, y64 = ref.norm(_np(x), _np(r) if residual else None, _np(w), EPS)
    tol = _rstd_tol(cols)
    assert np.all(np.abs(_np(rstd) - r64) <= tol * r64)
    # the fp32 sum of x and residual is rounded once before the stream's own rounding
    u = U16 if stream == "bf16" else U32
    assert np.all(np.abs(_np(h) - a64) <= (u + U32) * np.abs(a64))
    assert np.all(np.abs(_np(y) - y64) <= (U16 + 2 * (tol + 4 * U32)) * np.abs(y64) + 1e-38)


@pytest.mark.parametrize("rows,cols", [(1, 128), (7, 7168), (33, 512), (3, 640), (2, 16384),
                                       (1, 16512), (2, 1152)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("with_y", [True, False])
def test_codes_are_those_of_the_bf16_output(rows, cols, stream, with_y):
    x, r, w = _data(rows, cols, stream, "bf16", seed=1)
    x[0, :min(cols, 128)] = 0
    r[0, :min(cols, 128)] = 0       # a block of zeros: scale byte 127
    y = torch.empty(rows, cols, dtype=BF16, device=DEV)
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, cols // 128, dtype=torch.uint8, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, EPS, y=y)
    moe.moe_add_rmsnorm(x, r, w, EPS, y=torch.empty_like(y) if with_y else None, q=q, s=s)
    rq, rs = o.quant_act(bits_np(y))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    moe.moe_quant_act(y, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_outputs_in_the_inputs_buffers():
    for cols in (512, 7168, 1023, 20008):
        x, r, w = _data(6, cols, "bf16", "bf16", seed=2)
        h, y = torch.empty_like(r), torch.empty_like(x)
        moe.moe_add_rmsnorm(x, r, w, EPS, h=h, y=y)
        x2, r2 = x.clone(), r.clone()
        moe.moe_add_rmsnorm(x2, r2, w, EPS, h=r2, y=x2)
        assert torch.equal(h, r2) and torch.equal(y, x2)
        x3 = x.clone()
        moe.moe_add_rmsnorm(x3, r, w, EPS, h=x3, y=torch.empty_like(y))
        assert torch.equal(h, x3)


def test_rows_do_not_meet():
    """An infinity or NaN stays in its row, zeros have a finite norm."""
    for cols in (256, 1000, 7168):
        x, r, w = _data(5, cols, "bf16", "bf16", seed=3)
        clean = torch.empty_like(x)
        moe.moe_add_rmsnorm(x, r, w, EPS, y=clean)
        x[1, 3], x[2, 0] = float("nan"), float("inf")
        x[3], r[3] = 0, 0
        y = torch.empty_like(x)
        moe.moe_add_rmsnorm(x, r, w, EPS, y=y)
        assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2, 0]))
        assert torch.count_nonzero(y[3]).item() == 0


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream,gain,dh_in", [("bf16", "bf16", True), ("fp32", "fp32", True),
                                               ("bf16", "fp32", False), ("fp32", "bf16", False)])
def test_backward(rows, cols, stream, gain, dh_in):
    g = torch.Generator().manual_seed(rows + 13 * cols)
    _, h, w = _data(rows, cols, stream, gain, seed=4)
    dy = torch.randn(rows, cols, generator=g).to(BF16).to(DEV)
    di = torch.randn(rows, cols, generator=g).to(DT[stream]).to(DEV) if dh_in else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dh, dx = torch.empty_like(h), torch.empty_like(dy)
    dg = torch.empty(cols, dtype=F32, device=DEV)
    ws = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(rows, cols))
    ws.fill_(0xA5)
    moe.moe_add_rmsnorm_backward(dy, h, w, rstd, ws, dh_in=di, dh=dh, dx=dx, dgain=dg)
    a = [_np(t) for t in (dy, h, rstd, w)]
    dh64, dg64 = ref.norm_bwd(*a, _np(di) if dh_in else None)
    n = np.abs(a[1] * a[2][:, None])
    u = np.abs(a[0] * a[3])
    size = a[2][:, None] * (u + n * np.mean(u * n, axis=1, keepdims=True))
    size = size + (np.abs(_np(di)) if dh_in else 0)
    # the row's sum has at most 64 + cols / 512 roundings on any path, the rest a few
    tol = (80 + cols / 512) * U32 * size
    assert np.all(np.abs(_np(dx) - dh64) <= tol + U16 * (np.abs(dh64) + tol) + 1e-38)
    u_out = U16 if stream == "bf16" else U32
    assert np.all(np.abs(_np(dh) - dh64) <= tol + u_out * (np.abs(dh64) + tol) + 1e-38)
    # a sum of `rows` fp32 products, whatever its order
    assert np.all(np.abs(_np(dg) - dg64) <= (rows + 8) * U32 * np.sum(np.abs(a[0]) * n, axis=0))
    # the same call gives the same bits; outputs in the inputs' buffers too
    dg2, dh2 = torch.empty_like(dg), di.clone() if dh_in else h.clone()
    moe.moe_add_rmsnorm_backward(dy, h if dh_in else dh2, w, rstd, ws, dh_in=dh2 if dh_in else None,
                                 dh=dh2, dgain=dg2)
    assert torch.equal(dg, dg2) and torch.equal(dh, dh2)


def test_backward_against_differences():
    """Central differences of the float64 forward, fp32 stream: the kernel's rounding is
    some 80 * 2^-24 of the terms, the differences' error of order step^2."""
    rows, cols, step = 3, 24, 1e-5
    _, h, w = _data(rows, cols, "fp32", "fp32", seed=5)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(9)).to(BF16).to(DEV)
    h64, w64, dy64 = _np(h), _np(w), _np(dy)
    rstd = torch.tensor(ref.norm(h64, None, w64, EPS)[1], dtype=F32, device=DEV)
    dh, dg = torch.empty_like(h), torch.empty(cols, dtype=F32, device=DEV)
    ws = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(rows, cols))
    moe.moe_add_rmsnorm_backward(dy, h, w, rstd, ws, dh=dh, dgain=dg)
    f = lambda a, b: float(np.sum(dy64 * ref.norm(a, None, b, EPS)[2]))  # noqa: E731
    for i in range(rows):
        for j in range(cols):
            d = np.zeros_like(h64)
            d[i, j] = step
            assert abs((f(h64 + d, w64) - f(h64 - d, w64)) / (2 * step) - dh[i, j].item()) < 1e-4
    for j in range(cols):
        d = np.zeros_like(w64)
        d[j] = step
        assert abs((f(h64, w64 + d) - f(h64, w64 - d)) / (2 * step) - dg[j].item()) < 1e-4


@pytest.mark.parametrize("cols", [512, 1000, 7168, 1023])
def test_buffers_aligned_to_16_bytes_only(cols):
    """fp32 rows that start at an odd multiple of 16 bytes."""
    def off(t):
        flat = torch.empty(t.numel() + 4, dtype=t.dtype, device=DEV)[4:] if t.dtype is F32 else (
            torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8:])
        flat = flat.view(t.shape)
        flat.copy_(t)
        return flat
    x, r, w = _data(5, cols, "fp32", "fp32", seed=8)
    outs = lambda: (torch.empty_like(r), torch.empty_like(x))  # noqa: E731
    h, y = outs()
    moe.moe_add_rmsnorm(x, r, w, EPS, h=h, y=y)
    h2, y2 = (off(t) for t in outs())
    moe.moe_add_rmsnorm(off(x), off(r), off(w), EPS, h=h2, y=y2)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    ws = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(5, cols))
    dh, dg = torch.empty_like(h), torch.empty(cols, dtype=F32, device=DEV)
    moe.moe_add_rmsnorm_backward(y, h, w, rstd, ws, dh_in=r, dh=dh, dgain=dg)
    dh2, dg2 = off(dh), torch.empty_like(dg)
    moe.moe_add_rmsnorm_backward(off(y), off(h), off(w), rstd, ws, dh_in=off(r), dh=dh2, dgain=dg2)
    assert torch.equal(dh, dh2) and torch.equal(dg, dg2)


def test_no_rows():
    x = torch.empty(0, 256, dtype=BF16, device=DEV)
    w = torch.ones(256, dtype=BF16, device=DEV)
    moe.moe_add_rmsnorm(x, None, w, EPS, y=torch.empty_like(x))
    dg = torch.full((256,), 7.0, dtype=F32, device=DEV)
    ws = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(0, 256))
    moe.moe_add_rmsnorm_backward(x, x, w, torch.empty(0, dtype=F32, device=DEV), ws, dgain=dg)
    assert torch.count_nonzero(dg).item() == 0


def test_on_another_stream():
    x, r, w = _data(64, 7168, "bf16", "bf16", seed=6)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, r, w, EPS, y=y0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(x, r, w, EPS, y=y1, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y0, y1)
    with torch.cuda.stream(st):
        y2 = torch.zeros_like(x)
        moe.moe_add_rmsnorm(x, r, w, EPS, y=y2)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y0, y2)


@pytest.mark.parametrize("cols", [8192, 8191])
def test_offsets_past_32_bits(cols):
    """More than 2^31 values: the last rows come out as in a call of their own."""
    rows = (1 << 31) // cols + 300
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(rows, cols, dtype=BF16, device=DEV).normal_(generator=g)
    w = torch.ones(cols, dtype=BF16, device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, dtype=F32, device=DEV)
    moe.moe_add_rmsnorm(x, None, w, EPS, y=y, rstd=rstd)
    last, y1, r1 = x[-5:].clone(), torch.empty(5, cols, dtype=BF16, device=DEV), rstd[-5:].clone()
    moe.moe_add_rmsnorm(last, None, w, EPS, y=y1)
    assert torch.equal(y[-5:], y1)
    dh, dh1 = torch.empty_like(x), torch.empty_like(last)
    moe.moe_add_rmsnorm_backward(y, x, w, rstd, None, dh=dh)
    moe.moe_add_rmsnorm_backward(y1, last, w, r1, None, dh=dh1)
    assert torch.equal(dh[-5:], dh1)


# Several rows a CTA (a warp) in each form: rows of one warp, of a CTA's registers with two and
# four vectors a thread, and odd widths with four and eight columns a thread.
LONG = [(25000, 256), (4000, 2048), (2000, 7168), (700, 16384), (5000, 1023), (1500, 2049)]


@pytest.mark.parametrize("rows,cols", LONG)
@pytest.mark.parametrize("stream,gain,residual", [("bf16", "fp32", True), ("fp32", "bf16", True),
                                                  ("bf16", "bf16", False)])
def test_forward_of_many_rows(rows, cols, stream, gain, residual):
    test_forward(rows, cols, stream, gain, residual)


@pytest.mark.parametrize("rows,cols", [s for s in LONG if s[1] % 128 == 0])
def test_codes_of_many_rows(rows, cols):
    test_codes_are_those_of_the_bf16_output(rows, cols, "bf16", True)


@pytest.mark.parametrize("rows,cols", LONG)
@pytest.mark.parametrize("stream,dh_in", [("bf16", True), ("bf16", False), ("fp32", True),
                                          ("fp32", False)])
def test_backward_of_many_rows(rows, cols, stream, dh_in):
    test_backward(rows, cols, stream, "bf16", dh_in)
