"""Dense projection (moe_linear) and its gradient against float64: one token to several
hundred and more tiles than the GPU holds, odd sizes and strides, every activation and type.

Two kinds of checks.  Small-integer operands have exact fp32 sums, so the fp32 output has to
be equal and a bf16 output its one rounding: every element is in its place.  Normal operands:
a sum of K products carries at most K roundings (the tensor cores may truncate: 2^-23 each)
of at most the sum of the magnitudes; an activation's slope is at most 1.13 and its value and
slope are within 32 * 2^-24 * (1 + |z|); the output type's rounding comes on top."""

import numpy as np
import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U16, U32 = ref.U16, ref.U32

SHAPES = [(1, 1, 1), (1, 128, 64), (7, 7168, 512), (16, 130, 72), (17, 129, 65), (33, 257, 129),
          (64, 64, 64), (65, 300, 200), (130, 384, 320), (333, 1111, 777), (300, 20000, 64),
          (2600, 2100, 136), (5000, 1024, 1), (256, 7168, 1024), (700, 1984, 2100),
          (600, 1031, 3001)]


def _ints(g, *shape, hi=3):
    return torch.randint(-hi, hi + 1, shape, generator=g, device=DEV).to(BF16)


def _gen(*seed):
    return torch.Generator(device=DEV).manual_seed(sum(s * 1009 ** i for i, s in enumerate(seed)))


def _ws(M, N, K, ldx=0, ldw=0):
    return moe.alloc_workspace(moe.linear_workspace_size(M, N, K, ldx, ldw))


def _act64(z, act):
    return torch.from_numpy(ref.act(z.cpu().numpy(), act)).to(DEV)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("extras", [False, True])
def test_integers_exactly(M, N, K, y_dtype, extras):
    g = _gen(M, N, K)
    x, w = _ints(g, M, K), _ints(g, N, K)
    bias = _ints(g, N, hi=50).float() if extras else None
    res = _ints(g, M, N, hi=100).to(y_dtype) if extras else None
    y, ws = torch.full((M, N), float("nan"), dtype=y_dtype, device=DEV), _ws(M, N, K)
    z = torch.full((M, N), float("nan"), dtype=BF16, device=DEV) if extras else None
    moe.moe_linear(x, w, y, ws, bias=bias, residual=res, z=z, act="relu" if extras else "none")
    want = x.to(F64) @ w.to(F64).t()
    if extras:
        want = want + bias.to(F64)
        assert torch.equal(z, want.float().to(BF16))
        want = want.clamp(min=0) + res.to(F64)
    assert torch.equal(y, want.float().to(y_dtype))
    assert moe.moe_check_status(ws) == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act,bias_dtype,y_dtype", [("none", None, BF16), ("silu", F32, BF16),
                                                    ("gelu", BF16, F32), ("relu", F32, BF16)])
def test_forward(M, N, K, act, bias_dtype, y_dtype):
    g = _gen(M, N, K, 1)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF16)
    w = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(BF16)
    bias = torch.randn(N, generator=g, device=DEV).to(bias_dtype) if bias_dtype else None
    res = torch.randn(M, N, generator=g, device=DEV).to(y_dtype)
    y, z, ws = torch.empty_like(res), torch.empty(M, N, dtype=BF16, device=DEV), _ws(M, N, K)
    moe.moe_linear(x, w, y, ws, bias=bias, residual=res, z=z, act=act)
    z64 = x.to(F64) @ w.to(F64).t()
    size = x.to(F64).abs() @ w.to(F64).abs().t()
    if bias is not None:
        z64 = z64 + bias.to(F64)
    ez = K * 2 * U32 * size + U32 * z64.abs()
    assert bool(((z.to(F64) - z64).abs() <= ez + U16 * (z64.abs() + ez)).all())
    a64 = _act64(z64, act)
    y64 = a64 + res.to(F64)
    e = 1.13 * ez + (0 if act in ("none", "relu") else 32 * U32 * (1 + z64.abs())) + U32 * y64.abs()
    u = U16 if y_dtype is BF16 else U32
    assert bool(((y.to(F64) - y64).abs() <= e + u * (y64.abs() + e)).all())
    # the residual's own buffer as the output, and the same bits again
    moe.moe_linear(x, w, res, ws, bias=bias, residual=res, act=act)
    assert torch.equal(res, y)


@pytest.mark.parametrize("M,N,K", [(5, 200, 96), (70, 136, 72), (300, 264, 200), (1, 40, 24)])
@pytest.mark.parametrize("pad", [8, 3])
def test_row_strides(M, N, K, pad):
    """Every matrix inside a wider one; with stride 3 more, rows are no whole vectors."""
    g = _gen(M, N, K, pad)
    wide = lambda r, c, dt: torch.full((r, c + pad), 5.0, dtype=dt, device=DEV)  # noqa: E731
    x, w, res = wide(M, K, BF16), wide(N, K, BF16), wide(M, N, F32)
    y, z = wide(M, N, F32), wide(M, N, BF16)
    x[:, :K], w[:, :K] = _ints(g, M, K), _ints(g, N, K)
    res[:, :N] = _ints(g, M, N).float()
    ws = _ws(M, N, K, K + pad, K + pad)
    moe.moe_linear(x[:, :K], w[:, :K], y[:, :N], ws, residual=res[:, :N], z=z[:, :N])
    want = x[:, :K].to(F64) @ w[:, :K].to(F64).t()
    assert torch.equal(z[:, :N], want.float().to(BF16))
    assert torch.equal(y[:, :N], (want + res[:, :N].to(F64)).float())
    assert bool((y[:, N:] == 5).all()) and bool((z[:, N:] == 5).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward_integers_exactly(M, N, K):
    g = _gen(M, N, K, 2)
    x, w, dy = _ints(g, M, K), _ints(g, N, K), _ints(g, M, N)
    dx = torch.full((M, K), float("nan"), dtype=BF16, device=DEV)
    dw = torch.full((N, K), float("nan"), dtype=BF16, device=DEV)
    db = torch.full((N,), float("nan"), dtype=F32, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K))
    moe.moe_linear_backward(x, w, dy, ws, dx=dx, dw=dw, dbias=db)
    assert torch.equal(dx, (dy.to(F64) @ w.to(F64)).float().to(BF16))
    assert torch.equal(dw, (dy.to(F64).t() @ x.to(F64)).float().to(BF16))
    assert torch.equal(db, dy.to(F64).sum(0).float())
    # relu with z > 0 where even: dz stays an integer; outputs one at a time
    z = (torch.arange(M * N, device=DEV).view(M, N) % 2 * 2 - 1).to(BF16)
    dz = torch.where(z > 0, dy, torch.zeros_like(dy)).to(F64)
    for kw in (dict(dx=dx), dict(dw=dw), dict(dbias=db)):
        moe.moe_linear_backward(x, w, dy, ws, z=z, act="relu", **kw)
    assert torch.equal(dx, (dz @ w.to(F64)).float().to(BF16))
    assert torch.equal(dw, (dz.t() @ x.to(F64)).float().to(BF16))
    assert torch.equal(db, dz.sum(0).float())
    assert moe.moe_check_status(ws) == 0


@pytest.mark.parametrize("M,N,K", [(7, 64, 96), (130, 72, 200), (333, 111, 77), (2600, 2100, 136)])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_backward(M, N, K, act):
    g = _gen(M, N, K, 3)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, w, z, dy = r(M, K), r(N, K), r(M, N), r(M, N)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K))
    moe.moe_linear_backward(x, w, dy, ws, z=z, act=act, dx=dx, dw=dw, dbias=db)
    z64 = z.to(F64)
    dz = dy.to(F64) * torch.from_numpy(ref.act_slope(z64.cpu().numpy(), act)).to(DEV)
    # the slope's error, then dz's rounding to bf16 as the products' operand
    es = dy.to(F64).abs() * 32 * U32 * (1 + z64.abs())
    ed = es + U16 * (dz.abs() + es)
    for got, a, b, ea in ((dx, dz, w.to(F64), ed), (dw, dz.t(), x.to(F64), ed.t())):
        want = a @ b
        e = ea @ b.abs() + a.shape[1] * 2 * U32 * ((a.abs() + ea) @ b.abs())
        assert bool(((got.to(F64) - want).abs() <= e + U16 * (want.abs() + e)).all())
    eb = es.sum(0) + (M + 8) * U32 * (dz.abs() + es).sum(0)
    assert bool(((db.to(F64) - dz.sum(0)).abs() <= eb).all())


def test_backward_against_differences():
    """Central differences of the float64 forward; the kernel's gradients carry bf16
    roundings of dz and of themselves: at most 2 * 2^-8 of the sum of the terms."""
    M, N, K, step, act = 3, 5, 8, 1e-5, "silu"
    g = _gen(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, w, dy, bias = r(M, K), r(N, K), r(M, N), torch.zeros(N, device=DEV)
    y, z = torch.empty(M, N, dtype=F32, device=DEV), torch.empty(M, N, dtype=BF16, device=DEV)
    moe.moe_linear(x, w, y, _ws(M, N, K), bias=bias, z=z, act=act)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K))
    moe.moe_linear_backward(x, w, dy, ws, z=z, act=act, dx=dx, dw=dw, dbias=db)
    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    a, b, c, gy = n(x), n(w), np.zeros(N), n(dy)
    f = lambda a, b, c: float(np.sum(gy * ref.act(a @ b.T + c, act)))  # noqa: E731
    # z's own rounding moves the slope: |act''| <= 0.5, |z| <= its largest here
    dz = np.abs(gy) * (2 * U16 * 1.1 + 0.5 * U16 * np.abs(a @ b.T).max())
    for got, i, tol in ((dx, 0, dz @ np.abs(b)), (dw, 1, dz.T @ np.abs(a)), (db, 2, dz.sum(0))):
        v = [a, b, c][i]
        for at in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[at] = step
            hi, lo = [a, b, c], [a, b, c]
            hi[i], lo[i] = v + d, v - d
            diff = (f(*hi) - f(*lo)) / (2 * step)
            assert abs(diff - n(got)[at]) <= tol[at] + U16 * abs(diff) + 1e-6


def test_rows_do_not_meet():
    """A NaN in one token's row, or in one feature's weights, stays there."""
    for M, N, K in ((5, 200, 128), (300, 300, 128), (2600, 2100, 72)):
        g = _gen(M)
        x, w = _ints(g, M, K), _ints(g, N, K)
        y0, y1 = (torch.empty(M, N, dtype=BF16, device=DEV) for _ in range(2))
        ws = _ws(M, N, K)
        moe.moe_linear(x, w, y0, ws)
        x[3, 1], w[7, 0] = float("nan"), float("inf")
        moe.moe_linear(x, w, y1, ws)
        keep = torch.ones(M, N, dtype=torch.bool, device=DEV)
        keep[3], keep[:, 7] = False, False
        assert torch.equal(y0[keep], y1[keep]) and bool(torch.isnan(y1[3]).all())


@pytest.mark.parametrize("N", [64, 61])
def test_relu_passes_nothing_where_it_is_off(N):
    """dy of NaN and infinities under z <= 0 reaches no gradient; a NaN in z does."""
    M, K = 70, 96
    g = _gen(M, N, K)
    x, w, dy = _ints(g, M, K), _ints(g, N, K), _ints(g, M, N)
    z = (torch.arange(M * N, device=DEV).view(M, N) % 3 - 1).to(BF16)
    off = z <= 0
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV, dtype=BF16)
    bad = torch.where(off, junk[torch.arange(M * N, device=DEV).view(M, N) % 3], dy)
    dz = torch.where(off, torch.zeros_like(dy), dy).to(F64)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K))
    moe.moe_linear_backward(x, w, bad, ws, z=z, act="relu", dx=dx, dw=dw, dbias=db)
    assert torch.equal(dx, (dz @ w.to(F64)).float().to(BF16))
    assert torch.equal(dw, (dz.t() @ x.to(F64)).float().to(BF16))
    assert torch.equal(db, dz.sum(0).float())
    z[3, 5] = float("nan")
    moe.moe_linear_backward(x, w, dy, ws, z=z, act="relu", dx=dx, dw=dw, dbias=db)
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isnan(dw[5]).all())
    assert torch.nonzero(torch.isnan(db)).flatten().tolist() == [5]


def test_no_rows():
    w = torch.ones(64, 32, dtype=BF16, device=DEV)
    x, y = torch.empty(0, 32, dtype=BF16, device=DEV), torch.empty(0, 64, dtype=BF16, device=DEV)
    moe.moe_linear(x, w, y, _ws(0, 64, 32))
    dw, db = torch.ones_like(w), torch.ones(64, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(0, 64, 32))
    moe.moe_linear_backward(x, w, y, ws, dw=dw, dbias=db)
    assert torch.count_nonzero(dw).item() == 0 and torch.count_nonzero(db).item() == 0


def test_on_another_stream():
    g = _gen(5)
    x, w = _ints(g, 9, 512), _ints(g, 640, 512)
    y, ws = torch.empty(9, 640, dtype=F32, device=DEV), _ws(9, 640, 512)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(x, w, y, ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y, (x.to(F64) @ w.to(F64).t()).float())


@pytest.mark.parametrize("N", [8192, 8191])
def test_offsets_past_32_bits(N):
    """More than 2^31 outputs: first, middle and last rows exactly."""
    M, K = (1 << 31) // N + 300, 40
    g = _gen(N)
    x, w = _ints(g, M, K), _ints(g, N, K)
    y, ws = torch.empty(M, N, dtype=BF16, device=DEV), _ws(M, N, K)
    moe.moe_linear(x, w, y, ws)
    for r in (slice(0, 7), slice(M // 2, M // 2 + 7), slice(M - 7, M)):
        assert torch.equal(y[r], (x[r].to(F64) @ w.to(F64).t()).float().to(BF16))
    dx, db = torch.empty_like(x), torch.empty(N, dtype=F32, device=DEV)
    wb = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K, act="none"))
    moe.moe_linear_backward(x, w, y, wb, dx=dx, dbias=db)
    r = slice(M - 7, M)
    want = y[r].to(F64) @ w.to(F64)
    e = N * 2 * U32 * (y[r].to(F64).abs() @ w.to(F64).abs())
    assert bool(((dx[r].to(F64) - want).abs() <= e + U16 * (want.abs() + e)).all())
    assert moe.moe_check_status(ws) == 0 and moe.moe_check_status(wb) == 0


# Every (tile, parts of the contraction) that the cost model chooses, of the split kernel
# (16 to 128 tokens a tile) and of SM pairs (one or two pairs a tile), for whole and ragged rows.
FORWARD = [(1, 8, 65), (1, 16, 74), (1, 8, 3426), (1, 16, 3360),                  # 16 tokens
           (20, 2048, 7168), (31, 2048, 7168), (4966, 8, 10), (5062, 16, 11),     # 32
           (624, 438, 359), (399, 656, 384), (610, 145, 423), (611, 176, 400),
           (230, 152, 4028), (439, 16, 3856),
           (5011, 132, 10), (980, 541, 742), (623, 944, 736), (392, 688, 688),    # 64
           (319, 328, 5391), (471, 144, 5840),
           (518, 6639, 16), (514, 6544, 32), (864, 816, 1184), (737, 518, 5091),  # 128
           (579, 688, 5056),
           (1288, 1327, 648), (300, 7001, 1100)]                                  # two pairs
BACKWARD = [(5034, 16, 390), (4886, 16, 144), (808, 1152, 1360),                  # dx: pairs
            (1, 66, 8), (1, 3454, 8), (4966, 8, 10), (5016, 8, 16),               # 16 and 32 tokens
            (488, 353, 514), (847, 336, 288), (409, 421, 278), (422, 400, 272),
            (209, 3929, 137), (255, 3856, 144),
            (4925, 14, 135), (1003, 720, 528), (636, 656, 448), (300, 5389, 334),  # 64
            (529, 11, 6648), (513, 16, 6672), (1131, 1232, 544), (639, 4695, 773),  # 128
            (707, 5184, 528),
            (849, 1570, 907), (1045, 917, 1184), (5000, 512, 520),                # dw: two pairs
            (1, 8, 16), (202, 8, 16), (2823, 16, 16),                             # 64
            (9, 6515, 513), (262, 68, 4947), (211, 80, 8288), (5393, 847, 385),   # 128
            (4676, 608, 816)]


@pytest.mark.parametrize("M,N,K", FORWARD)
@pytest.mark.parametrize("y_dtype", [BF16, F32])
def test_integers_exactly_on_every_tile(M, N, K, y_dtype):
    for extras in (False, True):
        test_integers_exactly(M, N, K, y_dtype, extras)


@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_backward_integers_exactly_on_every_tile(M, N, K):
    test_backward_integers_exactly(M, N, K)


EXTREMES = [float("inf"), -float("inf"), float("nan"), 3.3e38, -3.3e38, 1.8e19, -1.8e19, 200.0,
            -200.0, 100.0, -100.0, -89.0, -88.0, -87.0, -20.0, -6.0, 1e-38, -1e-38, 0.0, -0.0]


@pytest.mark.parametrize("M,N", [(3, 40), (3, 37), (2600, 2048), (2600, 2050)])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_activations_of_extreme_values(M, N, act):
    """Values as the formulas have them in fp32: finite for every finite z; -inf gives NaN in
    silu and gelu (infinity times 0), +inf stays."""
    z = torch.tensor((EXTREMES * (N // len(EXTREMES) + 1))[:N], device=DEV).to(BF16)
    x, w = torch.zeros(M, 8, dtype=BF16, device=DEV), torch.zeros(N, 8, dtype=BF16, device=DEV)
    x[:, 0], w[:, 0] = 1, z
    y = torch.empty(M, N, dtype=F32, device=DEV)
    moe.moe_linear(x, w, y, _ws(M, N, 8), act=act)
    z64 = z.to(F64)
    want = {"relu": z64.clamp(min=0), "silu": z64 / (1 + torch.exp(-z64)),
            "gelu": 0.5 * z64 * (1 + torch.erf(z64 * 0.5 ** 0.5))}[act]
    assert bool((y == y[:1]).logical_or(torch.isnan(y) & torch.isnan(y[:1])).all())
    assert torch.equal(torch.isnan(y[0]), torch.isnan(want))
    ok = torch.isfinite(want)
    assert torch.equal(y[0][~ok & ~torch.isnan(want)].to(F64), want[~ok & ~torch.isnan(want)])
    e = 32 * U32 * (1 + z64.abs())
    assert bool(((y[0].to(F64) - want).abs() <= e)[ok].all())


@pytest.mark.parametrize("N", [40, 37])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_of_extreme_values(N, act):
    """One token with dy = 1: dbias is the slope; silu's and gelu's of an infinite z are NaN."""
    z = torch.tensor((EXTREMES * 2)[:N], device=DEV).to(BF16).view(1, N)
    dy, x, w = torch.ones_like(z), torch.zeros(1, 8, dtype=BF16, device=DEV), torch.zeros(
        N, 8, dtype=BF16, device=DEV)
    db = torch.empty(N, device=DEV)
    ws = moe.alloc_workspace(moe.linear_backward_workspace_size(1, N, 8))
    moe.moe_linear_backward(x, w, dy, ws, z=z, act=act, dbias=db)
    z64 = z[0].to(F64)
    want = torch.from_numpy(ref.act_slope(z64.cpu().numpy(), act)).to(DEV)
    if act == "relu":
        want[torch.isnan(z64)] = float("nan")
    bad = torch.isnan(z64) if act == "relu" else ~torch.isfinite(z64)
    assert torch.equal(torch.isnan(db), bad)
    e = 32 * U32 * (1 + z64.abs())
    assert bool(((db.to(F64) - want).abs() <= e)[~bad].all())
