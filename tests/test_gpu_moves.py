"""moe_dispatch, its gradient and the combine's gradient against float64: single tokens, k = 1
and 16, every way a row's columns end in a CTA, dropped slots, in-place buffers.

Tolerances: copies are equal; a sum of n terms in fp32 is within n * 2^-24 of the sum of their
magnitudes, its rounding to bf16 within 2^-8 of the value; a dot over H goes through at most
8 * 4 products of a thread, 5 shuffles and 16 warps (53 roundings: 64 * 2^-24)."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _grad_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _routing(T, k, seed=0, drop=0.0):
    """inv as a random permutation of the rows, some slots without one."""
    g = torch.Generator().manual_seed(seed + 17 * T + k)
    inv = torch.randperm(T * k, generator=g).to(I32)
    if drop:
        gone = torch.rand(T * k, generator=g) < drop
        out = torch.tensor([-1, T * k, -2 ** 31, 2 ** 31 - 1, T * k + T - 1], dtype=torch.int64)
        pick = out[torch.randint(0, 5, (T * k,), generator=g)].to(I32)
        inv = torch.where(gone, pick, inv)
    return inv.to(DEV), g


def _rand(g, *s, dtype=BF):
    return torch.randn(*s, generator=g).to(dtype).to(DEV)


# T, H, k, shared, dropped
CASES = [(1, 128, 1, 0, 0), (1, 7168, 8, 1, 0), (7, 7168, 8, 1, 0), (3, 128, 16, 1, 0.5),
         (333, 640, 3, 0, 0.3), (64, 4096, 2, 1, 0), (65, 4224, 5, 1, 0.1), (5, 8320, 7, 0, 0),
         (2, 16512, 4, 1, 0), (1000, 384, 6, 1, 1.0), (257, 1152, 15, 0, 0), (9, 32768, 2, 1, 0)]


@pytest.mark.parametrize("T,H,k,sh,drop", CASES)
def test_dispatch(T, H, k, sh, drop):
    d = moe.dims(T, H, 128, 16, k, sh)
    inv, g = _routing(T, k, drop=drop)
    x = _rand(g, T, H)
    x.view(-1)[0] = float("nan")
    Rs = T * (k + sh)
    xp = torch.full((Rs, H), 7.0, dtype=BF, device=DEV)
    want = xp.clone()
    at, rows = ref.slots(inv, T * k)
    want[rows] = x[at // k]
    if sh:
        want[T * k:] = x
    moe.moe_dispatch(d, x, inv, xp)
    assert torch.equal(xp.view(torch.int16), want.view(torch.int16))  # rows of no slot: as before


@pytest.mark.parametrize("T,H,k,sh,drop", CASES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("more", ["none", "own", "in place"])
def test_dispatch_backward(T, H, k, sh, drop, dt, more):
    d = moe.dims(T, H, 128, 16, k, sh)
    inv, g = _routing(T, k, 1, drop)
    dxp = _rand(g, T * (k + sh), H)
    dx_in = None if more == "none" else _rand(g, T, H, dtype=dt)
    want, size = ref.dispatch_bwd(dxp, inv, T, k, T * k, sh, dx_in)
    dx = dx_in if more == "in place" else torch.full((T, H), 7.0, dtype=dt, device=DEV)
    moe.moe_dispatch_backward(d, dxp, inv, dx, dx_in=dx_in)
    tol = (k + 2) * ref.U32 * size + (ref.U16 * want.abs() if dt is BF else 0)
    assert torch.all((dx.double() - want).abs() <= tol * 1.001)


def test_dispatch_backward_does_not_read_rows_without_a_slot():
    T, H, k = 6, 256, 2
    d = moe.dims(T, H, 128, 4, k, 0)
    inv = torch.arange(T * k, dtype=I32, device=DEV)
    inv[3] = -1
    dxp = torch.ones(T * k, H, dtype=BF, device=DEV)
    dxp[3] = float("nan")
    dx = torch.empty(T, H, dtype=BF, device=DEV)
    moe.moe_dispatch_backward(d, dxp, inv, dx)
    assert torch.equal(dx[:, 0], torch.tensor([2, 1, 2, 2, 2, 2], dtype=BF, device=DEV))


@pytest.mark.parametrize("T,H,k,sh,drop", CASES)
@pytest.mark.parametrize("what", ["both", "dy2", "dw", "in place"])
def test_combine_backward(T, H, k, sh, drop, what):
    d = moe.dims(T, H, 128, 16, k, sh)
    inv, g = _routing(T, k, 2, drop)
    dout, y2 = _rand(g, T, H), _rand(g, T * (k + sh), H)
    w = torch.rand(T, k, generator=g).to(DEV)
    at, rows = ref.slots(inv, T * k)
    do = dout.double()[at // k]
    want = torch.full((T * (k + sh), H), 7.0, dtype=torch.float64, device=DEV)
    want[rows] = do * w.double().view(-1)[at, None]
    if sh:
        want[T * k:] = dout.double()
    dots = torch.zeros(2, T * k, dtype=torch.float64, device=DEV)
    prod = do * y2.double()[rows]
    dots[0, at], dots[1, at] = prod.sum(1), prod.abs().sum(1)
    dy2 = torch.full((T * (k + sh), H), 7.0, dtype=BF, device=DEV) if what != "dw" else None
    if what == "in place":
        keep = torch.ones(T * (k + sh), dtype=torch.bool, device=DEV)
        keep[rows] = False
        keep[T * k:] = False
        want[keep] = y2.double()[keep]
        dy2 = y2
    dw = torch.full((T, k), 7.0, device=DEV) if what != "dy2" else None
    moe.moe_combine_backward(d, dout, y2 if dw is not None else None, inv,
                             w if dy2 is not None else None, dy2=dy2, dw=dw)
    if dy2 is not None:
        assert torch.all((dy2.double() - want).abs() <= (ref.U16 + 2 * ref.U32) * want.abs())
    if dw is not None:
        assert torch.all((dw.double().view(-1) - dots[0]).abs() <= 64 * ref.U32 * dots[1])


def test_past_2_31_values():
    T, H, k = 40000, 7168, 8
    d = moe.dims(T, H, 128, 16, k, 0)
    inv = torch.arange(T * k, dtype=I32, device=DEV).flip(0).contiguous()
    x = torch.randn(T, H, device=DEV).to(BF)
    xp = torch.empty(T * k, H, dtype=BF, device=DEV)
    moe.moe_dispatch(d, x, inv, xp)
    for t in (0, 1, T // 2, T - 1):
        for j in (0, k - 1):
            assert torch.equal(xp[inv[t * k + j].item()], x[t])
    dx = torch.empty_like(x)
    moe.moe_dispatch_backward(d, xp, inv, dx)
    assert torch.equal(dx, (8 * x.float()).to(BF))
    w, dw = torch.full((T, k), 0.5, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_combine_backward(d, x, xp, inv, w, dy2=xp, dw=dw)
    assert torch.equal(xp[inv[T * k - 1].item()], (0.5 * x[T - 1].float()).to(BF))
    assert torch.equal(xp[inv[0].item()], (0.5 * x[0].float()).to(BF))
    rows = torch.tensor([0, T - 1], device=DEV)
    sq = x[rows].double().square().sum(1, keepdim=True)
    assert torch.all((dw[rows].double() - sq).abs() <= 64 * ref.U32 * sq)


def test_outputs_are_the_same_in_every_run():
    T, H, k = 300, 1152, 6
    d = moe.dims(T, H, 128, 16, k, 1)
    inv, g = _routing(T, k, 3)
    dout, y2 = _rand(g, T, H), _rand(g, T * (k + 1), H)
    w = torch.rand(T, k, generator=g).to(DEV)
    runs = []
    for _ in range(2):
        dw, dx = torch.empty(T, k, device=DEV), torch.empty(T, H, dtype=F32, device=DEV)
        moe.moe_combine_backward(d, dout, y2, inv, w, dw=dw)
        moe.moe_dispatch_backward(d, y2, inv, dx)
        runs.append((dw, dx))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
