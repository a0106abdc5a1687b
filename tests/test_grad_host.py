"""Refusals of the routed layer's gradient, before anything is launched (no GPU)."""

import ctypes
import os

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe

P = ctypes.c_void_p
OK, ARG, SHAPE, SMALL = 0, 1, 2, 3
A = P(0x10000)          # an aligned address that is never read
BAD = P(0x10000 + 8)    # not 16-byte aligned
ODD = P(0x10000 + 2)    # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from moe_expert_ffn_scan_gb300 import build
        build.build()
    return moe.lib()


def _with(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


def _d(T=4, H=256, I=128, E=8, k=2, sh=1):
    return ctypes.byref(moe.dims(T, H, I, E, k, sh))


BAD_DIMS = [dict(T=0), dict(T=-1), dict(H=200), dict(H=0), dict(I=64), dict(E=0), dict(E=1025),
            dict(k=0), dict(k=9), dict(E=64, k=17), dict(sh=2), dict(T=1 << 30, k=2)]


@pytest.mark.parametrize("bad", BAD_DIMS)
def test_dims_are_refused_by_every_call(lib, bad):
    d = _d(**bad)
    assert lib.moe_dispatch(d, A, A, A, None) == SHAPE
    assert lib.moe_dispatch_backward(d, A, A, A, 0, A, None) == SHAPE
    assert lib.moe_combine_backward(d, A, A, A, A, A, A, None) == SHAPE
    assert lib.moe_gemm_backward_workspace_size(d) == 0
    for f in (lib.moe_grouped_gemm_w2_backward, lib.moe_grouped_gemm_w13_backward):
        assert f(d, A, A, A, A, A, A, 1 << 30, None) == SHAPE
        assert f(None, A, A, A, A, A, A, 1 << 30, None) == SHAPE
    for f in (lib.moe_grouped_gemm_w2_backward_nvfp4, lib.moe_grouped_gemm_w13_backward_nvfp4):
        assert f(d, A, A, A, A, A, A, A, 1 << 30, None) == SHAPE
        assert f(None, A, A, A, A, A, A, A, 1 << 30, None) == SHAPE


def test_weights_past_the_tiles_row_coordinates_are_refused(lib):
    """The weight rows of all groups are one coordinate of 31 bits."""
    d = _d(H=1 << 21, I=256, E=1024)
    assert lib.moe_grouped_gemm_w2_backward(d, A, A, A, A, A, A, 1 << 30, None) == SHAPE


def test_dispatch_refusals(lib):
    good = [_d(), A, A, A, None]  # d x inv xp stream
    for i in (1, 2, 3):
        assert lib.moe_dispatch(*_with(good, i, None)) == ARG
        assert lib.moe_dispatch(*_with(good, i, BAD if i != 2 else ODD)) == ARG
    good = [_d(), A, A, A, 0, A, None]  # d dxp inv dx_in dtype dx stream
    for i in (1, 2, 5):
        assert lib.moe_dispatch_backward(*_with(good, i, None)) == ARG
    for i in (1, 3, 5):
        assert lib.moe_dispatch_backward(*_with(good, i, BAD)) == ARG
    assert lib.moe_dispatch_backward(*_with(good, 2, ODD)) == ARG
    for dt in (2, -1):
        assert lib.moe_dispatch_backward(*_with(good, 4, dt)) == ARG


def test_combine_backward_refusals(lib):
    f = lib.moe_combine_backward
    good = [_d(), A, A, A, A, A, A, None]  # d dout y2 inv w dy2 dw stream
    for i in (1, 2, 3, 4):
        assert f(*_with(good, i, None)) == ARG
    for i in (1, 2, 5):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (3, 4, 6):
        assert f(*_with(good, i, ODD)) == ARG
    assert f(_d(), A, A, A, A, None, None, None) == ARG  # no output


def test_swiglu_quant_save_refusals(lib):
    f = lib.moe_swiglu_quant_save
    good = [4, 256, A, A, A, A, A, None]  # rows I y13 hq hs yq ys stream
    assert f(*_with(good, 0, 0)) == OK
    for i, v in ((0, -1), (1, 0), (1, 200), (1, -128), (0, (1 << 30) + 1), (1, (1 << 29) + 128)):
        assert f(*_with(good, i, v)) == SHAPE
    for i in (2, 3, 4, 5, 6):
        assert f(*_with(good, i, None)) == ARG
    for i in (2, 3, 5):
        assert f(*_with(good, i, BAD)) == ARG


def test_swiglu_backward_refusals(lib):
    f = lib.moe_swiglu_backward
    desc = lambda rows=4, R=3, I=256: ctypes.byref(moe.moe_swiglu_backward_desc(rows, R, I))  # noqa: E731
    #       d       dh y13   yq ys hq hs perm w dy13 dw stream
    good = [desc(), A, None, A, A, A, A, A, A, A, A, None]
    assert f(*_with(good, 0, desc(rows=0, R=0))) == OK
    assert f(*_with(good, 0, None)) == SHAPE
    for bad in (dict(rows=-1), dict(R=5), dict(R=-1), dict(I=200), dict(I=0),
                dict(rows=(1 << 30) + 1), dict(I=(1 << 29) + 128)):
        assert f(*_with(good, 0, desc(**bad))) == SHAPE
    for i in (1, 3, 4, 5, 6, 7, 9):
        assert f(*_with(good, i, None)) == ARG
    assert f(*_with(good, 2, A)) == ARG                          # both forms of the input
    for i in (1, 3, 5, 9):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (7, 8, 10):
        assert f(*_with(good, i, ODD)) == ARG
    plain = [desc(), A, A, None, None, None, None, A, A, A, A, None]
    assert f(*_with(plain, 2, BAD)) == ARG
    assert f(*_with(plain, 4, A)) == ARG                         # scales without codes


@pytest.mark.parametrize("name", ["moe_grouped_gemm_w2_backward", "moe_grouped_gemm_w13_backward"])
def test_gradient_product_refusals(lib, name):
    f, size = getattr(lib, name), lib.moe_gemm_backward_workspace_size(_d())
    assert size >= 256
    good = [_d(), A, A, A, A, A, A, size, None]  # d dy offsets w w_s dx ws bytes stream
    for i in range(1, 7):
        assert f(*_with(good, i, None)) == ARG
    for i in (1, 3, 4, 5, 6):
        assert f(*_with(good, i, BAD)) == ARG
    assert f(*_with(good, 2, ODD)) == ARG
    assert f(*_with(good, 3, P(0x10010))) == ARG                 # codes: 32 bytes
    assert f(*_with(good, 6, P(0x10080))) == ARG                 # the workspace: 256
    assert f(*_with(good, 7, size - 1)) == SMALL


@pytest.mark.parametrize("name", ["moe_grouped_gemm_w2_backward_nvfp4",
                                  "moe_grouped_gemm_w13_backward_nvfp4"])
def test_nvfp4_gradient_product_refusals(lib, name):
    f, d = getattr(lib, name), _d(I=256)
    size = lib.moe_gemm_backward_workspace_size(d)
    good = [d, A, A, A, A, A, A, A, size, None]  # d dy offsets w w_s gs dx ws bytes stream
    for bad in (dict(), dict(H=384, I=256), dict(H=256, I=384)):  # whole 256s
        assert f(*_with(good, 0, _d(**bad))) == SHAPE
    for i in (1, 2, 3, 4, 6, 7):
        assert f(*_with(good, i, None)) == ARG
    for i in (1, 3, 4, 6, 7):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (2, 5):
        assert f(*_with(good, i, ODD)) == ARG
    assert f(*_with(good, 8, size - 1)) == SMALL


def test_binding_refuses_host_tensors_types_and_shapes():
    d = moe.dims(4, 256, 128, 8, 2, 1)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    inv = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_dispatch(d, bf(4, 256), inv, bf(12, 256))
    with pytest.raises(ValueError, match="x: expected"):
        moe.moe_dispatch(d, bf(5, 256), inv, bf(12, 256))
    with pytest.raises(ValueError, match="dx: expected bfloat16 or float32"):
        moe.moe_dispatch_backward(d, None, inv, bf(4, 256).half())
    with pytest.raises(ValueError, match="dout: expected"):
        moe.moe_combine_backward(d, bf(4, 128), None, inv, None)
    with pytest.raises(ValueError, match="y13: expected"):
        moe.moe_swiglu_quant_save(bf(4, 256).float(), None, None, None, None)
    with pytest.raises(ValueError, match="w: expected 8 values"):
        moe.moe_swiglu_backward(bf(12, 128), None, perm_src=inv, w=torch.zeros(7))
    with pytest.raises(ValueError, match="dy: expected"):
        moe.moe_grouped_gemm_w2_backward(d, bf(12, 128), inv, None, None, None, None)


@pytest.mark.parametrize("dims", [(256, 128, 8, 2, 1), (7168, 2048, 384, 8, 1), (128, 128, 1, 1, 0)])
def test_a_workspace_for_the_longest_step_does_for_every_shorter_one(lib, dims):
    sizes = [moe.gemm_backward_workspace_size(moe.dims(T, *dims)) for T in range(1, 3000)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
