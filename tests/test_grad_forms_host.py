"""The gradient products' form by name and by cost: refusals and choices, before anything is launched
(no GPU)."""

import ctypes

import pytest

import moe_expert_ffn_scan_gb300 as moe

P = ctypes.c_void_p
A, ARG, SHAPE, SMALL = P(0x10000), 1, 2, 3


def _d(T=4, H=256, I=256, E=8, k=2, sh=1):
    return ctypes.byref(moe.dims(T, H, I, E, k, sh))


@pytest.mark.parametrize("product", [2, 13])
@pytest.mark.parametrize("nv", [0, 1])
def test_refusals(product, nv):
    f = moe.lib().moe_gemm_backward_form
    # d product nvfp4 ctas dy offsets w w_s gs dx ws bytes stream
    good = [_d(), product, nv, 1, A, A, A, A, A if nv else None, A, A, 256, None]
    put = lambda i, v: f(*good[:i], v, *good[i + 1:])  # noqa: E731
    for i, v in ((1, 0), (1, 3), (2, 2), (2, -1), (3, 0), (3, 3), (8, P(0x10002)), (4, P(0x10008))):
        assert put(i, v) == ARG
    for i in (4, 5, 6, 7, 9, 10):
        assert put(i, None) == ARG
    assert put(0, None) == SHAPE and put(0, _d(H=200)) == SHAPE and put(0, _d(T=0)) == SHAPE
    assert put(11, 255) == SMALL
    if nv:
        assert put(0, _d(I=384)) == SHAPE
    else:
        assert put(8, A) == ARG  # tensor scales without NVFP4


def test_choices():
    f = moe.lib().moe_gemm_backward_ctas
    assert f(None, 2) == 0 and f(_d(H=200), 2) == 0 and f(_d(), 3) == 0
    # a verify step's few rows a group: single CTAs; many rows: SM pairs
    assert all(f(_d(T=7, H=7168, I=2048, E=128, k=8), p) == 1 for p in (2, 13))
    assert all(f(_d(T=8192, H=7168, I=2048, E=64, k=8), p) == 2 for p in (2, 13))
