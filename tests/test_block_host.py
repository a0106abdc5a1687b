"""Refusals of the operators around the expert FFN, before anything is launched (no GPU)."""

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


def test_add_rmsnorm_refusals(lib):
    f = lib.moe_add_rmsnorm
    #       rows cols x  res dt gain dt eps   h  y  q  s  rstd stream
    good = [4, 256, A, A, 0, A, 0, 1e-6, A, A, A, A, A, None]
    assert f(*_with(good, 0, 0)) == OK          # no rows: nothing to launch
    assert f(*_with(good, 0, -1)) == SHAPE
    assert f(*_with(good, 1, 0)) == SHAPE
    assert f(*_with(good, 1, 200)) == SHAPE     # codes want whole 128-column blocks
    for i in (2, 5):
        assert f(*_with(good, i, None)) == ARG
    for i in (2, 3, 5, 8, 9, 10):
        assert f(*_with(good, i, BAD)) == ARG
    assert f(*_with(good, 12, ODD)) == ARG
    for i in (4, 6):
        assert f(*_with(good, i, 2)) == ARG
    assert f(*_with(good, 7, -1.0)) == ARG and f(*_with(good, 7, float("nan"))) == ARG
    assert f(*_with(good, 11, None)) == ARG     # codes without scales
    assert f(*_with(good, 10, None)) == ARG     # scales without codes
    none = [4, 256, A, A, 0, A, 0, 1e-6, None, None, None, None, A, None]
    assert f(*none) == ARG                      # no output


def test_add_rmsnorm_backward_refusals(lib):
    f, size = lib.moe_add_rmsnorm_backward, lib.moe_add_rmsnorm_backward_workspace_size
    assert size(4, 256) >= 256 * 4 and size(10 ** 6, 256) < 2 ** 21
    assert size(-1, 256) == 0 and size(4, 0) == 0
    #       rows cols dy h dt gain dt rstd dh_in dh dx dgain ws bytes stream
    good = [4, 256, A, A, 0, A, 0, A, A, A, A, A, A, 1 << 20, None]
    assert f(*_with(good, 0, -1)) == SHAPE and f(*_with(good, 1, 0)) == SHAPE
    for i in (2, 3, 5, 7, 12):
        assert f(*_with(good, i, None)) == ARG
    for i in (2, 3, 5, 8, 9, 10, 12):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (7, 11):
        assert f(*_with(good, i, ODD)) == ARG
    for i in (4, 6):
        assert f(*_with(good, i, -1)) == ARG
    assert f(*_with(good, 13, 16)) == SMALL
    none = _with(_with(_with(good, 9, None), 10, None), 11, None)
    assert f(*none) == ARG


@pytest.mark.parametrize("cols", [(1 << 30) + 128, (1 << 31) - 512, (1 << 31) - 1])
def test_add_rmsnorm_refuses_rows_past_its_column_arithmetic(lib, cols):
    """32-bit column indices step by up to 512 past the row's end."""
    assert lib.moe_add_rmsnorm(1, cols, A, A, 0, A, 0, 1e-6, A, A, None, None, A, None) == SHAPE
    assert lib.moe_add_rmsnorm_backward(1, cols, A, A, 0, A, 0, A, A, A, A, A, A, 1 << 50,
                                        None) == SHAPE
    assert lib.moe_add_rmsnorm_backward_workspace_size(1, cols) == 0
    assert lib.moe_add_rmsnorm_backward_workspace_size(1, 1 << 30) > 4 << 30


def test_balance_loss_refusals(lib):
    f, size = lib.moe_balance_loss, lib.moe_balance_loss_workspace_size
    assert size(64, 8, 2, 1) > 0 and size(0, 8, 2, 1) > 0
    for bad in ((64, 0, 1, 1), (64, 1025, 2, 1), (64, 8, 9, 1), (64, 64, 17, 1), (64, 8, 0, 1),
                (-1, 8, 2, 1), (64, 8, 2, 0), (64, 8, 2, 65536), (1 << 28, 16, 8, 1)):
        assert size(*bad) == 0
        assert f(*bad, *[A] * 10, 1 << 40, None) == SHAPE
        assert lib.moe_balance_loss_backward(*bad, *[A] * 10, None) == SHAPE
    #       T   E  k  S  lg idx off mask counts n prob loss z ws bytes stream
    good = [64, 8, 2, 2, A, A, A, A, A, A, A, A, A, A, 1 << 40, None]
    for i in (4, 5, 6, 8, 9, 10, 11, 13):
        assert f(*_with(good, i, None)) == ARG
    for i in (4, 13):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (5, 6, 8, 9, 10, 11, 12):
        assert f(*_with(good, i, ODD)) == ARG
    assert f(*_with(good, 14, 64)) == SMALL


def test_balance_loss_backward_refusals(lib):
    f = lib.moe_balance_loss_backward
    #       T   E  k  S  lg idx off mask counts n dloss dz dw dlogits stream
    good = [64, 8, 2, 2, A, A, A, A, A, A, A, A, A, A, None]
    assert f(*_with(good, 0, 0)) == OK
    for i in (4, 5, 6, 8, 9, 13):
        assert f(*_with(good, i, None)) == ARG
    for i in (4, 13):
        assert f(*_with(good, i, BAD)) == ARG
    for i in (5, 6, 8, 9, 10, 11, 12):
        assert f(*_with(good, i, ODD)) == ARG


def test_binding_refuses_host_tensors_types_and_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_add_rmsnorm(x, None, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="x: expected"):
        moe.moe_add_rmsnorm(x.float(), None, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="expected bfloat16 or float32"):
        moe.moe_add_rmsnorm(x, x.half(), w, 1e-6, y=x)
    with pytest.raises(ValueError, match="logits: expected"):
        moe.moe_balance_loss_backward(x, torch.zeros(4, 2, dtype=torch.int32), None, None, None)


def _desc(**kw):
    d = dict(M=4, N=64, K=32, act=0, bias_dtype=0, y_dtype=0)
    d.update(kw)
    return ctypes.byref(moe.moe_linear_desc(**d))


def test_linear_refusals(lib):
    f, size = lib.moe_linear, lib.moe_linear_workspace_size
    big = 1 << 30
    assert size(_desc()) == 256                                    # the status word alone
    assert size(_desc(K=33)) > 256 and size(_desc(ldw=33)) > 256   # room for padded rows
    assert size(_desc(K=33, ldx=40, ldw=40)) == 256
    good = [A, A, A, A, A, A, A, big, None]  # x w bias residual y z ws bytes stream
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(ldx=31), dict(ldw=16), dict(ldy=63),
                dict(ldr=1), dict(ldz=-64), dict(N=(1 << 22) + 1), dict(M=1 << 29, N=1 << 20)):
        assert size(_desc(**bad)) == 0 and f(_desc(**bad), *good) == SHAPE
        assert lib.moe_linear_backward(_desc(**bad), *[A] * 8, big, None) == SHAPE
    assert f(None, *good) == SHAPE
    for bad in (dict(act=4), dict(act=-1), dict(y_dtype=2), dict(bias_dtype=7)):
        assert f(_desc(**bad), *good) == ARG
    assert f(_desc(M=0), *good) == OK
    for i in (0, 1, 4, 6):
        assert f(_desc(), *_with(good, i, None)) == ARG
    for i in (0, 1, 3, 4, 5, 6):
        assert f(_desc(), *_with(good, i, BAD)) == ARG
    assert f(_desc(), *_with(good, 2, ODD)) == ARG
    assert f(_desc(), *_with(good, 7, 255)) == SMALL


def test_linear_backward_refusals(lib):
    f, size = lib.moe_linear_backward, lib.moe_linear_backward_workspace_size
    good = [A, A, A, A, A, A, A, A, 1 << 30, None]  # x w z dy dx dw dbias ws bytes stream
    assert size(_desc(act=2)) > size(_desc()) > 0
    for i in (0, 1, 2, 3, 7):
        assert f(_desc(act=1), *_with(good, i, None)) == ARG
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert f(_desc(act=1), *_with(good, i, BAD)) == ARG
    assert f(_desc(), *_with(good, 6, ODD)) == ARG
    assert f(_desc(), *good[:4], None, None, None, *good[7:]) == ARG
    assert f(_desc(), *_with(good, 8, 256)) == SMALL


def test_linear_binding_refuses_shapes_types_and_strides():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16)
    y, ws = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x: expected"):
        moe.moe_linear(x.float(), w, y, ws)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_linear(x, w, y, ws)
    with pytest.raises(KeyError):
        moe.linear_backward_workspace_size(4, 64, 32, act="tanh")


@pytest.mark.parametrize("size", [
    *[lambda n, E=E, S=S: moe.balance_loss_workspace_size(n, E, 2, S)
      for E, S in ((8, 1), (384, 3), (61, 37), (1000, 1))],
    *[lambda n, cols=cols: moe.add_rmsnorm_backward_workspace_size(n, cols)
      for cols in (1, 512, 1023, 7168, 20008)],
    *[lambda n, N=N, K=K: moe.linear_workspace_size(n, N, K) for N, K in ((64, 64), (61, 77))],
    *[lambda n, N=N, K=K: moe.linear_backward_workspace_size(n, N, K)
      for N, K in ((64, 64), (61, 77), (8, 4096))]])
def test_a_workspace_for_the_longest_step_does_for_every_shorter_one(lib, size):
    sizes = [size(n) for n in range(6000)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
