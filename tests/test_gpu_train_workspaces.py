"""The workspaces of a layer's training steps: every stage's device-side checks reach the step's
status word."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from examples.moe_block import make_block
from tests.test_gpu_layer_grad import _layer

pytestmark = pytest.mark.gpu


def _stage(name, fmt):
    return name + ("_nvfp4" if fmt == "nvfp4" and name != "moe_route" else "")


def _with_bit(monkeypatch, name):
    """The stage runs, then its workspace's status word has the bit of an expired wait."""
    real = getattr(moe, name)

    def call(*a, **kw):
        real(*a, **kw)
        a[-1][:1].fill_(moe.STATUS_WAIT_TIMEOUT)
    monkeypatch.setattr(moe, name, call)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("stage", ["moe_route", "moe_grouped_gemm_w13", "moe_grouped_gemm_w2"])
def test_a_stage_that_failed_is_seen_at_the_end_of_the_step(monkeypatch, stage, fmt):
    layer, x, logits, dout = _layer(64, True, fmt=fmt)
    layer.forward_train(x, logits)
    assert moe.moe_check_status(layer.train_workspaces(64)[0]) == 0
    with monkeypatch.context() as m:
        _with_bit(m, _stage(stage, fmt))
        layer.forward_train(x, logits)
    assert moe.moe_check_status(layer.train_workspaces(64)[0]) == moe.STATUS_WAIT_TIMEOUT
    out, _ = layer.forward_train(x, logits)  # the next step starts from none
    assert moe.moe_check_status(layer.train_workspaces(64)[0]) == 0
    assert torch.equal(out, layer.forward(x, logits))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_an_index_out_of_range_in_w13_is_seen(monkeypatch, fmt):
    """(W13 leaves out the row of such an index; W2 has no part in it.)"""
    layer, x, logits, _ = _layer(64, True, fmt=fmt)
    name = _stage("moe_grouped_gemm_w13", fmt)
    real = getattr(moe, name)

    def call(d, xq, xs, perm, *a):
        perm = perm.clone()
        perm[5] = -layer.k
        real(d, xq, xs, perm, *a)
    monkeypatch.setattr(moe, name, call)
    layer.forward_train(x, logits)
    assert moe.moe_check_status(layer.train_workspaces(64)[0]) == moe.STATUS_BAD_INDEX


@pytest.mark.parametrize("stage", ["moe_route", "moe_grouped_gemm_w13", "moe_grouped_gemm_w2"])
def test_a_stage_of_the_example_that_failed_is_seen(monkeypatch, stage):
    block, attn, stream = make_block(64)
    block.forward(attn, stream)
    assert block.check() == [0, 0, 0, 0]
    with monkeypatch.context() as m:
        _with_bit(m, stage)
        block.forward(attn, stream, save=True)
    assert block.check() == [moe.STATUS_WAIT_TIMEOUT, 0, 0, 0]
