"""The operators together, as examples/moe_block.py runs them: against the layer's own forward
on the norm's bf16 output (the codes are the same, so the outputs are too), and the router's
gradients against float64."""

import numpy as np
import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from examples.moe_block import make_block
from tests import _block_ref as ref
from tests._parity import assert_float_close

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_forward_is_the_layers_own(T):
    block, attn, stream = make_block(T)
    f = block.forward(attn, stream)
    assert block.check() == [0, 0, 0, 0]
    h = _np(attn) @ _np(block.w_o).T + _np(stream)
    assert_float_close(_np(f["h"]), h, "h")
    y = ref.norm(_np(f["h"]), None, _np(block.gain), block.eps)[2]
    assert np.all(np.abs(_np(f["y"]) - y) <= 2.0 ** -8 * np.abs(y) * 1.01)
    own = block.layer.forward(f["y"], f["logits"])
    assert_float_close(_np(f["out"]), _np(own), "out", rel=1e-6, min_cos=0.999999)
    # and its addition to the stream in the next block's norm
    nxt, out = torch.empty_like(stream), torch.empty_like(stream)
    moe.moe_add_rmsnorm(f["out"], f["h"], block.gain, block.eps, h=nxt, y=out)
    assert torch.equal(nxt, (f["out"].float() + f["h"].float()).to(torch.bfloat16))


def test_router_step():
    T, S = 130, 3
    block, attn, stream = make_block(T, n_seq=S)
    off = torch.tensor([0, 50, 50, 130], dtype=torch.int32, device="cuda")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[40:60] = False
    f = block.forward(attn, stream)
    o, g = block.router_step(f, seq_offsets=off, token_mask=mask, balance=1.0, z=0.1)
    assert block.check() == [0, 0, 0, 0]
    args = (_np(f["logits"]), f["idx"].cpu().numpy(), off.cpu().numpy(), mask.cpu().numpy(), S)
    counts, n, prob, loss, z = ref.balance(*args)
    assert np.array_equal(o["counts"].cpu().numpy(), counts)
    assert o["n_tokens"].tolist() == [40, 0, 70]
    np.testing.assert_allclose(_np(o["loss"]), loss, rtol=1e-4)
    dl = ref.balance_bwd(*args, np.ones(S), np.full(S, 0.1), None)[0]
    assert_float_close(_np(g["dlogits"]), dl, "dlogits", rel=1e-4)
    # through the gate (bf16 weight), the norm and the projection: each from the bf16 gradient
    # that the stage behind it gave
    dl16, wg16 = _np(g["dlogits"].to(torch.bfloat16)), _np(block.wg.to(torch.bfloat16))
    assert_float_close(_np(g["dwg"]), dl16.T @ _np(f["y"]), "dwg")
    assert_float_close(_np(g["dy"]), dl16 @ wg16, "dy")
    dh, dgain = ref.norm_bwd(_np(g["dy"]), _np(f["h"]), _np(f["rstd"]), _np(block.gain))
    assert_float_close(_np(g["dh"]), dh, "dh", rel=4e-2)
    assert_float_close(_np(g["dgain"]), dgain, "dgain", rel=4e-2)
    assert_float_close(_np(g["dattn"]), _np(g["dh"]) @ _np(block.w_o), "dattn", rel=4e-2)
    assert_float_close(_np(g["dw_o"]), _np(g["dh"]).T @ _np(attn), "dw_o", rel=4e-2)
