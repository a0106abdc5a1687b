"""A workspace is written by the calls it is given to, in their streams, and by nothing that is
still queued elsewhere.  Each test keeps the current stream busy, runs a call on another stream
with a workspace made meanwhile, and marks the workspace's status word when that call is done:
the mark has to be there when the current stream is through as well."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from gen import inputs as gi

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 0x5A
BUSY = 1 << 29  # clock cycles: about a quarter of a second


def _layer():
    d, t = gi.make_layer("tiny", device=DEV)
    layer = moe.MoELayer(d.H, d.I, d.E, d.k, d.has_shared, t["w13"], t["w13_s"], t["w2"], t["w2_s"])
    x = gi.activations(d.T, d.H, 100, DEV)
    return layer, x, gi.router_logits("normal", x, d.E, 100, DEV)


def _mark(ws, st):
    with torch.cuda.stream(st):
        ws[:4].fill_(MARK)
    st.synchronize()


def _marked(ws):
    torch.cuda.synchronize()
    return ws[:4].tolist() == [MARK] * 4


def test_host_pipeline():
    layer, x, lg = _layer()
    xh, lh = x.cpu().pin_memory(), lg.cpu().pin_memory()
    oh = torch.empty_like(xh).pin_memory()
    want = layer.forward(x, lg)
    st = torch.cuda.Stream()
    # memory of the pipeline's size, with a write of its own still queued
    size = moe.host_pipeline_workspace_size(layer.dims(x.shape[0]), 2)
    before = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    before.fill_(0xFF)
    del before
    pipe = layer.host_pipeline(x.shape[0])
    pipe.submit(xh, lh, oh)
    pipe.sync()
    assert moe.moe_check_status(pipe.ws, st) == 0
    _mark(pipe.ws, st)
    assert _marked(pipe.ws)
    assert torch.equal(oh, want.cpu())
    pipe.close()


@pytest.mark.parametrize("host", [False, True])
def test_layer_on_another_stream(host):
    layer, x, lg = _layer()
    want = layer.forward(x, lg)
    fresh = _layer()[0]
    out = torch.empty_like(want)
    xh, lh, oh = x.cpu().pin_memory(), lg.cpu().pin_memory(), out.cpu().pin_memory()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    if host:
        fresh.forward_host(xh, lh, oh, stream=st)
        ws = fresh.host_workspace(x.shape[0])
    else:
        fresh.forward(x, lg, out=out, stream=st)
        ws = fresh.workspace(x.shape[0])
    assert moe.moe_check_status(ws, st) == 0
    _mark(ws, st)
    assert _marked(ws)
    assert torch.equal(oh if host else out.cpu(), want.cpu())


def test_linear_on_the_workspaces_stream():
    x, w = (torch.ones(9, 512, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    y = torch.empty(9, 9, device=DEV, dtype=torch.float32)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    ws = moe.alloc_workspace(moe.linear_workspace_size(9, 9, 512), stream=st)
    moe.moe_linear(x, w, y, ws, stream=st)
    assert moe.moe_check_status(ws, st) == 0
    _mark(ws, st)
    assert _marked(ws)
    assert torch.equal(y, torch.full_like(y, 512.0))
