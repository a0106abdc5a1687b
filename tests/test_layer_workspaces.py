"""A layer's workspaces over steps that get longer: what a captured graph goes on using stays, the
gradient products' status word is never replaced.  The bookkeeping on the CPU, with torch's
capture state and streams played by the test; on the GPU a graph replayed after longer steps."""

import ctypes
import gc
import weakref

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe


class _Recorded:
    """A workspace: its bytes, and the streams that it was recorded on."""

    def __init__(self, n):
        self.n, self.streams = n, []

    def numel(self):
        return self.n

    def record_stream(self, s):
        self.streams.append(s)


class _Stream(int):
    def synchronize(self):
        pass


@pytest.fixture
def played(monkeypatch):
    """The capture state, the current stream, and the workspaces that are alive."""
    now = dict(capturing=False, stream=1, alive=weakref.WeakSet())

    def alloc(n, device="cuda", stream=None):
        w = _Recorded(n)
        now["alive"].add(w)
        return w
    monkeypatch.setattr(moe, "alloc_workspace", alloc)
    monkeypatch.setattr(moe, "_raw_stream", lambda s: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: _Stream(now["stream"]))
    return now


def _layer(fmt="mxfp4"):
    w = [torch.zeros(1, dtype=torch.uint8) for _ in range(4)]
    return moe.MoELayer(512, 256, 8, 2, 1, *w, fmt=fmt)


GETS = {"workspace": lambda la, T: la.workspace(T), "host_workspace": lambda la, T: la.host_workspace(T),
        "train_workspaces": lambda la, T: la.train_workspaces(T)[0]}


@pytest.mark.parametrize("name", GETS)
def test_a_captured_workspace_outlives_longer_steps(played, name):
    layer, get = _layer(), GETS[name]
    small = weakref.ref(get(layer, 64))
    played["capturing"] = True
    assert get(layer, 64) is small()
    played["capturing"] = False
    sizes = [get(layer, T).numel() for T in (64, 128, 256)]
    gc.collect()
    assert small() is not None and sizes == sorted(sizes) and sizes[2] > sizes[0]
    # (that of 128 tokens, which no graph has, is given back)
    assert len({w.numel() for w in played["alive"]} & set(sizes)) == 2
    played["capturing"] = True  # a second graph, with the present one
    large = weakref.ref(get(layer, 100))
    played["capturing"] = False
    get(layer, 4096)
    gc.collect()
    assert small() is not None and large() is not None


@pytest.mark.parametrize("name", GETS)
def test_a_workspace_made_in_a_capture_is_that_graphs(played, name):
    layer, get = _layer(), GETS[name]
    played["capturing"] = True
    ws = weakref.ref(get(layer, 64))
    played["capturing"] = False
    assert get(layer, 64) is ws()  # (its status word is where that graph's checks are)
    get(layer, 2000)
    gc.collect()
    assert ws() is not None


@pytest.mark.parametrize("name", GETS)
def test_streams_that_use_a_workspace_are_recorded(played, name):
    layer, get = _layer(), GETS[name]
    ws = get(layer, 64)
    assert ws.streams == []
    played["stream"] = 2
    assert get(layer, 32) is ws and ws.streams == [2]
    new = get(layer, 2000)
    assert new is not ws and new.streams == []
    played["stream"] = 1
    get(layer, 64)
    assert new.streams == [1]


def test_the_gradient_products_keep_one_status_word(played):
    layer = _layer()
    first = layer.train_workspaces(1)[1]
    assert all(layer.train_workspaces(T)[1] is first for T in (64, 5000, 2))


def test_unsupported_dims_are_refused(played):
    w = [torch.zeros(1, dtype=torch.uint8) for _ in range(4)]
    for layer in (moe.MoELayer(200, 256, 8, 2, 1, *w), moe.MoELayer(384, 256, 8, 2, 1, *w, fmt="nvfp4")):
        for get in (GETS["workspace"], GETS["train_workspaces"]):
            with pytest.raises(ValueError, match="unsupported"):
                get(layer, 4)


def _filled(n):
    """Tensors over the memory that was given back, each filled."""
    t = [torch.full((1 << i,), 0x5A, dtype=torch.uint8, device="cuda") for i in range(9, 24) for _ in range(n)]
    torch.cuda.synchronize()
    return t


def _replayed_after_longer_steps(run, longer, inputs, outputs):
    """run captured; then longer steps, the memory they gave back filled, new inputs and a replay:
    the outputs are an eager run's, and what filled the memory is as it was."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outputs(run())
    longer()
    torch.cuda.synchronize()
    filled = _filled(6)
    g = torch.Generator().manual_seed(9)
    for t in inputs:
        t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool(torch.all(t == 0x5A)) for t in filled)
    got = [t.clone() for t in got]
    assert all(torch.equal(a, b) for a, b in zip(got, outputs(run())))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("form", ["fp8", "bf16", "forward"])
def test_a_graph_replayed_after_longer_steps(form, fmt):
    from tests.test_gpu_layer_grad import _layer as gpu_layer
    layer, x, logits, dout = gpu_layer(64, True, fmt=fmt)
    lx, llogits, ldout = (t.repeat(5, 1) for t in (x, logits, dout))
    out = torch.empty_like(x)

    def step(a, b, c, o=None):
        if form == "forward":
            return [layer.forward(a, b, out=o)]
        y, s = layer.forward_train(a, b, checkpoint=form)
        return [y, *layer.backward(c, s)]
    _replayed_after_longer_steps(lambda: step(x, logits, dout, out),
                                 lambda: [step(lx[:n], llogits[:n], ldout[:n]) for n in (128, 300)],
                                 [x, logits, dout], list)
    assert moe.moe_check_status(layer.train_workspaces(64)[1]) == 0


@pytest.mark.gpu
def test_a_host_graph_replayed_after_longer_steps():
    from tests.test_gpu_layer_grad import _layer as gpu_layer
    layer, x, logits, _ = gpu_layer(64, True)
    graph = layer.host_graph(64)
    pinned = [t.repeat(5, 1).cpu().pin_memory() for t in (x, logits, x)]
    layer.forward_host(*pinned)
    torch.cuda.synchronize()
    filled = _filled(6)
    graph.x_host.copy_(x.cpu())
    graph.logits_host.copy_(logits.cpu())
    got = graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, layer.forward(x, logits).cpu())
    assert all(bool(torch.all(t == 0x5A)) for t in filled)


def test_joined_status_words_refusals():
    P = ctypes.c_void_p
    f, A, odd = moe.lib().moe_join_status, P(0x10000), P(0x10080)
    two = (P * 2)(A, A)
    assert f(None, two, 2, None) == 1 and f(odd, two, 2, None) == 1 and f(A, None, 2, None) == 1
    assert f(A, two, 0, None) == 1 and f(A, (P * 9)(*[A] * 9), 9, None) == 1
    assert f(A, (P * 2)(A, None), 2, None) == 1 and f(A, (P * 2)(odd, A), 2, None) == 1


@pytest.mark.gpu
def test_joined_status_words():
    words = [0, 4, 1, 0, 2, 0, 0, 1]
    ws = [moe.alloc_workspace(256) for _ in words]
    for n in range(1, 9):
        for w, v in zip(ws, words):
            w[0] = v
        into = moe.alloc_workspace(256)
        into[0] = 8
        moe.moe_join_status(into, ws[:n])
        want = 8
        for v in words[:n]:
            want |= v
        assert moe.moe_check_status(into) == want
        assert [moe.moe_check_status(w) for w in ws] == words
