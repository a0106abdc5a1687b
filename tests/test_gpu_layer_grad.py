"""The gradient's operators together: MoELayer.forward_train / backward and the example's
training step against float64 (stage by stage on the saved state, and as a whole), difference
quotients of the formulas, streams, captured graphs."""

import numpy as np
import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from examples.moe_block import make_block
from gen import inputs as gi
from tests import _block_ref as block_ref
from tests import _grad_ref as ref
from tests._parity import assert_float_close, with_gate_logits

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _experts(x, w13, w2, chosen, w, I):
    """sum_j w_j W2_e (silu(g) u) of one token in float64, [g | u] = W13_e x; the shared expert
    last with weight 1."""
    out = 0
    for e, we in zip(chosen, w):
        y = w13[e] @ x
        out = out + we * (w2[e] @ (y[:I] * ref.sigmoid(y[:I]) * y[I:]))
    return out


def test_formulas_against_difference_quotients():
    """The chain that backward runs (dispatch, W2, SwiGLU with the weights, W13, sum), in float64
    on the CPU, against central differences of the layer's formula."""
    H, I, E, k = 12, 8, 4, 2
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    w13, w2, x, dout, w = r(E, 2 * I, H) * 0.4, r(E, H, I) * 0.4, r(H), r(H), torch.rand(k, generator=g, dtype=torch.float64)
    chosen = [2, 0]
    dx, dw = torch.zeros(H, dtype=torch.float64), []
    for e, we in zip(chosen, w):
        y = w13[e] @ x
        dh = dout @ w2[e]
        dg, du, _ = ref.swiglu_bwd(y[:I], y[I:], we * dh)
        dx += torch.cat([dg, du]) @ w13[e]
        dw.append(torch.dot(dh, y[:I] * ref.sigmoid(y[:I]) * y[I:]))
    f = lambda xx, ww: torch.dot(dout, _experts(xx, w13, w2, chosen, ww, I))  # noqa: E731
    eps = 1e-6
    for i in range(H):
        s = torch.zeros(H, dtype=torch.float64)
        s[i] = eps
        assert abs((f(x + s, w) - f(x - s, w)) / (2 * eps) - dx[i]) < 1e-7 * (1 + abs(dx[i]))
    for j in range(k):
        s = torch.zeros(k, dtype=torch.float64)
        s[j] = eps
        assert abs((f(x, w + s) - f(x, w - s)) / (2 * eps) - dw[j]) < 1e-7 * (1 + abs(dw[j]))


def _layer(T, shared, seed=0, fmt="mxfp4"):
    d, t = gi.make_layer("tiny", seed=seed)
    g = torch.Generator().manual_seed(seed + 5)
    t = with_gate_logits(t)
    sh = d.has_shared
    w = {n: t[n].to(DEV) for n in ("w13", "w13_s", "w2", "w2_s")}
    if shared and not sh:  # one more group from the first
        w = {n: torch.cat([v, v[:1].flip(1)]) for n, v in w.items()}
    more = {}
    if fmt == "nvfp4":  # E4M3 scales of 2^-4 .. 15 per 16, tensor scales around one
        for n in ("w13_s", "w2_s"):
            v = torch.randint(24, 80, (*w[n].shape[:2], w[n].shape[2] * 2), generator=g)
            w[n] = v.to(torch.uint8).to(DEV)
        G = d.E + int(shared)
        more = dict(fmt=fmt, w13_gs=(torch.rand(G, 2, generator=g) + 0.5).to(DEV),
                    w2_gs=(torch.rand(G, generator=g) + 0.5).to(DEV))
    layer = moe.MoELayer(d.H, d.I, d.E, d.k, int(shared), *w.values(), **more)
    x = torch.randn(T, d.H, generator=g).to(BF).to(DEV)
    logits = torch.randn(T, d.E, generator=g).to(DEV)
    dout = torch.randn(T, d.H, generator=g).to(BF).to(DEV)
    return layer, x, logits, dout


def _through(layer, name, dy, off, F):
    w, w_s = getattr(layer, name), getattr(layer, name + "_s")
    nv = layer.fmt == "nvfp4"
    return ref.expert_grad(dy, off, w, w_s, dy.shape[0], F,
                           getattr(layer, name + "_gs") if nv else None, nv)


def _whole(layer, s, dout, dx_in=None, dx_bf16=True):
    """dx and dw in float64 from the saved state, each with a bound of the kernels' error: the
    roundings of the steps (half a step of bf16 of dh, dy13, each row of dxp and dx; 2^-22 a
    step of 16 of the products' sums; the sigmoid's c; fp32 sums), each carried through the
    magnitudes of the steps behind it."""
    T, k, I, H = s["T"], layer.k, layer.I, layer.H
    R, sh = T * k, layer.has_shared
    perm, off = s["perm_src"].long(), s["offsets"]
    Rs = R + T * sh
    rows = torch.zeros(Rs, H, dtype=torch.float64, device=DEV)
    rows[:R] = dout.double()[perm // k]
    if sh:
        rows[R:] = dout.double()
    wr = torch.ones(Rs, 1, dtype=torch.float64, device=DEV)
    wr[:R, 0] = s["w"].double().view(-1)[perm]
    dh, size = _through(layer, 'w2', rows, off, I)
    # (with bf16 the weight comes in front of the product and its rounding, in that of dy2)
    e_dh = ref.U16 * dh.abs() + (H / 16 + 1) * 2.0 ** -22 * size
    if "yq" not in s:
        e_dh += ref.U16 * size
    y = ref.fp8_values(s["yq"], s["ys"]) if "yq" in s else s["y13"].double()
    g, u = y[:, :I], y[:, I:]
    dg, du, scale = ref.swiglu_bwd(g, u, dh * wr)
    c = (g.abs() + 16) * 2.0 ** -22
    sg = ref.sigmoid(g)
    e_g = (u * sg * (1 + g * (1 - sg))).abs() * wr * e_dh + ref.U16 * dg.abs() + c * scale
    e_u = (g * sg).abs() * wr * e_dh + (ref.U16 + c) * du.abs()
    dy, e_dy = torch.cat([dg, du], 1), torch.cat([e_g, e_u], 1)
    rows, size = _through(layer, 'w13', dy, off, H)
    e_rows = ref.U16 * rows.abs() + (2 * I / 16 + 1) * 2.0 ** -22 * size
    e_rows += _through(layer, 'w13', e_dy, off, H)[1]
    dx, size = ref.dispatch_bwd(rows, s["inv"], T, k, R, sh, dx_in)
    e_dx = (k + 2) * ref.U32 * size + ref.dispatch_bwd(e_rows, s["inv"], T, k, R, sh)[0]
    if dx_bf16:
        e_dx += ref.U16 * dx.abs()
    dw = torch.zeros(2, R, dtype=torch.float64, device=DEV)
    if "yq" in s:
        h = ref.fp8_values(s["hq"], s["hs"])
        dw[0, perm] = (dh * h)[:R].sum(1)
        dw[1, perm] = ((e_dh + 96 * ref.U32 * dh.abs()) * h.abs())[:R].sum(1)
    else:
        prod = dout.double()[perm // k] * s["y2"][:R].double()
        dw[0, perm], dw[1, perm] = prod.sum(1), 64 * ref.U32 * prod.abs().sum(1)
    # second-order terms: a percent of the bound
    return dx, 1.01 * e_dx, dw[0].view(T, k), 1.01 * dw[1].view(T, k)


def _close(got, want, bound, name):
    """Within the bound everywhere, and in norm within five roundings to bf16: each moves its
    step's values by at most 2^-8 of their norm, and the steps behind it carry that and the
    values alike (random signs)."""
    err = (got.double() - want).abs()
    assert torch.all(err <= bound), (name, (err - bound).max().item())
    assert err.norm() <= 5 * ref.U16 * want.norm(), (name, (err.norm() / want.norm()).item())


_np = lambda t: t.detach().double().cpu().numpy()  # noqa: E731


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 64, 300, 1500])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("form", ["fp8", "bf16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_layer(T, shared, form, fmt):
    layer, x, logits, dout = _layer(T, shared, fmt=fmt)
    out, s = layer.forward_train(x, logits, checkpoint=form)
    assert torch.equal(out, layer.forward(x, logits))
    dx, dw = layer.backward(dout, s)
    assert [moe.moe_check_status(w) for w in layer.train_workspaces(T)] == [0, 0]
    want_dx, e_dx, want_dw, e_dw = _whole(layer, s, dout)
    _close(dx, want_dx, e_dx, "dx")
    _close(dw, want_dw, e_dw, "dw")
    # with another gradient of x, in fp32
    more = torch.randn(T, layer.H, device=DEV)
    dx32, dw2 = layer.backward(dout, s, dx=torch.empty_like(more), dx_in=more)
    assert torch.equal(dw, dw2)
    want, bound = _whole(layer, s, dout, more, False)[:2]
    _close(dx32, want, bound, "dx + dx_in")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 400])
def test_full_size_layer_on_sampled_tokens(T):
    """384 experts of 7168 x 2048, top-8 and shared, uneven popularity; whole tokens in float64.
    Four roundings to bf16 on dx's way (dh, dy13, the rows, dx), each of at most 2^-8 of its
    values in norm, one on dw's."""
    H, I, E, k = 7168, 2048, 384, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    layer = moe.MoELayer(H, I, E, k, 1, ri(0, 256, E + 1, 2 * I, H // 2),
                         ri(114, 119, E + 1, 2 * I, H // 32), ri(0, 256, E + 1, H, I // 2),
                         ri(114, 119, E + 1, H, I // 32))
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dout, logits = rn(T, H).to(BF), rn(T, H).to(BF), rn(T, E) + 2 * rn(E)
    s = layer.forward_train(x, logits)[1]
    dx, dw = layer.backward(dout, s)
    assert [moe.moe_check_status(w) for w in layer.train_workspaces(T)] == [0, 0]
    assert torch.all(torch.isfinite(dx.float())) and torch.all(torch.isfinite(dw))
    for t in (0, T // 2, T - 1):
        rows, experts = s["inv"][t * k:(t + 1) * k].tolist() + [T * k + t], s["idx"][t].tolist() + [E]
        weights, want, wdw = s["w"][t].tolist() + [1.0], 0, []
        for r, e, w in zip(rows, experts, weights):
            dh = dout[t].double() @ ref.mxfp4(layer.w2[e], layer.w2_s[e])
            y = ref.fp8_values(s["yq"][r:r + 1], s["ys"][r:r + 1])[0]
            h = ref.fp8_values(s["hq"][r:r + 1], s["hs"][r:r + 1])[0]
            wdw.append((dh * h).sum())
            dg, du, _ = ref.swiglu_bwd(y[:I], y[I:], w * dh)
            want = want + torch.cat([dg, du]) @ ref.mxfp4(layer.w13[e], layer.w13_s[e])
        assert (dx[t].double() - want).norm() <= 4 * ref.U16 * want.norm()
        wdw = torch.stack(wdw[:k])
        # (dw's terms of random signs: the sum's error against the largest of the token's)
        assert torch.all((dw[t].double() - wdw).abs() <= 4 * ref.U16 * wdw.abs().max())


@pytest.mark.gpu
def test_the_two_checkpoints_agree():
    """The 8-bit checkpoint's rounding (half a step: 2^-4) is in dx of one and not the other, its
    sign random from value to value."""
    layer, x, logits, dout = _layer(300, True)
    grads = [layer.backward(dout, layer.forward_train(x, logits, checkpoint=f)[1])
             for f in ("fp8", "bf16")]
    for a, b in zip(*grads):
        err = (a.double() - b.double()).norm() / b.double().norm()
        assert err < 2.0 ** -4


@pytest.mark.gpu
def test_refusals_of_the_layer():
    layer, x, logits, dout = _layer(4, False)
    with pytest.raises(ValueError, match="checkpoint"):
        layer.forward_train(x, logits, checkpoint="int8")
    with pytest.raises(ValueError, match="dx: expected bfloat16 or float32"):
        layer.backward(dout, layer.forward_train(x, logits)[1], dx=torch.empty_like(dout).half())


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(monkeypatch):
    """(One GPU: the current device is made to look like another.)"""
    layer, x, logits, dout = _layer(4, False)
    s = layer.forward_train(x, logits)[1]
    d, bf = layer.dims(4), lambda *n: torch.empty(*n, dtype=BF, device=DEV)
    u8 = lambda *n: torch.empty(*n, dtype=torch.uint8, device=DEV)  # noqa: E731
    R, H, I = 4 * layer.k, layer.H, layer.I
    ws = layer.train_workspaces(4)[1]
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    calls = [lambda: moe.moe_dispatch(d, x, s["inv"], bf(R, H)),
             lambda: moe.moe_dispatch_backward(d, bf(R, H), s["inv"], bf(4, H)),
             lambda: moe.moe_combine_backward(d, dout, None, s["inv"], s["w"], dy2=bf(R, H)),
             lambda: moe.moe_swiglu_quant_save(bf(R, 2 * I), u8(R, I), u8(R, I // 128),
                                               u8(R, 2 * I), u8(R, I // 64)),
             lambda: moe.moe_swiglu_backward(bf(R, I), bf(R, 2 * I), y13=bf(R, 2 * I)),
             lambda: moe.moe_grouped_gemm_w2_backward(d, bf(R, H), s["offsets"], layer.w2,
                                                      layer.w2_s, bf(R, I), ws)]
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["fp8", "bf16"])
def test_captured_and_replayed_on_new_inputs(form):
    T = 130
    layer, x, logits, dout = _layer(T, True)
    layer.train_workspaces(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.backward(dout, layer.forward_train(x, logits, checkpoint=form)[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, s = layer.forward_train(x, logits, checkpoint=form)
        dx, dw = layer.backward(dout, s)
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=g).to(BF))
        logits.copy_(torch.randn(logits.shape, generator=g))
        dout.copy_(torch.randn(dout.shape, generator=g).to(BF))
        graph.replay()
        got = [t.clone() for t in (out, dx, dw)]
        own, s2 = layer.forward_train(x, logits, checkpoint=form)
        want = [own, *layer.backward(dout, s2)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_on_a_stream_of_its_own():
    T = 64
    layer, x, logits, dout = _layer(T, True)
    out, s = layer.forward_train(x, logits)
    want = layer.backward(dout, s)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, s2 = layer.forward_train(x, logits, stream=st)
    got = layer.backward(dout, s2, stream=st)
    st.synchronize()
    assert torch.equal(out, o2) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_block_training_step():
    T = 130
    block, attn, stream = make_block(T)
    f = block.forward(attn, stream, save=True)
    dout = torch.randn(f["out"].shape, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    o, g = block.router_step(f, dout=dout, balance=1.0, z=0.1)
    assert block.check() == [0, 0, 0, 0]
    s = dict(T=T, perm_src=f["perm"], offsets=f["offsets"], inv=f["inv"], w=f["w"],
             **{n: f[n] for n in ("yq", "ys", "hq", "hs")})
    dy, e_dy, dw, e_dw = _whole(block.layer, s, dout, dx_bf16=False)
    _close(g["dy_experts"], dy, e_dy, "dy of the experts")
    _close(g["dw"], dw, e_dw, "dw")
    dl = block_ref.balance_bwd(_np(f["logits"]), f["idx"].cpu().numpy(), None, None, 1, np.ones(1),
                               np.full(1, 0.1), _np(g["dw"]))[0]
    assert_float_close(_np(g["dlogits"]), dl, "dlogits", rel=1e-4)
    # through the gate and the norm, the residual stream's own gradient added
    wg16, dl16 = _np(block.wg.to(BF)), _np(g["dlogits"].to(BF))
    assert_float_close(_np(g["dy"]), dl16 @ wg16 + _np(g["dy_experts"]), "dy")
    dh, _ = block_ref.norm_bwd(_np(g["dy"]), _np(f["h"]), _np(f["rstd"]), _np(block.gain), _np(dout))
    # one rounding to bf16 behind fp32 sums over a row of terms of dh's size
    assert np.all(np.abs(_np(g["dh"]) - dh) <= ref.U16 * np.abs(dh) + 1e-4 * np.abs(dh).max(1, keepdims=True))


@pytest.mark.gpu
def test_saving_changes_no_output():
    block, attn, stream = make_block(64)
    a, b = block.forward(attn, stream), block.forward(attn, stream, save=True)
    assert torch.equal(a["out"], b["out"])
