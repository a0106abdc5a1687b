"""The device checks of the layer's gradient: a call runs on the current device, and each of its
tensors has to be there; the layer's training step checks what it is given.  Stand-ins for tensors of two GPUs and for the library; no GPU."""

import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class _T:
    """What the binding asks of a GPU tensor."""

    def __init__(self, *shape, dt=BF, device=0):
        self.shape, self.dtype, self.at = torch.Size(shape), dt, device

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


T, H, I, E, k = 4, 256, 256, 8, 2
R, Rs, G = T * k, T * k + T, E + 1
D = moe.dims(T, H, I, E, k, 1)
u8 = lambda *s: dict(shape=s, dt=U8)  # noqa: E731
f32 = lambda *s: dict(shape=s, dt=F32)  # noqa: E731
i32 = lambda *s: dict(shape=s, dt=I32)  # noqa: E731
bf = lambda *s: dict(shape=s, dt=BF)  # noqa: E731
W2 = dict(w2=u8(G, H, I // 2), w2_s=u8(G, H, I // 32))
W13 = dict(w13=u8(G, 2 * I, H // 2), w13_s=u8(G, 2 * I, H // 32))
N2 = dict(w2=u8(G, H, I // 2), w2_s=u8(G, H, I // 16), w2_gs=f32(G))
N13 = dict(w13=u8(G, 2 * I, H // 2), w13_s=u8(G, 2 * I, H // 16), w13_gs=f32(G, 2))
P2 = dict(dy2=bf(Rs, H), group_offsets=i32(G + 1), dh=bf(Rs, I), ws=u8(256))
P13 = dict(dy13=bf(Rs, 2 * I), group_offsets=i32(G + 1), dxp=bf(Rs, H), ws=u8(256))
SAVED = dict(yq=u8(Rs, 2 * I), ys=u8(Rs, 2 * I // 128), hq=u8(Rs, I), hs=u8(Rs, I // 128))
CALLS = [
    ("moe_dispatch", dict(x=bf(T, H), inv=i32(R), xp=bf(Rs, H))),
    ("moe_dispatch_backward", dict(dxp=bf(Rs, H), inv=i32(R), dx=bf(T, H), dx_in=bf(T, H))),
    ("moe_combine_backward", dict(dout=bf(T, H), y2=bf(Rs, H), inv=i32(R), w=f32(T, k), dy2=bf(Rs, H),
                                  dw=f32(T, k))),
    ("moe_swiglu_quant_save", dict(y13=bf(Rs, 2 * I), **SAVED)),
    ("moe_swiglu_backward", dict(dh=bf(Rs, I), dy13=bf(Rs, 2 * I), perm_src=i32(R), w=f32(T, k),
                                 dw=f32(T, k), **SAVED)),
    ("moe_swiglu_backward", dict(dh=bf(Rs, I), dy13=bf(Rs, 2 * I), y13=bf(Rs, 2 * I))),
    ("moe_grouped_gemm_w2_backward", dict(**P2, **W2)),
    ("moe_grouped_gemm_w13_backward", dict(**P13, **W13)),
    ("moe_grouped_gemm_w2_backward_nvfp4", dict(**P2, **N2)),
    ("moe_grouped_gemm_w13_backward_nvfp4", dict(**P13, **N13)),
]


class _Library:
    """Every entry point accepts its arguments and says how often one was called."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.mark.parametrize("name,args", CALLS, ids=lambda v: v if isinstance(v, str) else "")
def test_every_tensor_of_a_call(monkeypatch, name, args):
    library = _Library()
    monkeypatch.setattr(moe, "lib", lambda: library)
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    monkeypatch.setattr(moe, "_current_raw_stream", lambda d: 0)
    more = {} if "swiglu" in name else dict(d=D)

    def call(away=None):
        t = {n: _T(*v["shape"], dt=v["dt"], device=int(n == away)) for n, v in args.items()}
        getattr(moe, name)(**more, **t)
    call()
    assert library.calls == 1
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        call()
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    for n in args:
        with pytest.raises(ValueError, match="cuda:1"):
            call(away=n)
    assert library.calls == 1


@pytest.mark.parametrize("bad", [
    dict(x=f32(T, H)), dict(x=bf(T, H + 128)), dict(logits=bf(T, E)), dict(logits=f32(T - 1, E)),
    dict(logits=f32(T, E + 1)), dict(out=f32(T, H)), dict(out=bf(T + 1, H)),
    dict(x=dict(shape=(T, H), dt=BF, device=1)), dict(logits=dict(shape=(T, E), dt=F32, device=1)),
    dict(out=dict(shape=(T, H), dt=BF, device=1))], ids=str)
def test_forward_train_checks_its_tensors(monkeypatch, bad):
    """(Its stages take what they are given.)"""
    library = _Library()
    monkeypatch.setattr(moe, "lib", lambda: library)
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    layer = moe.MoELayer(H, I, E, k, 1, None, None, None, None)
    args = dict(x=bf(T, H), logits=f32(T, E), out=bf(T, H)) | bad
    name = next(iter(bad))
    tensors = {n: _T(*v["shape"], dt=v["dt"], device=v.get("device", 0)) for n, v in args.items()}
    with pytest.raises(ValueError, match=name + ("" if "device" not in bad[name] else ".*cuda:1|cuda:1")):
        layer.forward_train(**tensors)
    assert library.calls == 0
