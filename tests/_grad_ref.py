"""float64 torch forms of the routed layer's gradient (test code only), written from their
formulas."""

import torch

F64 = torch.float64
U32 = 2.0 ** -24  # half a unit in the last place of fp32, relative
U16 = 2.0 ** -8   # and of bf16
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def slots(inv, R):
    """(slots with a row, their rows)."""
    inv = inv.view(-1).long()
    at = torch.nonzero((inv >= 0) & (inv < R))[:, 0]
    return at, inv[at]


def dispatch_bwd(dxp, inv, T, k, R, shared, dx_in=None):
    """dx and the sum of its terms' magnitudes (the scale of its rounding)."""
    at, rows = slots(inv, R)
    dx = torch.zeros(T, dxp.shape[1], dtype=F64, device=dxp.device)
    size = torch.zeros_like(dx)
    for out, f in ((dx, lambda v: v), (size, torch.abs)):
        if dx_in is not None:
            out += f(dx_in.to(F64))
        out.index_add_(0, at // k, f(dxp[rows].to(F64)))
        if shared:
            out += f(dxp[R:R + T].to(F64))
    return dx, size


def sigmoid(g):
    return torch.where(g >= 0, 1 / (1 + torch.exp(-g.clamp(min=0))),
                       torch.exp(g.clamp(max=0)) / (1 + torch.exp(g.clamp(max=0))))


def swiglu_bwd(g, u, d):
    """dg, du, and for dg the magnitude that its rounding goes by."""
    s = sigmoid(g)
    return d * u * s * (1 + g * (1 - s)), d * g * s, (d * u).abs() * (s + (g * s).abs())


def fp8_values(q, s):
    """E4M3 codes and scale bytes per 128 columns."""
    v = q.view(torch.float8_e4m3fn).to(F64).view(q.shape[0], -1, 128)
    return (v * torch.exp2(s.to(F64) - 127)[:, :, None]).view(q.shape)


def mxfp4(codes, scales):
    """[.., F/2] codes and [.., F/32] scale bytes -> [.., F] values."""
    lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=F64, device=codes.device)
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.to(F64) - 127).repeat_interleave(32, -1)


def nvfp4(codes, scales, gs=None):
    """[.., C, F/2] codes, [.., C, F/16] E4M3 scales and the tensor scales of the equal parts of
    the C rows -> [.., C, F] values."""
    lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=F64, device=codes.device)
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    v = v * scales.view(torch.float8_e4m3fn).to(F64).repeat_interleave(16, -1)
    if gs is not None:
        gs = gs.to(F64).reshape(-1)
        v = v * gs.repeat_interleave(v.shape[-2] // gs.numel())[:, None]
    return v


def expert_grad(dy, off, w, w_s, rows, F, gs=None, nv=False):
    """dx (rows of no group: NaN) and the sum of its terms' magnitudes."""
    dx = torch.full((rows, F), float("nan"), dtype=F64, device=dy.device)
    size = torch.zeros_like(dx)
    off = off.tolist()
    for g in range(len(off) - 1):
        if off[g] < off[g + 1]:
            d = dy[off[g]:off[g + 1]].to(F64)
            v = nvfp4(w[g], w_s[g], None if gs is None else gs[g]) if nv else mxfp4(w[g], w_s[g])
            dx[off[g]:off[g + 1]] = d @ v
            size[off[g]:off[g + 1]] = d.abs() @ v.abs()
    return dx, size
