"""The expert FFN inside its transformer block: one forward step and the router's training step.

    python examples/moe_block.py [--tokens T]

Forward, for the T tokens of a step (a verify step's few or a prefill chunk):

    h    = attn W_o^T + stream                  moe_linear, the residual in its epilogue
    y, q = RMS norm of h in bf16 and FP8 codes  moe_add_rmsnorm
    idx  = top-k of y . W_g^T                   moe_router_logits, moe_route
    out  = routed experts of q                  moe_grouped_gemm_w13 / _w2 on the norm's own codes
    stream' = h + out                           the next norm's residual addition

Training the router (the experts' 4-bit weights stay as they are): balance loss and z loss of
the step's routing, and from them the gradients of the logits, of the gate weight, of the norm
and of the projection in front of it.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_expert_ffn_scan_gb300 as moe  # noqa: E402


class MoEBlock:
    """Weights, and the buffers and workspaces of a step of up to T tokens (any T at run time
    that does not exceed it)."""

    def __init__(self, layer, w_o, gain, wg, T, eps=1e-6, n_seq=1):
        self.layer, self.w_o, self.gain, self.wg, self.eps = layer, w_o, gain, wg, eps
        self.H, self.E, self.k = layer.H, layer.E, layer.k
        if layer.fmt != "mxfp4":
            raise ValueError("this block runs the MXFP4 stages")
        self.T, self.n_seq = T, n_seq
        dev = w_o.device
        d = layer.dims(T)
        N, K = w_o.shape
        self.ws = moe.alloc_workspace(max(moe.route_workspace_size(d), moe.gemm_workspace_size(d)),
                                      dev)
        self.ws_linear = moe.alloc_workspace(moe.linear_workspace_size(T, N, K), dev)
        self.ws_balance = moe.alloc_workspace(
            moe.balance_loss_workspace_size(T, self.E, self.k, n_seq), dev)
        self.ws_grad = moe.alloc_workspace(max(
            moe.linear_backward_workspace_size(T, N, K),
            moe.linear_backward_workspace_size(T, self.E, self.H)), dev)
        self.ws_norm = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(T, self.H), dev)

    def forward(self, attn, stream):
        """attn [T, K] bf16 (the attention's output), stream [T, H] bf16.  Returns the experts'
        output and everything that the next norm and the training step need."""
        T, H, E, k, sh = attn.shape[0], self.H, self.E, self.k, self.layer.has_shared
        d = self.layer.dims(T)
        R, Rs, I = T * k, T * k + T * sh, self.layer.I
        new = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=attn.device)  # noqa: E731
        f = dict(T=T, attn=attn, h=new(T, H), y=new(T, H), rstd=new(T, dt=torch.float32),
                 logits=new(T, E, dt=torch.float32), idx=new(T, k, dt=torch.int32),
                 w=new(T, k, dt=torch.float32), counts=new(E, dt=torch.int32))
        q, s = new(T, H, dt=torch.uint8), new(T, H // 128, dt=torch.uint8)
        moe.moe_linear(attn, self.w_o, f["h"], self.ws_linear, residual=stream)
        moe.moe_add_rmsnorm(f["h"], None, self.gain, self.eps, y=f["y"], q=q, s=s, rstd=f["rstd"])
        moe.moe_router_logits(f["y"], self.wg, f["logits"])
        offsets = new(E + sh + 1, dt=torch.int32)
        perm, inv = new(R, dt=torch.int32), new(R, dt=torch.int32)
        moe.moe_route(d, f["logits"], f["idx"], f["w"], f["counts"], offsets, perm, inv, self.ws)
        y13, hq = new(Rs, 2 * I), new(Rs, I, dt=torch.uint8)
        hs, y2, out = new(Rs, I // 128, dt=torch.uint8), new(Rs, H), new(T, H)
        L = self.layer
        moe.moe_grouped_gemm_w13(d, q, s, perm, offsets, L.w13, L.w13_s, y13, self.ws)
        moe.moe_swiglu_quant(y13, hq, hs)
        moe.moe_grouped_gemm_w2(d, hq, hs, offsets, L.w2, L.w2_s, y2, self.ws)
        moe.moe_combine(d, y2, inv, f["w"], out)
        f["out"] = out
        return f

    def router_step(self, f, seq_offsets=None, token_mask=None, balance=1e-2, z=1e-3):
        """Balance and z loss of a forward step, per sequence, and their gradients: of the
        gate weight, the norm's gain, the projection's weight and the two inputs."""
        T, E, H, S = f["T"], self.E, self.H, self.n_seq
        dev = f["y"].device
        new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        o = dict(counts=new(S, E, dt=torch.int32), n_tokens=new(S, dt=torch.int32),
                 prob=new(S, E), loss=new(S), z_loss=new(S))
        seqs = dict(seq_offsets=seq_offsets, token_mask=token_mask)
        moe.moe_balance_loss(f["logits"], f["idx"], ws=self.ws_balance, **o, **seqs)
        g = dict(dlogits=new(T, E))
        moe.moe_balance_loss_backward(
            f["logits"], f["idx"], o["counts"], o["n_tokens"], g["dlogits"],
            dloss=torch.full((S,), balance, device=dev), dz_loss=torch.full((S,), z, device=dev),
            **seqs)
        # the gate projection is one more product, its operands in bf16
        bf = torch.bfloat16
        g["dy"], g["dwg"] = new(T, H, dt=bf), new(E, H, dt=bf)
        moe.moe_linear_backward(f["y"], self.wg.to(bf), g["dlogits"].to(bf), self.ws_grad,
                                dx=g["dy"], dw=g["dwg"])
        g["dh"], g["dgain"] = new(T, H, dt=bf), new(H)
        moe.moe_add_rmsnorm_backward(g["dy"], f["h"], self.gain, f["rstd"], self.ws_norm,
                                     dh=g["dh"], dgain=g["dgain"])
        # h = attn W_o^T + stream: dh goes to the stream as it is
        g["dattn"], g["dw_o"] = torch.empty_like(f["attn"]), torch.empty_like(self.w_o)
        moe.moe_linear_backward(f["attn"], self.w_o, g["dh"], self.ws_grad, dx=g["dattn"],
                                dw=g["dw_o"])
        return o, g

    def check(self):
        """The device-side checks of the calls since the workspaces were made."""
        return [moe.moe_check_status(w) for w in (self.ws, self.ws_linear, self.ws_balance,
                                                 self.ws_grad)]


def make_block(T, size="tiny", seed=0, n_seq=1, device="cuda"):
    """A block around a seeded layer of gen/inputs.py, and one step's inputs."""
    from gen import inputs as gi
    d, t = gi.make_layer(size, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(torch.bfloat16).to(device)  # noqa: E731
    layer = moe.MoELayer(d.H, d.I, d.E, d.k, d.has_shared,
                         *[t[n].to(device) for n in ("w13", "w13_s", "w2", "w2_s")])
    wg = torch.randn(d.E, d.H, generator=g) * 0.02
    block = MoEBlock(layer, r(d.H, d.H, scale=d.H ** -0.5),
                     1 + r(d.H, scale=0.1), wg.to(device), T, n_seq=n_seq)
    return block, r(T, d.H), r(T, d.H, scale=2.0)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    block, attn, stream = make_block(a.tokens)
    f = block.forward(attn, stream)
    o, g = block.router_step(f)
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens: |out| {f['out'].float().norm():.4g}, balance loss "
          f"{o['loss'].item():.4f}, z loss {o['z_loss'].item():.4f}, |dW_g| "
          f"{g['dwg'].float().norm():.3g}, |dW_o| {g['dw_o'].float().norm():.3g}, "
          f"tokens per expert {o['counts'][0].tolist()}, checks {block.check()}")


if __name__ == "__main__":
    main()
