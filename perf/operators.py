"""Measured cases of the operators around the expert FFN: residual + RMS norm (bf16 and FP8
outputs), the router's balance loss, and the dense projection with its epilogue, each forward
and backward.

`run` computes a case with elementary torch operations in fp32 (own = False), or through the
package's entry points (own = True); `exact` computes it in float64 from the definitions.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu")

# The largest listed sizes; drawn cases stay within them.
NORM_MAX = 32768 * 7168
BALANCE_MAX = 32768 * 384
LINEAR_MAX = 16384 * 7168 * 7168
LINEAR_BWD_MAX = 4096 * 6144 * 7168


# ------------------------------------------------------------------------- cases
def _norm(name, T, H, stream, residual, quant, gain):
    return dict(name=name, op="norm", T=T, H=H, stream=stream, residual=residual, quant=quant,
                gain=gain)


def _norm_bwd(name, T, H, stream, dh_in, gain):
    return dict(name=name, op="norm_bwd", T=T, H=H, stream=stream, dh_in=dh_in, gain=gain)


def _balance(name, op, T, E, k, S, mask, dw):
    return dict(name=name, op=op, T=T, E=E, k=k, S=S, mask=mask, dw=dw)


def _linear(name, op, M, N, K, act, bias, residual, stream):
    return dict(name=name, op=op, M=M, N=N, K=K, act=act, bias=bias, residual=residual,
                stream=stream)


def listed():
    return [
        # the norm in front of the MoE layer in a 7-token verify step: FP8 for W13, bf16 for
        # the router
        _norm("norm_decode", 7, 7168, "bf16", True, True, "bf16"),
        # the same norm in a 32K-token prefill chunk
        _norm("norm_prefill", 32768, 7168, "bf16", True, True, "bf16"),
        # a small model's norm with an fp32 residual stream and an odd width, bf16 output only
        _norm("norm_odd", 1531, 1023, "fp32", True, False, "fp32"),
        # training step on 8K tokens, fp32 residual stream with its own incoming gradient
        _norm_bwd("norm_bwd_train", 8192, 7168, "fp32", True, "fp32"),
        # a short batch, bf16 stream
        _norm_bwd("norm_bwd_small", 64, 512, "bf16", True, "bf16"),
        # router statistics of a 32K-token step, 384 experts, one batch-wide loss
        _balance("balance_prefill", "balance", 32768, 384, 8, 1, False, False),
        # packed sequences of uneven (also zero) length with padding, an odd expert count
        _balance("balance_ragged", "balance", 4999, 61, 3, 37, True, False),
        # gradient of the logits for the 32K-token step, the combine weights' gradient included
        _balance("balance_bwd_prefill", "balance_bwd", 32768, 384, 8, 4, False, True),
        # output projection of a 7-token verify step, residual added in the epilogue
        _linear("linear_decode", "linear", 7, 7168, 7168, "none", False, True, "bf16"),
        # the same projection in a 16K-token prefill chunk
        _linear("linear_prefill", "linear", 16384, 7168, 7168, "none", False, True, "bf16"),
        # a head of odd sizes on a ragged batch, fp32 residual stream
        _linear("linear_odd", "linear", 333, 1111, 777, "gelu", True, True, "fp32"),
        # gradient of a dense layer's up projection over 4K tokens
        _linear("linear_bwd", "linear_bwd", 4096, 6144, 7168, "silu", True, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "balance", "balance_bwd", "linear", "linear_bwd"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("norm", "norm_bwd"):
        T = _log(rng, 1, 32768)
        H = min(_log(rng, 64, 8192), NORM_MAX // T)
        stream, gain = rng.choice(("bf16", "fp32")), rng.choice(("bf16", "fp32"))
        if op == "norm_bwd":
            # the fp32 stream moves more bytes a value: stay within the listed training case
            return dict(op=op, T=T, H=min(H, 8192 * 7168 // T), stream=stream, dh_in=flag(),
                        gain=gain)
        quant = flag()
        if quant:
            H = max(128, H // 128 * 128)
        if stream == "fp32":
            T = min(T, 16384)
        return dict(op=op, T=T, H=H, stream=stream, residual=flag(), quant=quant, gain=gain)
    if op in ("balance", "balance_bwd"):
        T = _log(rng, 1, 32768)
        E = min(_log(rng, 4, 1024), BALANCE_MAX // T)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=_log(rng, 1, 64),
                    mask=flag(), dw=flag() if op == "balance_bwd" else False)
    cap = LINEAR_MAX if op == "linear" else LINEAR_BWD_MAX
    N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
    if flag():  # half of the draws on whole 16-byte rows
        N, K = max(64, N // 8 * 8), max(64, K // 8 * 8)
    M = min(_log(rng, 1, 16384), cap // (N * K))
    return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), bias=flag(),
                residual=flag() if op == "linear" else False,
                stream=rng.choice(("bf16", "fp32")) if op == "linear" else "bf16")


# ------------------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    return {"norm": _prep_norm, "norm_bwd": _prep_norm_bwd, "balance": _prep_balance,
            "balance_bwd": _prep_balance, "linear": _prep_linear,
            "linear_bwd": _prep_linear_bwd}[case["op"]](dict(case), _gen(seed))


def _prep_norm(c, g):
    T, H, st = c["T"], c["H"], _dt(c["stream"])
    c["x"] = _normal(g, T, H)
    c["res"] = _normal(g, T, H, scale=2.0, dtype=st) if c["residual"] else None
    c["g"] = (1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(_dt(c["gain"]))
    c["h"] = _empty(T, H, dtype=st) if c["residual"] else None
    c["y"] = _empty(T, H, dtype=torch.bfloat16)
    c["q"] = _empty(T, H, dtype=torch.uint8) if c["quant"] else None
    c["s"] = _empty(T, H // 128, dtype=torch.uint8) if c["quant"] else None
    c["rstd"] = _empty(T, dtype=torch.float32)
    return c


def _prep_norm_bwd(c, g):
    T, H, st = c["T"], c["H"], _dt(c["stream"])
    c["h"] = _normal(g, T, H, scale=2.0, dtype=st)
    c["rstd"] = torch.rsqrt(c["h"].float().square().mean(1) + EPS)
    c["g"] = (1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(_dt(c["gain"]))
    c["dy"] = _normal(g, T, H)
    c["dhi"] = _normal(g, T, H, dtype=st) if c["dh_in"] else None
    c["dh"] = _empty(T, H, dtype=st)
    # with an fp32 stream the block output's gradient is wanted in its own type too
    c["dx"] = _empty(T, H, dtype=torch.bfloat16) if c["stream"] == "fp32" else None
    c["dgain"] = _empty(H, dtype=torch.float32)
    return c


def _prep_balance(c, g):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    # experts of uneven popularity, as a router that needs the loss has them
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
    logits += torch.randn(E, generator=g, device=DEV)
    c["idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    c["off"] = None
    if S > 1:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV).sort().values
        if S > 3:
            cuts[1] = cuts[0]  # one sequence without tokens at least
        ends = torch.tensor([0, T], device=DEV)
        c["off"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    c["msk"] = None
    if c["mask"]:
        keep = torch.rand(T, generator=g, device=DEV) < 0.8
        # rows of padding hold whatever the projection of unset memory gave
        junk = torch.rand(T, generator=g, device=DEV)
        logits[~keep & (junk < 0.2)] = float("nan")
        logits[~keep & (junk > 0.8)] = float("inf")
        c["msk"] = keep.to(torch.uint8)
    c["logits"] = logits
    c["counts"] = _empty(S, E, dtype=torch.int32)
    c["n"] = _empty(S, dtype=torch.int32)
    c["prob"] = _empty(S, E, dtype=torch.float32)
    c["loss"], c["z"] = _empty(S, dtype=torch.float32), _empty(S, dtype=torch.float32)
    if c["op"] == "balance_bwd":
        seg, keep = _segments(c)
        n = torch.zeros(S, dtype=torch.int64, device=DEV)
        n.index_add_(0, seg[keep], torch.ones_like(seg[keep]))
        flat = (seg[:, None] * E + c["idx"].long())[keep].reshape(-1)
        counts = torch.zeros(S * E, dtype=torch.int64, device=DEV)
        counts.index_add_(0, flat, torch.ones_like(flat))
        c["counts"], c["n"] = counts.view(S, E).to(torch.int32), n.to(torch.int32)
        c["dloss"] = torch.rand(S, generator=g, device=DEV) + 0.5
        c["dz"] = torch.rand(S, generator=g, device=DEV) * 0.1
        c["dw"] = torch.randn(T, k, generator=g, device=DEV) * 1e-3 if c["dw"] else None
        c["dlogits"] = _empty(T, E, dtype=torch.float32)
    return c


def _prep_linear(c, g):
    M, N, K, st = c["M"], c["N"], c["K"], _dt(c["stream"])
    c["x"] = _normal(g, M, K)
    c["w"] = _normal(g, N, K, scale=K ** -0.5)
    c["b"] = _normal(g, N, dtype=torch.float32) if c["bias"] else None
    c["res"] = _normal(g, M, N, scale=2.0, dtype=st) if c["residual"] else None
    c["y"] = _empty(M, N, dtype=st)
    return c


def _prep_linear_bwd(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    c["x"] = _normal(g, M, K)
    c["w"] = _normal(g, N, K, scale=K ** -0.5)
    c["z"] = _normal(g, M, N) if c["act"] != "none" else None
    c["dy"] = _normal(g, M, N)
    c["dx"] = _empty(M, K, dtype=torch.bfloat16)
    c["dwt"] = _empty(N, K, dtype=torch.bfloat16)
    c["db"] = _empty(N, dtype=torch.float32) if c["bias"] else None
    return c


# ------------------------------------------------------------------------- the calls
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _fp8(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _own_norm(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_add_rmsnorm(c["x"], c["res"], c["g"], EPS, h=c["h"], y=c["y"], q=c["q"], s=c["s"],
                        rstd=c["rstd"])
    q, s = _fp8(c["q"], c["s"]) if c["quant"] else (None, None)
    return dict(h=c["h"], y=c["y"], q=q, s=s, rstd=c["rstd"])


def _own_norm_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    ws = c.get("ws")
    if ws is None:
        ws = c["ws"] = moe.alloc_workspace(
            moe.add_rmsnorm_backward_workspace_size(c["T"], c["H"]))
    moe.moe_add_rmsnorm_backward(c["dy"], c["h"], c["g"], c["rstd"], ws, dh_in=c["dhi"],
                                 dh=c["dh"], dx=c["dx"], dgain=c["dgain"])
    return dict(dh=c["dh"], dx=c["dx"], dgain=c["dgain"])


def _own_balance(c):
    import moe_expert_ffn_scan_gb300 as moe
    ws = c.get("ws")
    if ws is None:
        ws = c["ws"] = moe.alloc_workspace(
            moe.balance_loss_workspace_size(c["T"], c["E"], c["k"], c["S"]))
    moe.moe_balance_loss(c["logits"], c["idx"], c["counts"], c["n"], c["prob"], c["loss"], c["z"],
                         ws, seq_offsets=c["off"], token_mask=c["msk"])
    return dict(counts=c["counts"], n=c["n"], prob=c["prob"], loss=c["loss"], z=c["z"])


def _own_balance_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_balance_loss_backward(c["logits"], c["idx"], c["counts"], c["n"], c["dlogits"],
                                  dloss=c["dloss"], dz_loss=c["dz"], dw=c["dw"],
                                  seq_offsets=c["off"], token_mask=c["msk"])
    return dict(dlogits=c["dlogits"])


def _own_linear(c):
    import moe_expert_ffn_scan_gb300 as moe
    ws = c.get("ws")
    if ws is None:
        ws = c["ws"] = moe.alloc_workspace(moe.linear_workspace_size(c["M"], c["N"], c["K"]))
    moe.moe_linear(c["x"], c["w"], c["y"], ws, bias=c["b"], residual=c["res"], act=c["act"])
    return dict(y=c["y"])


def _own_linear_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    ws = c.get("ws")
    if ws is None:
        ws = c["ws"] = moe.alloc_workspace(
            moe.linear_backward_workspace_size(c["M"], c["N"], c["K"]))
    moe.moe_linear_backward(c["x"], c["w"], c["dy"], ws, z=c["z"], act=c["act"], dx=c["dx"],
                            dw=c["dwt"], dbias=c["db"])
    return dict(dx=c["dx"], dw=c["dwt"], db=c["db"])


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance,
        "balance_bwd": _own_balance_bwd, "linear": _own_linear, "linear_bwd": _own_linear_bwd}


# ------------------------------------------------------------------------- plain forms
def _plain_norm(c):
    a = c["x"].float()
    if c["res"] is not None:
        a = a + c["res"].float()
    h = a.to(c["h"].dtype) if c["h"] is not None else None
    rstd = torch.rsqrt(a.square().mean(1) + EPS)
    y = (a * rstd[:, None] * c["g"].float()).to(torch.bfloat16)
    q = s = None
    if c["quant"]:
        # one power of two per row per 128 columns, the smallest with amax <= 448 * 2^e
        b = y.float().view(c["T"], -1, 128)
        amax = b.abs().amax(2)
        man, ex = torch.frexp(amax)  # amax = man * 2^ex, 0.5 <= man < 1; 448 = 0.875 * 2^9
        e = torch.where(amax > 0, ex - 9 + (man > 0.875), torch.zeros_like(ex)).clamp(-127, 127)
        q = torch.ldexp(b, -e[:, :, None]).view(c["T"], c["H"]).to(torch.float8_e4m3fn)
        s = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return dict(h=h, y=y, q=q, s=s, rstd=rstd)


def _plain_norm_bwd(c):
    dy, r = c["dy"].float(), c["rstd"][:, None]
    n = c["h"].float() * r
    u = dy * c["g"].float()
    dh = r * (u - n * (u * n).mean(1, keepdim=True))
    if c["dhi"] is not None:
        dh = dh + c["dhi"].float()
    dgain = (dy * n).sum(0)
    dx = dh.to(torch.bfloat16) if c["dx"] is not None else None
    return dict(dh=dh.to(c["dh"].dtype), dx=dx, dgain=dgain)


def _segments(c):
    """Each token's sequence, and whether it counts."""
    T = c["T"]
    if c["off"] is None:
        seg = torch.zeros(T, dtype=torch.int64, device=DEV)
    else:
        at = torch.arange(T, device=DEV, dtype=torch.int32)
        seg = torch.searchsorted(c["off"][1:].contiguous(), at, right=True)
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if c["msk"] is None else c["msk"] != 0
    return seg, keep


def _plain_softmax(logits, keep):
    """Probabilities and logsumexp; rows left out, and rows of -inf alone, have zeros."""
    x = torch.where(keep[:, None], logits, torch.zeros_like(logits))
    m = x.amax(1, keepdim=True)
    keep = keep & (m[:, 0] != float("-inf"))
    x = torch.where(keep[:, None], x - m, torch.zeros_like(x))
    ex = torch.exp(x)
    total = ex.sum(1, keepdim=True)
    live = keep[:, None].float()
    p = ex / total * live
    lse = torch.where(keep, m[:, 0] + torch.log(total[:, 0]), torch.zeros_like(total[:, 0]))
    return p, lse


def _plain_balance(c):
    E, k, S = c["E"], c["k"], c["S"]
    seg, keep = _segments(c)
    p, lse = _plain_softmax(c["logits"], keep)
    counts = torch.zeros(S, E, dtype=torch.int32, device=DEV)
    inc = keep.to(torch.int32)[:, None].expand(-1, k).reshape(-1)
    counts.view(-1).index_add_(0, (seg[:, None] * E + c["idx"].long()).reshape(-1), inc)
    n = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, seg, keep.to(torch.int32))
    if S == 1:
        sum_p, sum_z = p.sum(0, keepdim=True), lse.square().sum(0, keepdim=True)
    else:
        member = (seg[None, :] == torch.arange(S, device=DEV)[:, None]).float()
        sum_p, sum_z = member @ p, member @ lse.square()
    d = n.float().clamp(min=1)
    prob = sum_p / d[:, None]
    loss = (counts.float() * prob).sum(1) * (E / k) / d
    return dict(counts=counts, n=n, prob=prob, loss=loss, z=sum_z / d)


def _plain_balance_bwd(c):
    E, k = c["E"], c["k"]
    seg, keep = _segments(c)
    p, lse = _plain_softmax(c["logits"], keep)
    d = c["n"].float().clamp(min=1)
    a = c["counts"].float() * (c["dloss"] * (E / k) / (d * d))[:, None]
    a = a[seg]
    out = p * (a - (a * p).sum(1, keepdim=True))
    out = out + p * (2 * (c["dz"] / d)[seg] * lse)[:, None]
    if c["dw"] is not None:
        idx = c["idx"].long()
        chosen = torch.where(keep[:, None], c["logits"].gather(1, idx), torch.zeros(1, device=DEV))
        ex = torch.exp(chosen - chosen.amax(1, keepdim=True))
        w = ex / ex.sum(1, keepdim=True)
        g = w * (c["dw"] - (w * c["dw"]).sum(1, keepdim=True)) * keep[:, None].float()
        out = out.scatter_add(1, idx, g)
    return dict(dlogits=out)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    return cdf + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _plain_linear(c):
    y = c["x"].float() @ c["w"].float().t()
    if c["b"] is not None:
        y = y + c["b"]
    y = _act(y, c["act"])
    if c["res"] is not None:
        y = y + c["res"].float()
    return dict(y=y.to(c["y"].dtype))


def _plain_linear_bwd(c):
    dz = c["dy"].float()
    if c["z"] is not None:
        dz = dz * _act_slope(c["z"].float(), c["act"])
    db = dz.sum(0) if c["db"] is not None else None
    return dict(dx=(dz @ c["w"].float()).to(torch.bfloat16),
                dw=(dz.t() @ c["x"].float()).to(torch.bfloat16), db=db)


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance,
          "balance_bwd": _plain_balance_bwd, "linear": _plain_linear,
          "linear_bwd": _plain_linear_bwd}


# ------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, T, H = case["T"] * case["H"], case["T"], case["H"]
        st = 2 if case["stream"] == "bf16" else 4
        small = H * (2 if case["gain"] == "bf16" else 4) + 4 * T
        if op == "norm":
            byts = n * (2 + 2) + (2 * st * n if case["residual"] else 0)
            byts += n + n // 128 if case["quant"] else 0
            return dict(bytes=byts + small, flops=6 * n)
        byts = n * (2 + st + st) + (st * n if case["dh_in"] else 0) + (2 * n if st == 4 else 0)
        return dict(bytes=byts + small + 4 * H, flops=10 * n)
    if op in ("balance", "balance_bwd"):
        n, T, S = case["T"] * case["E"], case["T"], case["S"]
        byts = 4 * n + 4 * T * case["k"] + (T if case["mask"] else 0) + 4 * (S + 1)
        if op == "balance":
            return dict(bytes=byts + S * (8 * case["E"] + 12), flops=5 * n)
        return dict(bytes=byts + 4 * n + S * (4 * case["E"] + 12) +
                    (4 * T * case["k"] if case["dw"] else 0), flops=8 * n)
    M, N, K = case["M"], case["N"], case["K"]
    st = 2 if case["stream"] == "bf16" else 4
    if op == "linear":
        byts = 2 * (M * K + N * K) + st * M * N * (2 if case["residual"] else 1)
        return dict(bytes=byts + (4 * N if case["bias"] else 0), flops=2 * M * N * K)
    byts = 4 * (M * K + N * K) + 2 * M * N * (1 if case["act"] == "none" else 2)
    return dict(bytes=byts + (4 * N if case["bias"] else 0), flops=4 * M * N * K)


# ------------------------------------------------------------------------- float64
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "balance": _exact_balance,
            "balance_bwd": _exact_balance_bwd, "linear": _exact_linear,
            "linear_bwd": _exact_linear_bwd}[case["op"]](s)


def _rows(T, H):
    """Row ranges whose float64 temporaries stay small."""
    step = max(1, (1 << 26) // H)
    return [slice(i, min(T, i + step)) for i in range(0, T, step)]


def _exact_norm(c):
    T, H = c["T"], c["H"]
    f = torch.float64
    h = torch.empty(T, H, dtype=f, device=DEV) if c["h"] is not None else None
    y, rstd = torch.empty(T, H, dtype=f, device=DEV), torch.empty(T, dtype=f, device=DEV)
    q = torch.empty(T, H, dtype=f, device=DEV) if c["quant"] else None
    sc = torch.empty(T, H // 128, dtype=f, device=DEV) if c["quant"] else None
    gain = c["g"].to(f)
    for r in _rows(T, H):
        a = c["x"][r].to(f)
        if c["res"] is not None:
            a += c["res"][r].to(f)
        if h is not None:
            h[r] = a
        rstd[r] = 1 / torch.sqrt((a * a).sum(1) / H + EPS)
        y[r] = a * rstd[r, None] * gain
        if q is not None:
            # the codes are of the bf16 value of y
            b = y[r].to(torch.bfloat16).to(f).reshape(-1, H // 128, 128)
            top = b.abs().max(2).values
            e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448))
            e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
            e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
            e = torch.where(top > 0, e, torch.zeros_like(e)).clamp(-127, 127)
            sc[r] = torch.exp2(e)
            q[r] = (b / torch.exp2(e)[:, :, None]).reshape(-1, H).to(torch.float8_e4m3fn).to(f)
    return dict(h=h, y=y, q=q, s=sc, rstd=rstd)


def _exact_norm_bwd(c):
    T, H = c["T"], c["H"]
    f = torch.float64
    dh = torch.empty(T, H, dtype=f, device=DEV)
    dgain, gain = torch.zeros(H, dtype=f, device=DEV), c["g"].to(f)
    for r in _rows(T, H):
        dy, hh, rs = c["dy"][r].to(f), c["h"][r].to(f), c["rstd"][r].to(f)[:, None]
        dot = (dy * gain * hh).sum(1, keepdim=True)
        # d/dh of h * rstd * gain with rstd = (mean h^2 + eps)^(-1/2)
        dh[r] = dy * gain * rs - hh * dot * rs ** 3 / H
        if c["dhi"] is not None:
            dh[r] += c["dhi"][r].to(f)
        dgain += (dy * hh * rs).sum(0)
    return dict(dh=dh, dx=dh if c["dx"] is not None else None, dgain=dgain)


def _exact_parts(c):
    """For each sequence: its valid tokens, their float64 softmax and logsumexp."""
    T, S = c["T"], c["S"]
    off = [0, T] if c["off"] is None else c["off"].tolist()
    for s in range(S):
        rows = torch.arange(off[s], off[s + 1], device=DEV)
        if c["msk"] is not None:
            rows = rows[c["msk"][rows] != 0]
        x = c["logits"][rows].double()
        yield s, rows, torch.softmax(x, 1), torch.logsumexp(x, 1)


def _exact_balance(c):
    E, k, S = c["E"], c["k"], c["S"]
    f = torch.float64
    prob = torch.zeros(S, E, dtype=f, device=DEV)
    loss, z = torch.zeros(S, dtype=f, device=DEV), torch.zeros(S, dtype=f, device=DEV)
    for s, rows, p, lse in _exact_parts(c):
        n = rows.numel()
        if n == 0:
            continue
        share = torch.bincount(c["idx"][rows].long().reshape(-1), minlength=E).double() / (k * n)
        prob[s] = p.mean(0)
        loss[s], z[s] = E * torch.dot(share, prob[s]), (lse * lse).mean()
    return dict(counts=None, n=None, prob=prob, loss=loss, z=z)


def _exact_balance_bwd(c):
    T, E, k = c["T"], c["E"], c["k"]
    out = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for s, rows, p, lse in _exact_parts(c):
        n = rows.numel()
        if n == 0:
            continue
        # d loss / d p_te, the same for each token of the sequence; then through the softmax
        up = c["dloss"][s].double() * E * c["counts"][s].double() / (k * n * n)
        g = p * (up - (p @ up)[:, None]) + (2 * c["dz"][s].double() / n) * lse[:, None] * p
        if c["dw"] is not None:
            idx = c["idx"][rows].long()
            w = torch.softmax(c["logits"][rows].double().gather(1, idx), 1)
            dw = c["dw"][rows].double()
            g.scatter_add_(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)))
        out[rows] = g
    return dict(dlogits=out)


def _exact_linear(c):
    w = c["w"].double()
    y = torch.empty(c["M"], c["N"], dtype=torch.float64, device=DEV)
    for r in _rows(c["M"], max(c["N"], c["K"])):
        z = c["x"][r].double() @ w.t()
        if c["b"] is not None:
            z += c["b"].double()
        if c["act"] == "relu":
            z = torch.relu(z)
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif c["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        if c["res"] is not None:
            z += c["res"][r].double()
        y[r] = z
    return dict(y=y)


def _exact_linear_bwd(c):
    dz = c["dy"].double()
    if c["z"] is not None:
        z = c["z"].double()
        if c["act"] == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif c["act"] == "silu":
            sg = torch.sigmoid(z)
            dz = dz * (sg + z * sg * (1 - sg))
        else:
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return dict(dx=dz @ c["w"].double(), dw=dz.t() @ c["x"].double(),
                db=dz.sum(0) if c["db"] is not None else None)
