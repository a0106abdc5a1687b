"""Measured cases of the routed layer's gradient with its experts frozen in 4 bits: tokens
sorted by expert and back, the combine's gradient, the 8-bit activation checkpoint with the
SwiGLU gradient that reads it, and the gradient products of the MXFP4 experts.

`run` computes a case with elementary torch operations in fp32 (own = False), or through the
package's entry points (own = True); `exact` computes it in float64 from the definitions.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

# The largest listed sizes (values of the packed rows, products' multiplications and weights);
# drawn cases stay within them.
DISPATCH_MAX = 16384 * 9 * 7168
COMBINE_MAX = 8192 * 9 * 7168
SWIGLU_MAX = 73728 * 2048
PRODUCT_MAX = 73728 * 4096 * 7168
WEIGHT_MAX = 129 * 7168 * 2048


# ------------------------------------------------------------------------- cases
def _moves(name, op, T, H, E, k, shared, dt="bf16", more=False, drop=False):
    """more: dispatch_bwd: a gradient that reaches x by other ways; combine_bwd: y2 is there
    and the weights' gradient is wanted."""
    return dict(name=name, op=op, T=T, H=H, E=E, k=k, shared=shared, dt=dt, more=more, drop=drop)


def _swiglu(name, op, rows, I, k, saved, weighted):
    return dict(name=name, op=op, rows=rows, I=I, k=k, saved=saved, weighted=weighted)


def _product(name, op, T, H, I, E, k, shared):
    return dict(name=name, op=op, T=T, H=H, I=I, E=E, k=k, shared=shared)


def listed():
    return [
        # tokens of a 7-token step to the rows of their experts
        _moves("dispatch_verify", "dispatch", 7, 7168, 384, 8, True),
        # a training step's 16K tokens
        _moves("dispatch_train", "dispatch", 16384, 7168, 64, 8, True),
        # their rows' gradients back to the tokens, added to the fp32 stream's own
        _moves("dispatch_bwd_train", "dispatch_bwd", 16384, 7168, 64, 8, True, "fp32", True),
        # gradient of the weighted combine over 8K tokens, expert outputs kept
        _moves("combine_bwd_train", "combine_bwd", 8192, 7168, 64, 8, True, more=True),
        # a ragged batch with dropped tokens, no shared expert
        _moves("combine_bwd_ragged", "combine_bwd", 1001, 640, 13, 3, False, more=True, drop=True),
        # 8K tokens' expert activations to 8 bits: W2's operand, and the checkpoint
        _swiglu("save_train", "save", 73728, 2048, 8, True, False),
        # their gradient from the checkpoint, the combine weights' with it
        _swiglu("swiglu_bwd_train", "swiglu_bwd", 73728, 2048, 8, True, True),
        # a short ragged batch from activations kept in bf16
        _swiglu("swiglu_bwd_small", "swiglu_bwd", 333, 384, 3, False, True),
        # the down projection's gradient product over 8K tokens
        _product("w2_bwd_train", "w2_bwd", 8192, 7168, 2048, 64, 8, True),
        # the gate and up projections'
        _product("w13_bwd_train", "w13_bwd", 8192, 7168, 2048, 64, 8, True),
        # few tokens over many experts: the weights are what is read
        _product("w13_bwd_few", "w13_bwd", 24, 7168, 2048, 128, 8, True),
        # a small model's layer on a ragged batch
        _product("w2_bwd_ragged", "w2_bwd", 777, 1152, 640, 13, 3, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _cols(rng, lo, hi):
    return max(128, _log(rng, lo, max(lo, hi)) // 128 * 128)


def draw(rng):
    op = rng.choice(("dispatch", "dispatch_bwd", "combine_bwd", "save", "swiglu_bwd", "w2_bwd",
                     "w13_bwd"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("save", "swiglu_bwd"):
        I = _cols(rng, 128, 4096)
        rows = _log(rng, 1, min(73728, SWIGLU_MAX // I))
        k = rng.randint(1, 8)
        return dict(op=op, rows=rows, I=I, k=k, saved=True if op == "save" else flag(),
                    weighted=op != "save" and rows > k and flag())
    E = _log(rng, 2, 128)
    k, shared = rng.randint(1, min(8, E)), flag()
    rows = k + shared  # of a token
    if op in ("w2_bwd", "w13_bwd"):
        I = _cols(rng, 128, 4096)
        # (as much for w2 as for w13: a weight group is at most the listed one's size)
        H = _cols(rng, 128, min(7168, WEIGHT_MAX // ((E + shared) * I)))
        T = _log(rng, 1, min(16384, PRODUCT_MAX // (rows * H * 2 * I)))
        return dict(op=op, T=T, H=H, I=I, E=E, k=k, shared=shared)
    H = _cols(rng, 128, 8192)
    most = (COMBINE_MAX if op == "combine_bwd" else DISPATCH_MAX) // (H * (rows + 1))
    T = _log(rng, 1, min(16384, most))
    return dict(op=op, T=T, H=H, E=E, k=k, shared=shared,
                dt=rng.choice(("bf16", "fp32")) if op == "dispatch_bwd" else "bf16",
                more=flag() if op != "dispatch" else False, drop=flag())


# ------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)


def _normal(g, *shape, scale=1.0, dtype=BF16):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] in ("save", "swiglu_bwd"):
        return _prep_swiglu(c, g)
    if c["op"] in ("w2_bwd", "w13_bwd"):
        return _prep_product(c, g)
    return _prep_moves(c, g)


def _routing(c, g):
    """Chosen experts of uneven popularity, and the rows that the tokens sorted by them take:
    expert after expert, in each the tokens in order; then a shared row for each token."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
    logits += torch.randn(E, generator=g, device=DEV)
    top = torch.topk(logits, k, dim=1)
    flat = top.indices.reshape(-1)
    perm = torch.argsort(flat, stable=True)  # row -> t k + j
    c["w"] = torch.softmax(top.values, 1)
    c["perm"] = perm.to(I32)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    c["inv"] = inv.to(I32)
    counts = torch.bincount(flat, minlength=E).tolist() + ([T] if c["shared"] else [])
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    c["off_host"], c["off"] = off, torch.tensor(off, dtype=I32, device=DEV)
    c["R"], c["Rs"] = T * k, off[-1]


def _prep_moves(c, g):
    _routing(c, g)
    T, H, Rs = c["T"], c["H"], c["Rs"]
    if c["drop"]:  # tokens past their expert's capacity: no row is theirs
        gone = torch.rand(T * c["k"], generator=g, device=DEV) < 0.1
        c["inv"] = torch.where(gone, torch.full_like(c["inv"], -1), c["inv"])
    if c["op"] == "dispatch":
        c["x"] = _normal(g, T, H)
        c["xp"] = torch.zeros(Rs, H, dtype=BF16, device=DEV)
    elif c["op"] == "dispatch_bwd":
        dt = F32 if c["dt"] == "fp32" else BF16
        c["dxp"] = _normal(g, Rs, H)
        c["dx_in"] = _normal(g, T, H, dtype=dt) if c["more"] else None
        c["dx"] = torch.empty(T, H, dtype=dt, device=DEV)
    else:
        c["dout"] = _normal(g, T, H)
        c["y2"] = _normal(g, Rs, H) if c["more"] else None
        c["dy2"] = torch.zeros(Rs, H, dtype=BF16, device=DEV)
        c["dw"] = torch.empty(T, c["k"], device=DEV) if c["more"] else None
    return c


def _codes(v):
    """E4M3 codes and scale bytes of v by rows of 128 columns: the smallest power of two with
    amax <= 448 * 2^e."""
    b = v.float().view(v.shape[0], -1, 128)
    man, ex = torch.frexp(b.abs().amax(2))  # amax = man * 2^ex, 0.5 <= man < 1; 448 = 0.875 * 2^9
    e = torch.where(man > 0, ex - 9 + (man > 0.875), torch.zeros_like(ex)).clamp(-127, 127)
    q = torch.ldexp(b, -e[:, :, None]).view(v.shape).to(torch.float8_e4m3fn)
    return q, (e + 127).to(U8).view(torch.float8_e8m0fnu)


def _prep_swiglu(c, g):
    rows, I, k = c["rows"], c["I"], c["k"]
    y13 = torch.randn(rows, 2 * I, generator=g, device=DEV)
    y13 = y13.mul_(torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))).to(BF16)
    c["y13"], c["yq"], c["ys"], c["hq"], c["hs"] = y13, None, None, None, None
    if c["op"] == "save":
        for n, cols, dt in (("hq", I, U8), ("hs", I // 128, U8), ("yq", 2 * I, U8),
                            ("ys", 2 * I // 128, U8)):
            c[n] = torch.empty(rows, cols, dtype=dt, device=DEV)
        return c
    if c["saved"]:
        h = torch.empty(rows, I, dtype=F32, device=DEV)
        for r in _rows(rows, I):
            gate = y13[r, :I].float()
            h[r] = gate / (1 + torch.exp(-gate)) * y13[r, I:].float()
        hq, hs = _codes(h)
        yq, ys = _codes(y13)
        c["hq"], c["hs"], c["yq"], c["ys"] = (t.view(U8) for t in (hq, hs, yq, ys))
        c["y13"] = None
    c["dh"] = _normal(g, rows, I, scale=0.1)
    c["dy13"] = torch.empty(rows, 2 * I, dtype=BF16, device=DEV)
    c["w"] = c["perm"] = c["dw"] = None
    if c["weighted"]:  # T tokens' routed rows, then those of the shared expert
        T = rows // (k + 1)
        c["perm"] = torch.randperm(T * k, generator=g, device=DEV).to(I32)
        c["w"] = torch.rand(T, k, generator=g, device=DEV)
        c["dw"] = torch.empty(T, k, device=DEV)
    return c


def _prep_product(c, g):
    _routing(c, g)
    H, I, G, Rs = c["H"], c["I"], len(c["off_host"]) - 1, c["Rs"]
    c["K"], c["N"] = (H, I) if c["op"] == "w2_bwd" else (2 * I, H)
    c["dy"] = _normal(g, Rs, c["K"])
    # codes of every value; scales that keep the rows' products near one
    mid = 127 - int(round(math.log2(3 * math.sqrt(c["K"]))))
    c["wq"] = torch.randint(0, 256, (G, c["K"], c["N"] // 2), generator=g, device=DEV, dtype=U8)
    c["ws"] = torch.randint(mid - 2, mid + 3, (G, c["K"], c["N"] // 32), generator=g, device=DEV,
                            dtype=U8)
    c["dx"] = torch.zeros(Rs, c["N"], dtype=BF16, device=DEV)
    return c


# ------------------------------------------------------------------------- the calls
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _fp8(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _dims(moe, c):
    d = c.get("d")
    if d is None:
        d = c["d"] = moe.dims(c["T"], c["H"], c.get("I", 128), c["E"], c["k"], c["shared"])
    return d


def _own_dispatch(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_dispatch(_dims(moe, c), c["x"], c["inv"], c["xp"])
    return dict(xp=c["xp"])


def _own_dispatch_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_dispatch_backward(_dims(moe, c), c["dxp"], c["inv"], c["dx"], dx_in=c["dx_in"])
    return dict(dx=c["dx"])


def _own_combine_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_combine_backward(_dims(moe, c), c["dout"], c["y2"], c["inv"], c["w"], dy2=c["dy2"],
                             dw=c["dw"])
    return dict(dy2=c["dy2"], dw=c["dw"])


def _own_save(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_swiglu_quant_save(c["y13"], c["hq"], c["hs"], c["yq"], c["ys"])
    (hq, hs), (yq, ys) = _fp8(c["hq"], c["hs"]), _fp8(c["yq"], c["ys"])
    return dict(hq=hq, hs=hs, yq=yq, ys=ys)


def _own_swiglu_bwd(c):
    import moe_expert_ffn_scan_gb300 as moe
    moe.moe_swiglu_backward(c["dh"], c["dy13"], y13=c["y13"], yq=c["yq"], ys=c["ys"], hq=c["hq"],
                            hs=c["hs"], perm_src=c["perm"], w=c["w"], dw=c["dw"])
    return dict(dy13=c["dy13"], dw=c["dw"])


def _own_product(c):
    import moe_expert_ffn_scan_gb300 as moe
    d, ws = _dims(moe, c), c.get("work")
    if ws is None:
        ws = c["work"] = moe.alloc_workspace(moe.gemm_backward_workspace_size(d))
    call = moe.moe_grouped_gemm_w2_backward if c["op"] == "w2_bwd" \
        else moe.moe_grouped_gemm_w13_backward
    call(d, c["dy"], c["off"], c["wq"], c["ws"], c["dx"], ws)
    return dict(dx=c["dx"])


_OWN = {"dispatch": _own_dispatch, "dispatch_bwd": _own_dispatch_bwd,
        "combine_bwd": _own_combine_bwd, "save": _own_save, "swiglu_bwd": _own_swiglu_bwd,
        "w2_bwd": _own_product, "w13_bwd": _own_product}


# ------------------------------------------------------------------------- plain forms
def _slots(c):
    """Each routed slot's row, and whether it has one."""
    inv = c["inv"].long()
    return torch.where(inv >= 0, inv, torch.zeros_like(inv)), inv >= 0


def _plain_dispatch(c):
    T, k = c["T"], c["k"]
    row, has = _slots(c)
    out = torch.zeros(c["Rs"] + 1, c["H"], dtype=BF16, device=DEV)
    row = torch.where(has, row, torch.full_like(row, c["Rs"])).view(T, k)
    for j in range(k):
        out[row[:, j]] = c["x"]
    if c["shared"]:
        out[c["R"]:c["Rs"]] = c["x"]
    return dict(xp=out[:c["Rs"]])


def _plain_dispatch_bwd(c):
    row, has = _slots(c)
    row, has = row.view(c["T"], c["k"]), has.view(c["T"], c["k"])
    acc = torch.zeros(c["T"], c["H"], device=DEV) if c["dx_in"] is None else c["dx_in"].float()
    for j in range(c["k"]):
        acc = acc + torch.where(has[:, j, None], c["dxp"][row[:, j]].float(),
                                torch.zeros(1, device=DEV))
    if c["shared"]:
        acc = acc + c["dxp"][c["R"]:].float()
    return dict(dx=acc.to(c["dx"].dtype))


def _plain_combine_bwd(c):
    T, k = c["T"], c["k"]
    row, has = _slots(c)
    row, has = row.view(T, k), has.view(T, k)
    dout = c["dout"].float()
    dy2 = torch.zeros(c["Rs"] + 1, c["H"], dtype=BF16, device=DEV)
    dw = torch.empty(T, k, device=DEV) if c["dw"] is not None else None
    for j in range(k):
        at = torch.where(has[:, j], row[:, j], torch.full_like(row[:, j], c["Rs"]))
        dy2[at] = (dout * c["w"][:, j, None]).to(BF16)
        if dw is not None:
            dot = (dout * c["y2"][row[:, j]].float()).sum(1)
            dw[:, j] = torch.where(has[:, j], dot, torch.zeros_like(dot))
    if c["shared"]:
        dy2[c["R"]:c["Rs"]] = c["dout"]
    return dict(dy2=dy2[:c["Rs"]], dw=dw)


def _plain_save(c):
    I = c["I"]
    gate, up = c["y13"][:, :I].float(), c["y13"][:, I:].float()
    hq, hs = _codes(gate / (1 + torch.exp(-gate)) * up)
    yq, ys = _codes(c["y13"])
    return dict(hq=hq, hs=hs, yq=yq, ys=ys)


def _values(q, s):
    """What codes and scale bytes stand for, in fp32."""
    v = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, 128)
    return torch.ldexp(v, (s.int() - 127)[:, :, None]).view(q.shape)


def _plain_swiglu_bwd(c):
    I = c["I"]
    y = c["y13"].float() if c["y13"] is not None else _values(c["yq"], c["ys"])
    gate, up, dh = y[:, :I], y[:, I:], c["dh"].float()
    sg = 1 / (1 + torch.exp(-gate))
    dw, dhw = None, dh
    if c["w"] is not None:
        R = c["w"].numel()
        perm = c["perm"].long()
        h = _values(c["hq"], c["hs"]) if c["hq"] is not None else gate * sg * up
        dw = torch.empty(R, device=DEV)
        dw[perm] = (dh[:R] * h[:R]).sum(1)
        dw = dw.view(c["w"].shape)
        wr = torch.ones(c["rows"], 1, device=DEV)
        wr[:R, 0] = c["w"].reshape(-1)[perm]
        dhw = dh * wr
    dy = torch.cat([dhw * up * sg * (1 + gate * (1 - sg)), dhw * gate * sg], 1)
    return dict(dy13=dy.to(BF16), dw=dw)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_product(c):
    """Expert after expert: the weights' values in fp32, and one fp32 product."""
    lut = c.get("lut")
    if lut is None:
        v = torch.tensor(E2M1, device=DEV)
        lut = c["lut"] = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)  # of a byte
    out = torch.empty(c["Rs"], c["N"], dtype=BF16, device=DEV)
    off = c["off_host"]
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        w = lut[c["wq"][e].int()].view(c["K"], -1, 32)
        w = torch.ldexp(w, (c["ws"][e].int() - 127)[:, :, None]).view(c["K"], c["N"])
        out[off[e]:off[e + 1]] = (c["dy"][off[e]:off[e + 1]].float() @ w).to(BF16)
    return dict(dx=out)


_PLAIN = {"dispatch": _plain_dispatch, "dispatch_bwd": _plain_dispatch_bwd,
          "combine_bwd": _plain_combine_bwd, "save": _plain_save, "swiglu_bwd": _plain_swiglu_bwd,
          "w2_bwd": _plain_product, "w13_bwd": _plain_product}


# ------------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    if op == "save":
        n = c["rows"] * c["I"]
        return dict(bytes=7 * n + 3 * n // 128, flops=10 * n)
    if op == "swiglu_bwd":
        n = c["rows"] * c["I"]
        byts = n * (2 + 4 + (2 if c["saved"] else 4)) + (2 * n // 128 if c["saved"] else 0)
        if c["weighted"]:
            byts += (n + n // 128 if c["saved"] else 0) + 12 * c["rows"]
        return dict(bytes=byts, flops=20 * n)
    T, H, k, sh = c["T"], c["H"], c["k"], int(c["shared"])
    R, Rs = T * k, T * (k + sh)
    if op == "dispatch":
        return dict(bytes=2 * H * (T + Rs) + 4 * R, flops=0)
    if op == "dispatch_bwd":
        st = 4 if c["dt"] == "fp32" else 2
        return dict(bytes=H * (2 * Rs + st * T * (2 if c["more"] else 1)) + 4 * R, flops=Rs * H)
    if op == "combine_bwd":
        byts = 2 * H * (T + Rs + (R if c["more"] else 0)) + 8 * R + (4 * R if c["more"] else 0)
        return dict(bytes=byts, flops=R * H * (3 if c["more"] else 1))
    I, E = c["I"], c["E"]
    K, N = (H, I) if op == "w2_bwd" else (2 * I, H)
    # experts that are chosen at all (as if at random), and the shared one
    groups = E * (1 - (1 - k / E) ** T) + sh
    return dict(bytes=groups * K * N * (0.5 + 1 / 32) + 2 * Rs * (K + N), flops=2 * Rs * K * N)


# ------------------------------------------------------------------------- float64
def _rows(n, width):
    """Row ranges whose float64 temporaries stay small."""
    step = max(1, (1 << 26) // width)
    return [slice(i, min(n, i + step)) for i in range(0, n, step)]


def exact(case, seed):
    c = prepare(case, seed)
    return {"dispatch": _exact_dispatch, "dispatch_bwd": _exact_dispatch_bwd,
            "combine_bwd": _exact_combine_bwd, "save": _exact_save,
            "swiglu_bwd": _exact_swiglu_bwd, "w2_bwd": _exact_product,
            "w13_bwd": _exact_product}[c["op"]](c)


def _pairs(c):
    """(row, token, slot) of every row that a token has, the shared ones with slot -1."""
    inv = c["inv"].long()
    at = torch.nonzero(inv >= 0)[:, 0]
    row, tok, slot = inv[at], at // c["k"], at % c["k"]
    if c["shared"]:
        t = torch.arange(c["T"], device=DEV)
        row, tok = torch.cat([row, c["R"] + t]), torch.cat([tok, t])
        slot = torch.cat([slot, torch.full_like(t, -1)])
    return row, tok, slot


def _exact_dispatch(c):
    row, tok, _ = _pairs(c)
    xp = torch.zeros(c["Rs"], c["H"], dtype=torch.float64, device=DEV)
    for r in _rows(row.numel(), c["H"]):
        xp[row[r]] = c["x"][tok[r]].double()
    return dict(xp=xp)


def _exact_dispatch_bwd(c):
    row, tok, _ = _pairs(c)
    dx = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    if c["dx_in"] is not None:
        dx += c["dx_in"].double()
    for r in _rows(row.numel(), c["H"]):
        dx.index_add_(0, tok[r], c["dxp"][row[r]].double())
    return dict(dx=dx)


def _exact_combine_bwd(c):
    row, tok, slot = _pairs(c)
    dy2 = torch.zeros(c["Rs"], c["H"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=DEV)
    for r in _rows(row.numel(), c["H"]):
        do, routed = c["dout"][tok[r]].double(), slot[r] >= 0
        w = c["w"].double()[tok[r], slot[r].clamp(min=0)]
        dy2[row[r]] = do * torch.where(routed, w, torch.ones_like(w))[:, None]
        if c["dw"] is not None:
            dot = torch.einsum("rh,rh->r", do, c["y2"][row[r]].double())
            dw[tok[r][routed], slot[r][routed]] = dot[routed]
    return dict(dy2=dy2, dw=dw if c["dw"] is not None else None)


def _exact_codes(v):
    b = v.reshape(v.shape[0], -1, 128)
    top = b.abs().max(2).values
    some = top > 0
    e = torch.ceil(torch.log2(torch.where(some, top, torch.full_like(top, 448.0)) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(some & (top <= 448 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(some, e, torch.zeros_like(e)).clamp(-127, 127)
    q = (b / torch.exp2(e)[:, :, None]).reshape(v.shape).to(torch.float8_e4m3fn).double()
    return q, torch.exp2(e)


def _exact_save(c):
    I, parts = c["I"], []
    for r in _rows(c["rows"], 2 * I):
        y = c["y13"][r].double()
        parts.append(_exact_codes(torch.nn.functional.silu(y[:, :I]) * y[:, I:]) + _exact_codes(y))
    hq, hs, yq, ys = (torch.cat(p) for p in zip(*parts))
    return dict(hq=hq, hs=hs, yq=yq, ys=ys)


def _exact_values(q, s):
    scale = torch.exp2(s.double() - 127)
    return q.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(128, 1)


def _exact_swiglu_bwd(c):
    rows, I = c["rows"], c["I"]
    dy = torch.empty(rows, 2 * I, dtype=torch.float64, device=DEV)
    dw = None
    wr = torch.ones(rows, dtype=torch.float64, device=DEV)
    if c["w"] is not None:
        R, perm = c["w"].numel(), c["perm"].long()
        wr[:R] = c["w"].double().view(-1)[perm]
        dw = torch.zeros(R, dtype=torch.float64, device=DEV)
    for r in _rows(rows, 2 * I):
        y = c["y13"][r].double() if c["y13"] is not None else _exact_values(c["yq"][r], c["ys"][r])
        gate, up, dh = y[:, :I], y[:, I:], c["dh"][r].double()
        sg = torch.sigmoid(gate)
        silu = torch.nn.functional.silu(gate)
        if dw is not None:
            h = _exact_values(c["hq"][r], c["hs"][r]) if c["hq"] is not None else silu * up
            n = max(0, min(r.stop, R) - r.start)
            dw[perm[r.start:r.start + n]] = torch.einsum("ri,ri->r", dh[:n], h[:n])
        dh = dh * wr[r, None]
        dy[r, :I] = dh * up * (sg + silu * (1 - sg))
        dy[r, I:] = dh * silu
    return dict(dy13=dy, dw=dw.view(c["w"].shape) if dw is not None else None)


def _exact_product(c):
    off = c["off_host"]
    if 2.0 * c["Rs"] * c["K"] * c["N"] > 8e12:  # float64's rate is about 1 TFLOP/s
        return None
    values = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    dx = torch.empty(c["Rs"], c["N"], dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a < b:
            w = torch.empty(c["K"], c["N"], dtype=torch.float64, device=DEV)
            w[:, 0::2] = values[(c["wq"][e] & 15).long()]
            w[:, 1::2] = values[(c["wq"][e] >> 4).long()]
            w *= torch.exp2(c["ws"][e].double() - 127).repeat_interleave(32, 1)
            dx[a:b] = c["dy"][a:b].double() @ w
    return dict(dx=dx)
