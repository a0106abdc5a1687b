"""Router balance loss (moe_balance_loss) and its gradient against float64: expert counts
across the vector and scalar rows, k = 1 and 16, single tokens, ragged and empty sequences,
masked tokens full of NaN and infinities, rows of -inf.

Tolerances: a probability carries the exponent's rounding (|v - m| <= 32 units of 2^-24 for
any p that matters, a few for expf, the row's sum of 32 + 5 terms and the quotient), so it is
within 128 * 2^-24, relative; sums over tokens and CTAs add one rounding a term on a path:
at most 128 more at these sizes."""

import numpy as np
import pytest
import torch

import moe_expert_ffn_scan_gb300 as moe
from tests import _block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 256 * ref.U32
F32, I32 = torch.float32, torch.int32


def _make(T, E, k, S, mask, seed=0):
    g = torch.Generator().manual_seed(seed * 131 + T * 7 + E)
    lg = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g)
    idx = torch.topk(lg, k, dim=1).indices.to(I32)
    off = None
    if S > 1:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g).sort().values
        if S > 2:
            cuts[1] = cuts[0]
        off = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(I32)
    m = None
    if mask:
        m = (torch.rand(T, generator=g) < 0.7).to(torch.uint8)
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])
        lg[m == 0] = bad[torch.randint(0, 4, (int((m == 0).sum()), 1), generator=g)]
        idx[m == 0] = -7  # what a masked token chose is not looked at
    return lg, idx, off, m


def _dev(*ts):
    return [t.to(DEV) if t is not None else None for t in ts]


def _forward(lg, idx, off, m, S, E):
    k, T = idx.shape[1], lg.shape[0]
    o = dict(counts=torch.full((S, E), -1, dtype=I32, device=DEV),
             n_tokens=torch.full((S,), -1, dtype=I32, device=DEV),
             prob=torch.full((S, E), -1.0, device=DEV), loss=torch.full((S,), -1.0, device=DEV),
             z_loss=torch.full((S,), -1.0, device=DEV))
    ws = moe.alloc_workspace(moe.balance_loss_workspace_size(T, E, k, S))
    ws.fill_(0xA5)
    moe.moe_balance_loss(lg, idx, ws=ws, seq_offsets=off, token_mask=m, **o)
    return o, ws


CASES = [(1, 1, 1, 1, False), (1, 8, 2, 1, False), (7, 384, 8, 1, False), (64, 8, 2, 3, False),
         (300, 61, 3, 9, True), (130, 1024, 16, 2, True), (65, 1023, 4, 5, False),
         (200, 33, 1, 64, True), (5000, 128, 8, 4, True), (97, 500, 6, 1, True),
         (40, 256, 8, 7, False), (129, 130, 2, 2, True), (2, 3, 3, 5, True)]


@pytest.mark.parametrize("T,E,k,S,mask", CASES)
def test_forward(T, E, k, S, mask):
    lg, idx, off, m = _make(T, E, k, S, mask)
    o, ws = _forward(*_dev(lg, idx, off, m), S, E)
    assert moe.moe_check_status(ws) == 0
    c, n, p, loss, z = ref.balance(lg.double().numpy(), idx.numpy(),
                                   off.numpy() if off is not None else None,
                                   m.numpy() if mask else None, S)
    got = {a: b.cpu().double().numpy() for a, b in o.items()}
    assert np.array_equal(got["counts"], c) and np.array_equal(got["n_tokens"], n)
    assert np.all(np.abs(got["prob"] - p) <= TOL * p + 1e-30)
    assert np.all(np.abs(got["loss"] - loss) <= 2 * TOL * loss + 1e-30)
    # logsumexp = max + log(sum): an absolute error of a few units of the larger of the two
    assert np.all(np.abs(got["z_loss"] - z) <= 2 * TOL * (z + 1e-2))
    again, _ = _forward(*_dev(lg, idx, off, m), S, E)
    assert all(torch.equal(o[a], again[a]) for a in o)


@pytest.mark.parametrize("T,E,k,S,mask", CASES)
@pytest.mark.parametrize("parts", ["all", "loss", "dw"])
def test_backward(T, E, k, S, mask, parts):
    lg, idx, off, m = _make(T, E, k, S, mask, seed=1)
    d_lg, d_idx, d_off, d_m = _dev(lg, idx, off, m)
    o, _ = _forward(d_lg, d_idx, d_off, d_m, S, E)
    g = torch.Generator().manual_seed(5)
    dloss = torch.randn(S, generator=g) if parts != "dw" else None
    dz = torch.randn(S, generator=g) if parts == "all" else None
    dw = torch.randn(T, k, generator=g) if parts != "loss" else None
    out = torch.full((T, E), float("nan"), device=DEV)
    a = _dev(dloss, dz, dw)
    moe.moe_balance_loss_backward(d_lg, d_idx, o["counts"], o["n_tokens"], out, *a,
                                  seq_offsets=d_off, token_mask=d_m)
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    want, size = ref.balance_bwd(lg.double().numpy(), idx.numpy(),
                                 off.numpy() if off is not None else None,
                                 m.numpy() if mask else None, S, f(dloss), f(dz), f(dw))
    got = out.cpu().double().numpy()
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= TOL * size + 1e-30)
    if mask:
        assert np.count_nonzero(got[m.numpy() == 0]) == 0


def test_backward_against_differences():
    """Central differences of the float64 loss, z loss and combine weights."""
    T, E, k, S, step = 6, 12, 3, 2, 1e-5
    lg, idx, _, _ = _make(T, E, k, 1, False, seed=2)
    off = torch.tensor([0, 2, 6], dtype=I32)
    g = torch.Generator().manual_seed(3)
    dloss, dz, dw = torch.randn(S, generator=g), torch.randn(S, generator=g), torch.randn(
        T, k, generator=g)
    d = _dev(lg, idx, off)
    o, _ = _forward(*d, None, S, E)
    out = torch.empty(T, E, device=DEV)
    moe.moe_balance_loss_backward(d[0], d[1], o["counts"], o["n_tokens"], out, dloss.to(DEV),
                                  dz.to(DEV), dw.to(DEV), seq_offsets=d[2])

    def total(x):
        loss, z = ref.balance(x, idx.numpy(), off.numpy(), None, S)[3:]
        sel = np.take_along_axis(x, idx.numpy().astype(np.int64), 1)
        w = ref.softmax(sel)[0]
        return (loss @ dloss.double().numpy() + z @ dz.double().numpy() +
                np.sum(w * dw.double().numpy()))

    x = lg.double().numpy()
    for t in range(T):
        for e in range(E):
            s = np.zeros_like(x)
            s[t, e] = step
            assert abs((total(x + s) - total(x - s)) / (2 * step) - out[t, e].item()) < 1e-4


def test_rows_of_minus_infinity():
    """Experts masked by -inf have probability 0; a token without any has none at all."""
    T, E, k = 20, 48, 4
    lg, idx, _, _ = _make(T, E, k, 1, False, seed=4)
    lg[:, 30:] = -float("inf")
    lg[5] = -float("inf")
    lg[6, :] = torch.finfo(F32).min
    idx = torch.topk(lg, k, dim=1).indices.to(I32)
    d = _dev(lg, idx)
    o, ws = _forward(d[0], d[1], None, None, 1, E)
    c, n, p, loss, z = ref.balance(lg.double().numpy(), idx.numpy(), None, None, 1)
    assert np.array_equal(o["counts"].cpu().numpy(), c) and o["n_tokens"].item() == T
    assert np.all(np.abs(o["prob"].cpu().double().numpy() - p) <= TOL * p + 1e-30)
    out = torch.empty(T, E, device=DEV)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    one = torch.ones(1)
    moe.moe_balance_loss_backward(d[0], d[1], o["counts"], o["n_tokens"], out, one.to(DEV), None,
                                  dw.to(DEV))
    want, size = ref.balance_bwd(lg.double().numpy(), idx.numpy(), None, None, 1,
                                 one.double().numpy(), None, dw.double().numpy())
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= TOL * size + 1e-30)
    assert torch.count_nonzero(out[5]).item() == 0


def test_nan_shows():
    """A NaN in a token that counts is seen in its sequence's sums, and only there."""
    lg, idx, _, _ = _make(40, 100, 4, 1, False, seed=9)
    off = torch.tensor([0, 15, 40], dtype=I32)
    clean, _ = _forward(*_dev(lg, idx, off), None, 2, 100)
    lg[20, 77] = float("nan")
    o, _ = _forward(*_dev(lg, idx, off), None, 2, 100)
    assert torch.equal(o["counts"], clean["counts"])
    for n in ("loss", "z_loss", "prob"):
        assert torch.equal(o[n][0], clean[n][0]) and bool(torch.isnan(o[n][1]).all())


def test_device_checks():
    """Experts out of range are reported and not counted; so are decreasing offsets."""
    lg, idx, _, _ = _make(50, 16, 2, 1, False, seed=6)
    idx[3, 1], idx[40, 0] = 16, -1
    o, ws = _forward(*_dev(lg, idx), None, None, 1, 16)
    assert moe.moe_check_status(ws) == moe.STATUS_BAD_INDEX
    assert o["counts"].sum().item() == 98
    off = torch.tensor([0, 30, 20, 50], dtype=I32)
    idx = idx.clamp(0, 15)
    _, ws = _forward(*_dev(lg, idx, off), None, 3, 16)
    assert moe.moe_check_status(ws) == moe.STATUS_BAD_PLAN
    # the next call on the same workspace clears the word
    o, _ = _forward(*_dev(lg, idx), None, None, 1, 16)
    assert o["counts"].sum().item() == 100


def test_tokens_outside_the_sequences():
    lg, idx, _, _ = _make(30, 16, 2, 1, False, seed=7)
    off = torch.tensor([4, 10, 25], dtype=I32)
    d = _dev(lg, idx, off)
    o, ws = _forward(*d, None, 2, 16)
    assert moe.moe_check_status(ws) == 0 and o["n_tokens"].tolist() == [6, 15]
    assert o["counts"].sum(1).tolist() == [12, 30]
    out = torch.empty(30, 16, device=DEV)
    moe.moe_balance_loss_backward(d[0], d[1], o["counts"], o["n_tokens"], out,
                                  torch.ones(2, device=DEV), dw=torch.ones(30, 2, device=DEV),
                                  seq_offsets=d[2])
    assert torch.count_nonzero(out[:4]).item() == 0 and torch.count_nonzero(out[25:]).item() == 0


def test_no_tokens():
    lg, idx = torch.empty(0, 24, device=DEV), torch.empty(0, 2, dtype=I32, device=DEV)
    o, ws = _forward(lg, idx, torch.zeros(4, dtype=I32, device=DEV), None, 3, 24)
    assert moe.moe_check_status(ws) == 0
    assert all(torch.count_nonzero(t).item() == 0 for t in o.values())


def test_counts_agree_with_the_route():
    d = moe.dims(500, 128, 128, 64, 4, 0)
    lg = torch.randn(500, 64, generator=torch.Generator().manual_seed(8)).to(DEV)
    e = lambda *s, dt=I32: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    idx, w, counts = e(500, 4), e(500, 4, dt=F32), e(64)
    moe.moe_route(d, lg, idx, w, counts, e(65), e(2000), e(2000),
                  moe.alloc_workspace(moe.route_workspace_size(d)))
    o, _ = _forward(lg, idx, None, None, 1, 64)
    assert torch.equal(o["counts"][0], counts)


@pytest.mark.parametrize("E", [1024, 1023])
def test_offsets_past_32_bits(E):
    """More than 2^31 logits: the last sequence comes out as in a call of its own."""
    T, k, n = (1 << 31) // E + 500, 4, 300
    g = torch.Generator(device=DEV).manual_seed(2)
    lg = torch.empty(T, E, device=DEV).normal_(generator=g)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=I32)
    off = torch.tensor([0, T - n, T], dtype=I32, device=DEV)
    o, ws = _forward(lg, idx, off, None, 2, E)
    assert moe.moe_check_status(ws) == 0 and o["n_tokens"].tolist() == [T - n, n]
    assert o["counts"].sum(1).tolist() == [(T - n) * k, n * k]
    last, li = lg[-n:].clone(), idx[-n:].clone()
    own, _ = _forward(last, li, None, None, 1, E)
    assert torch.equal(o["counts"][1], own["counts"][0])
    assert bool(((o["prob"][1] - own["prob"][0]).abs() <= TOL * own["prob"][0]).all())
    out, one = torch.empty_like(lg), torch.ones(2, device=DEV)
    moe.moe_balance_loss_backward(lg, idx, o["counts"], o["n_tokens"], out, one, one,
                                  seq_offsets=off)
    o1 = torch.empty_like(last)
    moe.moe_balance_loss_backward(last, li, own["counts"], own["n_tokens"], o1, one[:1], one[:1])
    assert torch.equal(out[-n:], o1)


@pytest.mark.parametrize("off", [[0, 30, 20, 50], [0, 32, 20, 50], [0, 50, 5, 50],
                                 [0] * 1500 + [17, 16, 50], [50, 0], [0, 48, 50, 49]])
def test_decreasing_offsets_are_reported_wherever_they_lie(off):
    """Also where no block of rows that is summed at once has the pair inside it.  Nothing is
    summed then: no counts, and the sums are NaN."""
    lg, idx, _, _ = _make(50, 16, 2, 1, False, seed=6)
    S, off = len(off) - 1, torch.tensor(off, dtype=I32)
    o, ws = _forward(*_dev(lg, idx, off), None, S, 16)
    assert moe.moe_check_status(ws) == moe.STATUS_BAD_PLAN
    assert torch.count_nonzero(o["counts"]).item() == 0
    assert torch.count_nonzero(o["n_tokens"]).item() == 0
    assert all(bool(torch.isnan(o[n]).all()) for n in ("prob", "loss", "z_loss"))
    # the gradient from these counts is zero
    out = torch.full((50, 16), 7.0, device=DEV)
    one = torch.ones(S, device=DEV)
    moe.moe_balance_loss_backward(*_dev(lg, idx), o["counts"], o["n_tokens"], out, one, one,
                                  seq_offsets=off.to(DEV))
    assert torch.count_nonzero(out).item() == 0


@pytest.mark.parametrize("off,inside", [([0, 20, 60], [0, 20, 50]), ([-3, 20, 50], [0, 20, 50]),
                                        ([-9, -1, 70], [0, 0, 50])])
def test_offsets_outside_the_tokens_are_reported(off, inside):
    """They are read as the nearest token there is."""
    lg, idx, _, _ = _make(50, 16, 2, 1, False, seed=6)
    o, ws = _forward(*_dev(lg, idx, torch.tensor(off, dtype=I32)), None, 2, 16)
    assert moe.moe_check_status(ws) == moe.STATUS_BAD_PLAN
    want, ws = _forward(*_dev(lg, idx, torch.tensor(inside, dtype=I32)), None, 2, 16)
    assert moe.moe_check_status(ws) == 0
    assert all(torch.equal(o[n], want[n]) for n in o)


@pytest.mark.parametrize("E", [33, 64, 200, 1024])
@pytest.mark.parametrize("gap", [12.0, 18.0, 40.0, 60.0])
def test_small_losses(E, gap):
    """Tokens that chose experts of small probability (e^-gap): the loss is small, and as near
    to its value as any other."""
    T, k, S = 70, 2, 3
    g = torch.Generator().manual_seed(E)
    lg = torch.randn(T, E, generator=g)
    lg[:, E // 2:] -= gap
    idx = (E // 2 + torch.randint(0, E // 4, (T, k), generator=g)).to(I32)
    off = torch.tensor([0, 30, 30, 70], dtype=I32)
    o, ws = _forward(*_dev(lg, idx, off), None, S, E)
    assert moe.moe_check_status(ws) == 0
    loss = ref.balance(lg.double().numpy(), idx.numpy(), off.numpy(), None, S)[3]
    got = o["loss"].cpu().double().numpy()
    assert np.all(np.abs(got - loss) <= 2 * TOL * loss) and got[1] == 0
    again, _ = _forward(*_dev(lg, idx, off), None, S, E)
    assert torch.equal(o["loss"], again["loss"])


# Expert counts of every shape that a row has in the lanes: scalar rows of up to 128 and 512
# experts (100 and 500 above are whole vectors), and the ends of the vector rows.
MORE = [(150, 101, 5, 3, True), (170, 385, 16, 2, True), (90, 511, 7, 4, False),
        (60, 255, 4, 1, False), (80, 384, 8, 3, True), (77, 512, 8, 2, False),
        (50, 260, 3, 2, True), (40, 516, 16, 1, False), (70, 513, 9, 2, True)]


@pytest.mark.parametrize("T,E,k,S,mask", MORE)
def test_forward_of_every_row_shape(T, E, k, S, mask):
    test_forward(T, E, k, S, mask)


@pytest.mark.parametrize("T,E,k,S,mask", MORE)
@pytest.mark.parametrize("parts", ["all", "loss", "dw"])
def test_backward_of_every_row_shape(T, E, k, S, mask, parts):
    test_backward(T, E, k, S, mask, parts)
