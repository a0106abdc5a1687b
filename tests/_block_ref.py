"""float64 numpy forms of the operators around the expert FFN (test code only), written
from their formulas."""

import numpy as np
from scipy.special import erf

U32 = 2.0 ** -24  # half a unit in the last place of fp32, relative
U16 = 2.0 ** -8   # and of bf16


def norm(x, res, gain, eps):
    a = x if res is None else x + res
    rstd = 1.0 / np.sqrt(np.mean(a * a, axis=1) + eps)
    return a, rstd, a * rstd[:, None] * gain


def norm_bwd(dy, h, rstd, gain, dh_in=None):
    n = h * rstd[:, None]
    u = dy * gain
    dh = rstd[:, None] * (u - n * np.mean(u * n, axis=1, keepdims=True))
    if dh_in is not None:
        dh = dh + dh_in
    return dh, np.sum(dy * n, axis=0)


def softmax(x):
    """Rows of probabilities and their logsumexp; rows of -inf alone: zeros."""
    m = np.max(x, axis=1, keepdims=True)
    none = np.isneginf(m)
    with np.errstate(invalid="ignore"):
        e = np.exp(x - np.where(none, 0.0, m))
    s = e.sum(axis=1, keepdims=True)
    p = np.where(none, 0.0, e / np.where(none, 1.0, s))
    lse = np.where(none, 0.0, np.where(none, 0.0, m) + np.log(np.where(none, 1.0, s)))
    return p, lse[:, 0]


def tokens_of(s, off, mask, T):
    b, e = (0, T) if off is None else (int(off[s]), int(off[s + 1]))
    rows = np.arange(b, e)
    return rows if mask is None else rows[mask[rows] != 0]


def balance(logits, idx, off, mask, S):
    T, E = logits.shape
    k = idx.shape[1]
    counts, n = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    prob, loss, z = np.zeros((S, E)), np.zeros(S), np.zeros(S)
    for s in range(S):
        rows = tokens_of(s, off, mask, T)
        n[s] = len(rows)
        if not len(rows):
            continue
        p, lse = softmax(logits[rows])
        flat = idx[rows].reshape(-1)
        counts[s] = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        prob[s] = p.mean(axis=0)
        loss[s] = np.sum(counts[s] * (E / (k * n[s])) * prob[s])
        z[s] = np.mean(lse ** 2)
    return counts, n, prob, loss, z


def balance_bwd(logits, idx, off, mask, S, dloss, dz, dw):
    """The gradient, and the sum of its terms' magnitudes (the scale of its rounding)."""
    T, E = logits.shape
    k = idx.shape[1]
    counts, n = balance(logits, idx, off, mask, S)[:2]
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for s in range(S):
        rows = tokens_of(s, off, mask, T)
        if not len(rows):
            continue
        p, lse = softmax(logits[rows])
        a = np.zeros(E) if dloss is None else dloss[s] * counts[s] * (E / (k * n[s] ** 2))
        c = 0.0 if dz is None else 2 * dz[s] / n[s]
        out[rows] = p * (a - (p @ a)[:, None]) + p * (c * lse)[:, None]
        size[rows] = p * (np.abs(a) + (p @ np.abs(a))[:, None]) + p * np.abs(c * lse)[:, None]
        if dw is not None:
            for t in rows:
                j = [i for i in range(k) if 0 <= idx[t, i] < E]
                sel = logits[t, idx[t, j]]
                if np.all(np.isneginf(sel)):
                    continue
                w = np.exp(sel - sel.max())
                w /= w.sum()
                d = w * (dw[t, j] - np.dot(w, dw[t, j]))
                np.add.at(out[t], idx[t, j], d)
                np.add.at(size[t], idx[t, j], w * (np.abs(dw[t, j]) + np.dot(w, np.abs(dw[t, j]))))
    return out, size


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z / (1 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + erf(z / np.sqrt(2)))
    return z


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0).astype(z.dtype)
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    return np.ones_like(z)
