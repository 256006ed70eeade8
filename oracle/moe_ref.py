"""Oracle of the operators around the packed-MXFP4 products -- test
infrastructure.  Plain NumPy in 64 bits, from the definitions: activations of
an epilogue, the router, products grouped by expert, the weighted sum."""
from __future__ import annotations

import math

import numpy as np

F64 = np.float64


def activate(a, act):
    a = np.asarray(a, F64)
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "relu":
            return np.where(a < 0, 0.0, a)
        if act == "silu":
            return a / (1.0 + np.exp(-a))
        if act == "gelu":
            return a * np.vectorize(lambda v: math.erfc(-v / math.sqrt(2.0)), otypes=[F64])(a) / 2.0
        if act == "gelu_tanh":      # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
            return a / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))
    assert act == "none"
    return a


def route(logits, k, score="softmax", normalize=True, bias=None, weight_scale=1.0):
    """dict(expert, weight (fp64), offsets, token, pos), token by token."""
    x = np.asarray(logits, F64)
    t, e = x.shape
    expert, weight = np.full((t, k), -1, np.int32), np.zeros((t, k))
    with np.errstate(over="ignore", invalid="ignore"):
        for i in range(t):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-x[i]))
            else:
                top = x[i].max()                                    # NaN if any is
                s = np.where(x[i] == -np.inf, 0.0, np.exp(x[i] - top))
                if s.sum() != 0:
                    s = s / s.sum()
            by = x[i] if bias is None else np.where(x[i] == -np.inf, -np.inf, s + np.asarray(bias, F64))
            rank = sorted(range(e), key=lambda j: (0 if np.isnan(by[j]) else 1, 0.0 if np.isnan(by[j]) else -by[j], j))
            chosen = [j for j in rank if not by[j] == -np.inf][:k]
            w = s[chosen]
            if normalize and w.sum() != 0:
                w = w / w.sum()
            expert[i, :len(chosen)] = chosen
            weight[i, :len(chosen)] = w * F64(np.float32(weight_scale))
    flat = expert.reshape(-1)
    slots = np.concatenate([np.flatnonzero(flat == j) for j in range(e)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([(flat == j).sum() for j in range(e)])]).astype(np.int32)
    token, pos = np.full(t * k, -1, np.int32), np.full(t * k, -1, np.int32)
    token[:len(slots)] = slots // k
    pos[slots] = np.arange(len(slots))
    return dict(expert=expert, weight=weight, offsets=offsets, token=token, pos=pos.reshape(t, k))


def grouped(x, w, offsets, rows=None, bias=None):
    """Rows of x [R, K] times their expert's w [E, N, K], plus its bias: (values, written) of the M rows."""
    m = x.shape[0] if rows is None else len(rows)
    y, written = np.zeros((m, w.shape[1])), np.zeros(m, bool)
    for e in range(w.shape[0]):
        for p in range(offsets[e], offsets[e + 1]):
            r = p if rows is None else rows[p]
            y[p] = (x[r] if 0 <= r < x.shape[0] else np.zeros(x.shape[1])) @ w[e].T
            if bias is not None:
                y[p] += bias[e]
            written[p] = True
    return y, written


def combine(z, pos, weight, residual=None):
    """(values, sum of magnitudes) of the weighted sums."""
    t, k = pos.shape
    z = np.asarray(z, F64)
    y = np.zeros((t, z.shape[1])) if residual is None else np.array(residual, F64)
    mag = np.abs(y)
    for i in range(t):
        for j in range(k):
            if 0 <= pos[i, j] < z.shape[0]:
                y[i] += F64(weight[i, j]) * z[pos[i, j]]
                mag[i] += np.abs(F64(weight[i, j]) * z[pos[i, j]])
    return y, mag
