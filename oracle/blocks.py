"""64-bit reference of the building blocks: permute / unpermute over a schedule
and linear (dense or grouped by expert), forward and backward, from their
formulas.  Plain NumPy; rows of the schedule as in ``row_of_slot`` [T * k]."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erf

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def permute(x, row_of_slot, k):
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0] * k, x.shape[1]))
    out[np.asarray(row_of_slot)] = np.repeat(x, k, axis=0)
    return out


def permute_backward(dxs, row_of_slot, k):
    dxs = np.asarray(dxs, np.float64)[np.asarray(row_of_slot)]
    return dxs.reshape(-1, k, dxs.shape[1]).sum(1)


def unpermute(o, row_of_slot, w, residual=None):
    T, k = w.shape
    rows = np.asarray(o, np.float64)[np.asarray(row_of_slot)].reshape(T, k, -1)
    y = np.einsum("tkh,tk->th", rows, np.asarray(w, np.float64))
    return y if residual is None else y + np.asarray(residual, np.float64)


def unpermute_backward(o, dy, row_of_slot, w, idx, E):
    """(do, dw, d_logits)"""
    T, k = w.shape
    row_of_slot = np.asarray(row_of_slot)
    w, dy = np.asarray(w, np.float64), np.asarray(dy, np.float64)
    rows = np.asarray(o, np.float64)[row_of_slot].reshape(T, k, -1)
    do = np.zeros((T * k, dy.shape[1]))
    do[row_of_slot] = (w[:, :, None] * dy[:, None, :]).reshape(T * k, -1)
    dw = np.einsum("tkh,th->tk", rows, dy)
    dl = np.zeros((T, E))
    # added, not put: a caller's table may name an expert twice
    np.add.at(dl, (np.arange(T)[:, None], np.asarray(idx, np.int64)), w * (dw - (w * dw).sum(1, keepdims=True)))
    return do, dw, dl


def act(name, z):
    z = np.asarray(z, np.float64)
    if name == "none":
        return z.copy()
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    raise ValueError(name)


def act_grad(name, z):
    z = np.asarray(z, np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    raise ValueError(name)


def _groups(M, w, offsets):
    """(expert, first row, end row, its weights) of each group; w [N, K] for a dense product."""
    if offsets is None:
        return [(0, 0, M, np.asarray(w, np.float64))]
    return [(e, int(offsets[e]), int(offsets[e + 1]), np.asarray(w[e], np.float64)) for e in range(len(offsets) - 1)]


def linear(x, w, bias=None, residual=None, name="none", offsets=None):
    """(y, z, mag): mag = |x| |w|^T + |bias|, the scale of z's rounding errors.
    Rows in no group are NaN."""
    x = np.asarray(x, np.float64)
    M, N = x.shape[0], w.shape[-2]
    z, mag = np.full((M, N), np.nan), np.full((M, N), np.nan)
    for e, a, b, we in _groups(M, w, offsets):
        z[a:b] = x[a:b] @ we.T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(we).T
        if bias is not None:
            be = np.asarray(bias if offsets is None else bias[e], np.float64)
            z[a:b] += be
            mag[a:b] += np.abs(be)
    y = act(name, z)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z, mag


def linear_backward(x, w, z, dy, name="none", offsets=None):
    """{"dx", "dw", "db"} and under "mag" the same sums over absolute values."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    M, K = x.shape
    N = dy.shape[1]
    dz = dy * (act_grad(name, z) if name != "none" else 1.0)
    lead = () if offsets is None else (len(offsets) - 1,)
    out, mag = [{"dx": np.full((M, K), np.nan), "dw": np.zeros((*lead, N, K)), "db": np.zeros((*lead, N))}
                for _ in range(2)]
    for e, a, b, we in _groups(M, w, offsets):
        for o, f in ((out, lambda v: v), (mag, np.abs)):
            d = f(dz[a:b])
            dwe, dbe = d.T @ f(x[a:b]), d.sum(0)
            o["dx"][a:b] = d @ f(we)
            if offsets is None:
                o["dw"], o["db"] = dwe, dbe
            else:
                o["dw"][e], o["db"][e] = dwe, dbe
    out["mag"] = mag
    return out
