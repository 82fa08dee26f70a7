"""64-bit reference of routing with scores and groups, layer / rms norm and
linear with 4-bit weights, forward and backward, from their formulas.  Plain
NumPy."""
from __future__ import annotations

import numpy as np

from .blocks import act


# ------------------------------------------------------------------ routing
def scores(logits, score):
    l = np.array(logits, np.float64)
    l[np.isnan(l)] = -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
        z = e.sum(1, keepdims=True)
        return np.divide(e, z, out=np.zeros_like(e), where=z > 0)


def _best(c, n, allowed=None):
    """The indices of the n largest of c, in descending order, ties to the lower one."""
    at = [i for i in range(len(c)) if allowed is None or allowed[i]]
    return sorted(at, key=lambda i: (-c[i], i))[:n]


def chosen_share(logits, idx, score):
    """The chosen scores over their sum (0 where that is 0), without underflow where all are tiny."""
    l = np.array(logits, np.float64)
    l[np.isnan(l)] = -np.inf
    l = np.take_along_axis(l, idx, 1)
    m = l.max(1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            p = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
        else:                                    # log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|))
            logs = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
            p = np.where(l == -np.inf, 0.0, np.exp(logs - logs.max(1, keepdims=True)))
    s = p.sum(1, keepdims=True)
    return np.divide(p, s, out=np.zeros_like(p), where=s > 0)


def route(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(idx, w, scores)"""
    s = scores(logits, score)
    T, E = s.shape
    if bias is None and (n_group == 1 or group_top == 1):
        c = np.array(logits, np.float64)          # the scores' own order, where 64 bits of them would tie
    else:
        c = s + (0 if bias is None else np.asarray(bias, np.float64))
    c[np.isnan(c)] = -np.inf
    per = E // n_group
    idx = np.zeros((T, k), np.int64)
    for t in range(T):
        allowed = None
        if n_group > 1:
            g = np.sort(c[t].reshape(n_group, per), 1)[:, ::-1]
            with np.errstate(invalid="ignore"):
                g = g[:, 0] + g[:, 1] if group_top == 2 else g[:, 0]
            g = np.where(np.isnan(g), -np.inf, g)
            allowed = np.zeros(n_group, bool)
            allowed[_best(g, topk_group)] = True
            allowed = np.repeat(allowed, per)
        idx[t] = _best(c[t], k, allowed)
    w = chosen_share(logits, idx, score) if renorm else np.take_along_axis(s, idx, 1)
    return idx, w * scale, s


def route_backward(logits, idx, dw, score="softmax", renorm=True, scale=1.0, d_scores=None):
    """d_logits; idx entries outside [0, E) are left out, an expert named twice gets the sum of both."""
    s = scores(logits, score)
    T, E = s.shape
    out = np.zeros((T, E))
    for t in range(T):
        ok = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        at = idx[t, ok]
        a = np.zeros(len(ok))
        if ok and renorm:
            p = chosen_share(np.asarray(logits)[t:t + 1], at[None], score)[0]
            a = scale * p * (dw[t, ok] - (p * dw[t, ok]).sum())
        elif ok:
            a = scale * dw[t, ok] * s[t, at]
        full = np.zeros(E)                       # the scores' gradient times the scores
        np.add.at(full, at, a)
        if d_scores is not None:
            full += s[t] * np.asarray(d_scores, np.float64)[t]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = full / (1 + np.exp(np.asarray(logits, np.float64)[t]))
        else:
            out[t] = full - s[t] * full.sum()
    return out


# ------------------------------------------------------------------ norm
def norm(h, gamma, beta=None, kind="layer", eps=1e-5):
    """(y, mean, rstd) of the rows h (x with the residual added and rounded)"""
    h = np.asarray(h, np.float64)
    mean = h.mean(1) if kind == "layer" else np.zeros(len(h))
    d = h - mean[:, None]
    rstd = 1 / np.sqrt((d ** 2).mean(1) + eps)
    y = d * rstd[:, None] * np.asarray(gamma, np.float64)
    return (y if beta is None else y + np.asarray(beta, np.float64)), mean, rstd


def norm_backward(h, gamma, mean, rstd, dy, kind="layer", d_total=None):
    """(dx, dgamma, dbeta) with the statistics given"""
    h, dy = np.asarray(h, np.float64), np.asarray(dy, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (h - (np.asarray(mean, np.float64)[:, None] if kind == "layer" else 0)) * r
    g = dy * np.asarray(gamma, np.float64)
    dx = g - xh * (g * xh).mean(1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdims=True)
    dx = dx * r
    return (dx if d_total is None else dx + np.asarray(d_total, np.float64)), (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------ 4-bit weights
def w4_codes(codes):
    """codes [.., K / 2] -> [.., K]: the low nibble of a byte first."""
    codes = np.asarray(codes)
    out = np.empty((*codes.shape[:-1], codes.shape[-1] * 2), np.int64)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def w4_weights(codes, scales, zeros=None):
    """The weights [.., N, K] that codes [.., N, K / 2], scales and zeros [.., K / group, N] stand for."""
    q = w4_codes(codes)
    scales = np.swapaxes(np.asarray(scales, np.float64), -1, -2)
    G = q.shape[-1] // scales.shape[-1]
    z = 8 if zeros is None else np.repeat(np.swapaxes(np.asarray(zeros, np.int64), -1, -2), G, -1)
    return (q - z) * np.repeat(scales, G, -1)


def linear_w4(x, codes, scales, zeros=None, bias=None, residual=None, activation="none", offsets=None):
    """(y, z, the sum of magnitudes that the fp32 products of codes minus zeros go through)"""
    w = w4_weights(codes, scales, zeros)
    x = np.asarray(x, np.float64)
    dense = offsets is None
    w = w[None] if dense else w
    off = [0, len(x)] if dense else list(offsets)
    b = None if bias is None else np.asarray(bias, np.float64).reshape(len(w), -1)
    z, mag = np.zeros((len(x), w.shape[1])), np.zeros((len(x), w.shape[1]))
    for e in range(len(w)):
        r = slice(off[e], off[e + 1])
        z[r] = x[r] @ w[e].T + (0 if b is None else b[e])
        mag[r] = np.abs(x[r]) @ np.abs(w[e]).T + (0 if b is None else np.abs(b[e]))
    y = act(activation, z)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z, mag


def _to_odd(v):
    """Values that are not negative as float32 for a rounding to 16 bits: towards zero, the last bit set
    where something is lost, so that the second rounding is that of v."""
    f = np.asarray(v, np.float64).astype(np.float32)
    f = np.where(f.astype(np.float64) > v, np.nextafter(f, np.float32(0)), f)
    return np.where(f.astype(np.float64) == v, f, (f.view(np.int32) | 1).view(np.float32))


def w4_quantize(w, group, round_to, zeros=False):
    """(codes [.., N, K], scales [.., K / group, N], zeros or None); round_to(float32 array) gives the
    scales' type's values as float64."""
    w = np.asarray(w, np.float64)
    g = w.reshape(*w.shape[:-1], -1, group)
    lo, hi = np.minimum(g.min(-1), 0), np.maximum(g.max(-1), 0)
    rng = (hi - lo) / 15 if zeros else np.maximum(hi, -lo) / 7
    s = round_to(_to_odd(rng))
    live = s > 0
    safe = np.where(live, s, 1.0)
    z = np.where(live, np.clip(np.rint(-lo / safe), 0, 15), 0) if zeros else np.full(s.shape, 8.0)
    q = np.where(live[..., None], np.clip(np.rint(g / safe[..., None]) + z[..., None], 0, 15), z[..., None])
    out = np.swapaxes(s, -1, -2), (np.swapaxes(z, -1, -2).astype(np.int64) if zeros else None)
    return q.reshape(w.shape).astype(np.int64), *out
