"""Operators around the routed FFN in 64 bits: routing rules, block norms, the
linear layer, and their gradients, written from the formulas of include/moe.h.

Inputs are float arrays that hold the values the kernels read.  Functions whose
results are sums also return `mag`, the same sums taken over magnitudes: the
scale that a bound on rounding errors is proportional to.
"""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


# ------------------------------------------------------------------ routing
def clean_scores(s):
    """Scores as the rules read them: NaN masks like -inf, +inf is the largest finite value."""
    s = np.asarray(s, dtype=np.float64)
    return np.minimum(np.where(np.isnan(s), -np.inf, s), F32_MAX)


def probabilities(s, score):
    s = clean_scores(s)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-s))
    top = s.max(axis=1, keepdims=True)
    live = s > -np.inf
    e = np.where(live, np.exp(np.where(live, s - np.where(np.isfinite(top), top, 0.0), 0.0)), 0.0)
    total = e.sum(axis=1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route(s, k, score="softmax", bias=None, n_group=1, topk_group=1, group_best=1, renormalise=True, scale=1.0):
    """(ids, w, margin): margin[t] = the smallest nonzero gap between two values whose
    order the selection of row t used (inf if none was close)."""
    s = clean_scores(s)
    T, E = s.shape
    p = probabilities(s, score)
    live = s > -np.inf
    key = s + 0.0 if bias is None else p + np.asarray(bias, dtype=np.float64)[None, :]
    ids = np.zeros((T, k), dtype=np.int32)
    margin = np.full(T, np.inf)
    gs = E // n_group
    for t in range(T):
        groups = range(n_group)
        if n_group > 1:
            rank = []
            for g in range(n_group):
                at = [e for e in range(g * gs, (g + 1) * gs) if live[t, e]]
                v = [p[t, e] if bias is None and group_best == 2 else key[t, e] for e in at]
                v = sorted(v, reverse=True)[:group_best]
                rank.append(sum(v) if v else -np.inf)
            order = sorted(groups, key=lambda g: (-rank[g], g))
            groups = sorted(order[:topk_group])
            if topk_group < n_group:
                margin[t] = min(margin[t], _gap(rank[order[topk_group - 1]], rank[order[topk_group]]))
        at = [e for g in groups for e in range(g * gs, (g + 1) * gs)]
        order = sorted(at, key=lambda e: (0, -key[t, e], e) if live[t, e] else (1, 0.0, e))
        ids[t] = order[:k]
        for a, b in zip(order[:k], order[1:k + 1]):
            if live[t, a] and live[t, b]:
                margin[t] = min(margin[t], _gap(key[t, a], key[t, b]))
    w = np.take_along_axis(p, ids.astype(np.int64), 1)
    if renormalise:
        w = shares(np.take_along_axis(s, ids.astype(np.int64), 1), score)
    return ids, w * scale, margin


def log_sigmoid(s):
    """log(1 / (1 + e^-s)) of cleaned scores, exact where the sigmoid itself underflows."""
    return np.where(s < 0, s, 0.0) - np.log1p(np.exp(-np.abs(s)))


def shares(s, score):
    """p / sum(p) along each row: a softmax of the logarithms of p."""
    return probabilities(log_sigmoid(s) if score == "sigmoid" else s, "softmax")


def _gap(a, b):
    return abs(a - b) if a != b and np.isfinite(a) and np.isfinite(b) else np.inf


def route_backward(s, ids, dw, score="softmax", renormalise=True, scale=1.0):
    """Gradient of sum(w * dw) into the scores, for given ids."""
    s = clean_scores(s)
    ids = np.asarray(ids, dtype=np.int64)
    g = scale * np.asarray(dw, dtype=np.float64)
    ds = np.zeros_like(s)
    rows = np.arange(s.shape[0])[:, None]
    if renormalise and score == "softmax":
        r = probabilities(np.take_along_axis(s, ids, 1), "softmax")
        ds[rows, ids] = r * (g - (r * g).sum(axis=1, keepdims=True))
        return ds
    p = probabilities(s, score)
    ps = np.take_along_axis(p, ids, 1)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            q = 1.0 / (1.0 + np.exp(np.take_along_axis(s, ids, 1)))
        if renormalise:
            r = shares(np.take_along_axis(s, ids, 1), score)
            ds[rows, ids] = r * (g - (r * g).sum(axis=1, keepdims=True)) * q
        else:
            ds[rows, ids] = g * ps * q
        return ds
    full = np.zeros_like(s)
    full[rows, ids] = g
    return p * (full - (ps * g).sum(axis=1, keepdims=True))


# ------------------------------------------------------------------ block norms
def _vec(v, H, none):
    return np.full(H, none) if v is None else np.asarray(v, dtype=np.float64)


def _unit(v, kind, eps):
    """(normalised rows, 1 / std)"""
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    return v * r, r


def _gate(gate):
    if gate is None:
        return 1.0
    g = np.asarray(gate["values"], dtype=np.float64)
    return g[:, None] if gate["kind"] == "token" else g


def norm(h, o, gate, w_post, b_post, w_pre, b_pre, post, pre, eps, alpha, beta):
    """(h_out, x_out, mag of h_out, mag of x_out); post / pre: None, "rms" or "layer"."""
    h, o = np.asarray(h, np.float64), np.asarray(o, np.float64)
    H = h.shape[1]
    n, mag_n = o, np.abs(o)
    if post:
        u, r = _unit(o, post, eps)
        n = u * _vec(w_post, H, 1.0) + _vec(b_post, H, 0.0)
        mag_n = (np.abs(o) + np.abs(o).mean(axis=1, keepdims=True)) * r * np.abs(_vec(w_post, H, 1.0)) + np.abs(
            _vec(b_post, H, 0.0))
    g = _gate(gate)
    out = beta * h + alpha * g * n
    mag = np.abs(beta * h) + np.abs(alpha * g) * mag_n
    if not pre:
        return out, None, mag, None
    u, r = _unit(out, pre, eps)
    w, b = _vec(w_pre, H, 1.0), _vec(b_pre, H, 0.0)
    x = u * w + b
    mag_x = (mag + mag.mean(axis=1, keepdims=True)) * r * np.abs(w) + np.abs(b)
    # the second moment's own error scales the whole row
    mag_x = mag_x + np.abs(u * w) * (mag * np.abs(out)).mean(axis=1, keepdims=True) * r * r
    return out, x, mag, mag_x


def _unit_grad(v, dn, kind, eps):
    """(gradient into v of its normalised value, u, its mag)"""
    u, r = _unit(v, kind, eps)
    m1 = (dn * u).mean(axis=1, keepdims=True)
    d = dn - u * m1
    mag = np.abs(dn) + np.abs(u) * np.abs(dn * u).mean(axis=1, keepdims=True)
    if kind == "layer":
        d = d - dn.mean(axis=1, keepdims=True)
        mag = mag + np.abs(dn).mean(axis=1, keepdims=True)
        # u itself is a difference
        mag = mag + (np.abs(v) + np.abs(v).mean(axis=1, keepdims=True)) * r * np.abs(dn * u).mean(axis=1, keepdims=True)
    return d * r, u, mag * r


def norm_backward(dh_out, dx_out, h_out, o, gate, w_post, b_post, w_pre, post, pre, eps, alpha, beta):
    """{name: (value, mag)} for dh, do, dgate, dw_post, db_post, dw_pre, db_pre."""
    o = np.asarray(o, np.float64)
    H = o.shape[1]
    G = np.zeros_like(o) if dh_out is None else np.asarray(dh_out, np.float64)
    mag = np.abs(G)
    out = {}
    if pre:
        dx = np.asarray(dx_out, np.float64)
        d, u, m = _unit_grad(np.asarray(h_out, np.float64), dx * _vec(w_pre, H, 1.0), pre, eps)
        G, mag = G + d, mag + m
        out["dw_pre"] = ((dx * u).sum(axis=0), (np.abs(dx) * (np.abs(u) + 1.0)).sum(axis=0))
        out["db_pre"] = (dx.sum(axis=0), np.abs(dx).sum(axis=0))
    out["dh"] = (beta * G, abs(beta) * mag)
    g = _gate(gate)
    dn, mag_dn = alpha * g * G, np.abs(alpha * g) * mag
    n = o
    if post:
        w = _vec(w_post, H, 1.0)
        do, u, m = _unit_grad(o, dn * w, post, eps)
        _, r = _unit(o, post, eps)
        mw = mag_dn * np.abs(w)
        m = m + r * (mw + np.abs(u) * (mw * np.abs(u)).mean(axis=1, keepdims=True) + mw.mean(axis=1, keepdims=True))
        out["do"] = (do, m)
        out["dw_post"] = ((dn * u).sum(axis=0), (mag_dn * (np.abs(u) + 1.0)).sum(axis=0))
        out["db_post"] = (dn.sum(axis=0), mag_dn.sum(axis=0))
        n = u * w + _vec(b_post, H, 0.0)
        mag_n = (np.abs(u) + 1.0) * np.abs(w) + np.abs(_vec(b_post, H, 0.0))
    else:
        out["do"] = (dn, mag_dn)
        mag_n = np.abs(o)
    if gate is not None:
        t, mt = alpha * G * n, abs(alpha) * mag * mag_n
        axis = {"channel": 0, "token": 1, "full": None}[gate["kind"]]
        out["dgate"] = (t, mt) if axis is None else (t.sum(axis=axis), mt.sum(axis=axis))
    return out


# ------------------------------------------------------------------ linear layer
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def linear(x, w, bias, residual, name, alpha):
    """(y, z, mag of z)"""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, mag = z + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    y = alpha * act(z, name)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z, mag


def linear_backward(dy, x, w, z, name, alpha):
    """{name: (value, mag)} for dx, dw, dbias."""
    dy, x, w = (np.asarray(v, np.float64) for v in (dy, x, w))
    dz = alpha * dy * (1.0 if name == "none" else act_grad(np.asarray(z, np.float64), name))
    return {"dx": (dz @ w, np.abs(dz) @ np.abs(w)), "dw": (dz.T @ x, np.abs(dz).T @ np.abs(x)),
            "dbias": (dz.sum(axis=0), np.abs(dz).sum(axis=0))}
