"""The dense blocks' operators in 64 bits: the gated linear layer and its gradient,
quantisation in blocks of 128, and products of e4m3 operands with block scales, written
from the formulas of include/moe.h.

As in oracle/blocks.py a sum comes with its `mag`, the sum over magnitudes that bounds on
rounding errors are proportional to.
"""
from __future__ import annotations

import numpy as np

from .blocks import act, act_grad
from .formats import e4m3_decode, e4m3_encode

GROUP = 128


def _pre(x, w, bias):
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        b = np.asarray(bias, np.float64)
        z, mag = z + b, mag + np.abs(b)
    return z, mag


def gated(x, w, bias, name):
    """(h, z, mag of z), z = [g, u] = x w^T + bias, h = act(g) u."""
    z, mag = _pre(x, w, bias)
    N = z.shape[1] // 2
    return act(z[:, :N], name) * z[:, N:], z, mag


def gated_backward(dh, x, w, z, name):
    """{name: (value, mag, soft)} for dx, dw, dbias; soft sums the magnitudes that an absolute
    error of the activation or its slope at g, in units of 1 + |g|, is multiplied by."""
    dh, x, w, z = (np.asarray(v, np.float64) for v in (dh, x, w, z))
    N = z.shape[1] // 2
    g, u = z[:, :N], z[:, N:]
    dz = np.concatenate([dh * u * act_grad(g, name), dh * act(g, name)], 1)
    soft = np.concatenate([np.abs(dh * u), np.abs(dh)], 1) * (1.0 + np.abs(np.concatenate([g, g], 1)))
    a = np.abs(dz)
    return {"dx": (dz @ w, a @ np.abs(w), soft @ np.abs(w)), "dw": (dz.T @ x, a.T @ np.abs(x), soft.T @ np.abs(x)),
            "dbias": (dz.sum(axis=0), a.sum(axis=0), soft.sum(axis=0))}


def quantise(v, block_rows):
    """(codes uint8 [M, K], fp32 scales [ceil(M / block_rows), ceil(K / 128)]) of fp32 values: s =
    amax / 448 per block in fp32 (1 where that is 0), code e4m3(v / s) of the fp32 quotient.  NaN
    has no part in amax and the code 0x7f or 0xff; an infinity makes s infinite."""
    v = np.asarray(v, np.float32)
    M, K = v.shape
    scales = np.empty((-(-M // block_rows), -(-K // GROUP)), np.float32)
    codes = np.empty((M, K), np.uint8)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                at = np.s_[i * block_rows:(i + 1) * block_rows, j * GROUP:(j + 1) * GROUP]
                b = v[at]
                s = np.float32(np.nanmax(np.abs(b))) / np.float32(448) if not np.all(np.isnan(b)) else np.float32(0)
                s = s if s > 0 else np.float32(1)
                scales[i, j] = s
                q = b / s
                codes[at] = np.where(np.isnan(q), np.where(np.signbit(q), 0xff, 0x7f), e4m3_encode(np.where(np.isnan(q), 0, q)))
    return codes, scales


def dequantise(codes, scales, block_rows):
    """The values that codes and scales stand for, in 64 bits."""
    M, K = codes.shape
    s = np.asarray(scales, np.float64)
    return e4m3_decode(codes).astype(np.float64) * s.repeat(block_rows, 0)[:M].repeat(GROUP, 1)[:, :K]
