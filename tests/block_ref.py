"""Float64 references of the operators around the scan, in numpy, from their definitions."""
from __future__ import annotations

import math

import numpy as np

EPS32 = 2.0 ** -24   # half a unit in the last place of float32
EPSB = 2.0 ** -8     # of bfloat16 (8 significant bits)


def norm(x, weight, residual, eps):
    h = x if residual is None else x + residual
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * weight
    return y, h


def f8_step(v):
    """Distance of the e4m3 values around v (3 mantissa bits, 2^-9 below 2^-6)."""
    _, e = np.frexp(v)
    return np.ldexp(1.0, np.maximum(e - 1, -6) - 3)


def act(v, name):
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v * 0.5 * (1.0 + np.tanh(0.5 * v))
    if name == "gelu":
        return 0.5 * v * np.vectorize(math.erfc)(-v / math.sqrt(2.0))
    return v


def linear(x, w, bias=None, residual=None, activation=None, xs=None, ws=None):
    """(result, the magnitude that a rounding error of the sum scales with)"""
    s = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if xs is not None:
        s, mag = s * xs[:, None] * ws, mag * xs[:, None] * np.abs(ws)
    if bias is not None:
        s, mag = s + bias, mag + np.abs(bias)
    y = act(s, activation)
    return (y if residual is None else y + residual), mag


def beam(logits, scores, finished=None, end=None):
    """scores, parent, token, finished, and the smallest gap between the values that decide them."""
    B, K, V = logits.shape
    x = np.where(np.isnan(logits), -np.inf, np.minimum(logits, np.finfo(np.float32).max))
    sc = np.where(scores < np.inf, scores, -np.inf)  # False for NaN too
    top = x.max(-1, keepdims=True)
    base = np.where(top == -np.inf, 0.0, top)
    with np.errstate(divide="ignore", invalid="ignore"):
        total = np.log(np.exp(x - base).sum(-1, keepdims=True))
        cand = np.where(x == -np.inf, -np.inf, sc[:, :, None] + ((x - base) - total))
    cand = np.where(sc[:, :, None] == -np.inf, -np.inf, cand)
    if finished is not None:
        cand[finished] = -np.inf
        cand[finished, end] = sc[finished]
    flat = cand.reshape(B, K * V)
    order = np.argsort(-flat, axis=1, kind="stable")
    pick = order[:, :K]
    best = np.take_along_axis(flat, order[:, :K + 1], 1)
    with np.errstate(invalid="ignore"):
        gap = -np.diff(best, axis=1)
    gap = gap[np.isfinite(gap) & (gap > 0)]
    parent, token = pick // V, pick % V
    done = np.zeros((B, K), bool) if finished is None else np.take_along_axis(finished, parent, 1)
    if end is not None:
        done = done | (token == end)
    return np.take_along_axis(flat, pick, 1), parent, token, done, (gap.min() if gap.size else np.inf)
