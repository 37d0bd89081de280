"""fp64 gradients of the layer (numpy): the reference of the backward entry points' tests.

TEST INFRASTRUCTURE, like the rest of this package. Each function restates one entry point's formula
(include/stepmoe.h); ``tests/test_oracle_backward_pins.py`` checks every one of them against
differences of the forward oracle, so a wrong derivation fails there, on the CPU.

The checkpoint: blocks of 32 neighbouring features of a row share the least power of two that brings
their magnitudes to 448 or less; codes are e4m3, rounded to nearest even.
"""
from __future__ import annotations

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode, e4m3_round
from .moe import sigmoid

BLOCK = 32


def checkpoint(v: np.ndarray):
    """(values held [n, m], exponent bytes [m / 32, n]) of rows v [n, m] (m a multiple of 32)."""
    n, m = v.shape
    b = np.asarray(v, dtype=np.float64).reshape(n, m // BLOCK, BLOCK)
    top = np.abs(b).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(top / E4M3_MAX))
    e = np.maximum(e, -126).astype(np.int64)
    scale = np.exp2(e.astype(np.float64))[:, :, None]
    held = e4m3_round((b / scale).astype(np.float32)) * scale
    return held.reshape(n, m), (e + 127).astype(np.uint8).T.copy()


def checkpoint_values(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """Values that codes [n, m] with exponent bytes [m / 32, n] stand for."""
    scale = np.exp2(exps.T.astype(np.float64) - 127.0)
    return e4m3_decode(codes) * np.repeat(scale, BLOCK, axis=1)


def combine_backward(dout, y, perm_row, w):
    """(dy [T*k, H], dw [T, k]) of out[t] = y[T*k + t] + sum_j w[t, j] y[perm_row[t*k + j]]."""
    T, k = w.shape
    pr = perm_row.reshape(T, k)
    dy = np.zeros((T * k, dout.shape[1]))
    dw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            dy[pr[t, j]] = w[t, j] * dout[t]
            dw[t, j] = dout[t] @ y[pr[t, j]]
    return dy, dw


def route_backward(x, logits, idx, dw, scale):
    """(dlogits [T, k] of the selected logits, dW_r [E, H]) of w_j = scale s_j / sum s, s = sigmoid(l)."""
    T, k = idx.shape
    dl = np.zeros((T, k))
    dwr = np.zeros((logits.shape[1], x.shape[1]))
    for t in range(T):
        s = sigmoid(logits[t, idx[t]])
        S = s.sum()
        ds = scale * (dw[t] / S - (dw[t] @ s) / S ** 2)      # quotient rule
        dl[t] = ds * s * (1.0 - s)
        for j in range(k):
            dwr[idx[t, j]] += dl[t, j] * x[t]
    return dl, dwr


def swiglu_backward(g, u, dh, limit=0.0):
    """(h, dg, du) of h = SiLU(min(g, L)) * clip(u, -L, L) (no clamp for L = 0)."""
    gc, uc = (np.minimum(g, limit), np.clip(u, -limit, limit)) if limit > 0 else (g, u)
    s = sigmoid(gc)
    dg, du = dh * uc * s * (1.0 + gc * (1.0 - s)), dh * gc * s
    if limit > 0:
        dg, du = np.where(g <= limit, dg, 0.0), np.where(np.abs(u) <= limit, du, 0.0)
    return gc * s * uc, dg, du


def expert_backward(x, g, u, dy, Wg, Wu, Wd, limit=0.0):
    """(dx, dW_g, dW_u, dW_d) of y = (SiLU(g) u) W_d^T over one expert's rows, g and u as held."""
    h, dg, du = swiglu_backward(g, u, dy @ Wd, limit)
    return dg @ Wg + du @ Wu, dg.T @ x, du.T @ x, dy.T @ h


def permute_backward(dx_rows, perm_row, idx, dl, w_router):
    """dx [T, H]: the shared row, the k routed rows and the router's share of every token."""
    T, k = idx.shape
    dx = dx_rows[T * k: T * k + T].copy()
    pr = perm_row.reshape(T, k)
    for t in range(T):
        for j in range(k):
            dx[t] += dx_rows[pr[t, j]]
            if dl is not None:
                dx[t] += dl[t, j] * w_router[idx[t, j]]
    return dx
