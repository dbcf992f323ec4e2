"""Mixture of experts for few tokens (oracle side).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

The router: logits X Wr^T, scores by softmax or sigmoid, the top_k experts by
score + bias (largest first, the lower index first among equals, a NaN behind
every other value), weights the scores, optionally divided by their sum (0 when
that is 0), times a scale.  The experts: h = act(X Wg^T + bg) (X Wu^T + bu),
Y = sum_j weights_j (h_j Wd^T + bd) over a token's experts, the weights 4-bit
(oracle/quant.py); an expert index outside [0, E) adds nothing.  All in float64
on the exact operands.

Pinned by: tests/test_oracle_moe.py.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import layer as Ly


def _softmax(l):
    with np.errstate(invalid="ignore"):
        e = np.exp(l - np.fmax.reduce(l, axis=1, initial=-np.inf, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)


def route(X_bits, Wr_bits, top_k: int, bias=None, sigmoid=False, renorm=True, scale=1.0):
    """ids (int32 M x top_k) and weights (float64)."""
    with np.errstate(invalid="ignore", over="ignore"):
        logits = F.bf16_value(X_bits) @ F.bf16_value(Wr_bits).T
        p = 1.0 / (1.0 + np.exp(-logits)) if sigmoid else _softmax(logits)
        key = p if bias is None else p + np.asarray(bias, np.float64)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]          # NaN sorts last
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        s = w.sum(axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            w = np.where(s == 0, 0.0, w / np.where(s == 0, 1.0, s))
    return ids.astype(np.int32), w * scale


def silu(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def experts(X_bits, ids, weights, gate_up, gu_bias, down, dn_bias, gelu_act=False, mags=None, eps=None):
    """Y (float64 M x N).  gate_up (E x 2F x H) and down (E x N x F) are dequantized values,
    biases float64 or None.  With mags = (gate_up, down) magnitudes as they enter a kernel's sums
    and eps = (relative rounding of the gate and up sums, of the down sums), also returns a bound
    on |error of Y| per element."""
    x = F.bf16_value(X_bits).astype(np.float64)
    E, F2, _ = gate_up.shape
    half = F2 // 2
    Y, bound = np.zeros((x.shape[0], down.shape[1])), np.zeros((x.shape[0], down.shape[1]))
    for m in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e, wt = int(ids[m, j]), float(weights[m, j])
            if not 0 <= e < E:
                continue
            z = gate_up[e] @ x[m] + (0.0 if gu_bias is None else gu_bias[e])
            g, u = z[:half], z[half:]
            a = Ly.gelu(g) if gelu_act else silu(g)
            h = a * u
            o = down[e] @ h + (0.0 if dn_bias is None else dn_bias[e])
            Y[m] += wt * o
            if mags is not None:
                dz = eps[0] * (mags[0][e] @ np.abs(x[m]) + np.abs(z))
                # act' is below 1.13 for both; the activation itself is computed to 2^-20 of
                # max(|g|, 1) (its exponential or polynomial)
                da = 1.13 * dz[:half] + 2.0 ** -20 * np.maximum(np.abs(g), 1.0)
                dh = da * (np.abs(u) + dz[half:]) + np.abs(a) * dz[half:] + 2.0 ** -22 * np.abs(h)
                bound[m] += abs(wt) * (np.abs(down[e]) @ dh + eps[1] * (mags[1][e] @ (np.abs(h) + dh) + np.abs(o)))
    return (Y, bound) if mags is not None else Y
