"""A key-value cache held in 4 bits and the attention over it (oracle side).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

New rows: every Q and K head RMS-normalized and turned by positions of several
axes, K rounded to float32 and to bf16, K and V quantized per token and head by
the Q4 rule (oracle/quant.py) with groups along the head's features, NaN taken as 0
and infinities as the largest bf16.  Attention: softmax(scale Q K^T) V over the tokens that a
row sees, in float64, and a bound on the error of a computation whose scores,
probabilities and sums are float32.

Pinned by: tests/test_oracle_kv.py.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import quant as Q

BF16_MAX = float(F.bf16_value(np.array([0x7F7F], np.uint16))[0])


def finite(x):
    x = np.where(np.isnan(x), 0.0, np.asarray(x, np.float64))
    return np.clip(x, -BF16_MAX, BF16_MAX)


def hold(x, fmt):
    """The values that the cache holds of rows x (..., D) of bf16 values."""
    x = finite(x)
    flat = x.reshape(-1, x.shape[-1]).astype(np.float32)
    c, s = Q.quantize(flat, fmt)
    return Q.dequantize(c, s, fmt).reshape(x.shape)


def turn(x, angle, halves):
    """x (M, heads, D), angle (M, pairs): the first 2 pairs features of each head."""
    P = angle.shape[1]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = x.copy()
    i = np.arange(P) if halves else 2 * np.arange(P)
    j = i + P if halves else i + 1
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def head_rows(x, norm=None, eps=1e-6, freq=None, axis=None, pos=None, halves=False):
    """Heads x (M, heads, D) normalized and turned, float64; pos (axes, M)."""
    x = np.asarray(x, np.float64)
    if norm is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + float(np.float32(eps))) * norm
    if freq is not None and len(freq):
        axis = np.zeros(len(freq), int) if axis is None else axis
        x = turn(x, pos[axis].T.astype(np.float64) * np.asarray(freq, np.float32).astype(np.float64), halves)
    return x


def bf16_of(x):
    """Through float32, as the cache's K rows are rounded."""
    with np.errstate(over="ignore"):
        return F.to_bf16(np.asarray(x, np.float64).astype(np.float32).astype(np.float64))


def attend(q, k, v, first, behind, scale, u_p, k_mag=None, v_mag=None):
    """One sequence and K/V head: q (rows, D), k, v (tokens, D); row i sees tokens [first[i], behind[i]).
    Returns O, lse and bounds on their errors: scores and sums in float32, exp2 good to 2^-21, a
    probability rounded to u_p of itself before it meets V.  k_mag, v_mag: magnitudes as they enter the
    sums, where these are not |k|, |v|."""
    n, D = k.shape
    O, lse = np.zeros((len(q), D)), np.full(len(q), -np.inf)
    bo, bl = np.zeros((len(q), D)), np.zeros(len(q))
    k_mag, v_mag = np.abs(k) if k_mag is None else k_mag, np.abs(v) if v_mag is None else v_mag
    for i in range(len(q)):
        lo, hi = max(int(first[i]), 0), min(int(behind[i]), n)
        if hi <= lo:
            continue
        z = scale * (k[lo:hi] @ q[i])
        top = z.max()
        e = np.exp(z - top)
        l = e.sum()
        p = e / l
        O[i], lse[i] = p @ v[lo:hi], top + np.log(l)
        # a score: D products summed, scaled, the maximum taken off (relative to it, to the maximum and to the
        # running maximum, within 2^4 of it)
        dz = 2.0 ** -24 * (D + 4) * scale * (k_mag[lo:hi] @ np.abs(q[i])) + 2.0 ** -22 * (np.abs(z) + abs(top) + 4)
        dp = np.expm1(dz) + 2.0 ** -21
        sums = (hi - lo + 64) * 2.0 ** -24
        dl = (p * dp).sum() + sums                             # relative, of the sum
        bl[i] = dl + 2.0 ** -22 * (abs(lse[i]) + np.log(hi - lo + 1) + 4)
        w = p[:, None] * v_mag[lo:hi]
        bo[i] = ((dp + u_p)[:, None] * w).sum(0) + (sums + dl + 2.0 ** -22) * w.sum(0) + 2.0 ** -30 * v_mag[lo:hi].max(0)
    return O, lse, bo, bl
