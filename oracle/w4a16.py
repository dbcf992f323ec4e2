"""4-bit weight x 16-bit activation linear (oracle side).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

The Nunchaku in Diffusers page (section "Introducing Nunchaku Lite") names the
second kernel family next to the SVDQuant W4A4 layer: 4-bit weights with 16-bit
activations (AWQ) for the adaptive-normalization and modulation projections,
which are memory-bound and precision-sensitive.  The SVDQuant notes page (its
comparison of SmoothQuant and AWQ with SVDQuant) describes AWQ as
activation-aware weight quantization: the salient
channels are protected by a per-channel scale moved between weights and
activations, which is folded into the weight before quantization (and into the
producer of X), so the kernel itself computes

    Y = X . deQ(Q4(W))^T + b,

X in bf16 (not quantized), W (N x K) quantized with the INT4 rule of
oracle/quant.py (groups of 64 along K, fp16 scale), accumulation exact here
(float64), b in bf16.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import layer as Ly
from . import quant as Q


def forward(X_bits: np.ndarray, W_nk: np.ndarray, b_bits) -> dict:
    """X (M x K bf16 bits), W (N x K float32), b (N bf16 bits or None)."""
    cW, sW = Q.quantize(np.asarray(W_nk, dtype=np.float32), "int4")
    wq = Q.dequantize(cW, sW, "int4")
    x = F.bf16_value(X_bits).astype(np.float64)
    Y = x @ wq.T
    if b_bits is not None:
        Y = Y + F.bf16_value(b_bits).astype(np.float64)[None, :]
    return {"Y": Y, "cW": cW, "sW": sW}


def layer_forward(X_bits, lam, L1_bits, L2_bits, R_nk, b_bits, fmt: str, gelu_act: bool = False) -> dict:
    """A whole packed layer with 16-bit activations: Y = act(X_hat deQ(Q(R))^T + (X_hat L1) L2
    + b), X_hat = fp32(X / lambda) exact from there on.  Also returns the sums of magnitudes
    that bound a kernel's rounding: B (of the 4-bit product's terms, INT4 codes counted as they
    enter the kernel's sums, |24 + q| + 24) and B_lr (of the low-rank product's terms)."""
    x = Ly.smooth(X_bits, lam).astype(np.float64)
    R = np.asarray(R_nk, dtype=np.float32)
    gs = Q.nvfp4_global_scale(R) if fmt == "nvfp4" else np.float32(1.0)
    cR, sR = Q.quantize(R, fmt, gs)
    w = Q.dequantize(cR, sR, fmt, gs)
    mag = np.abs(w)
    if fmt == "int4":
        mag = (np.abs(24 + cR.astype(np.float64)) + 24) * np.repeat(F.fp16_value(sR), 64, axis=1)
    y, B, B_lr = x @ w.T, np.abs(x) @ mag.T, 0.0
    if L1_bits is not None and np.asarray(L1_bits).shape[1] > 0:
        L1, L2 = F.bf16_value(L1_bits), F.bf16_value(L2_bits)
        y = y + (x @ L1) @ L2
        B_lr = (np.abs(x) @ np.abs(L1)) @ np.abs(L2)
    if b_bits is not None:
        y = y + F.bf16_value(b_bits)[None, :]
    return {"Y": Ly.gelu(y) if gelu_act else y, "pre": y, "B": B, "B_lr": B_lr, "w": w, "mag": mag}
