"""Pins of the mixture-of-experts oracle (oracle/moe.py) and of the whole-layer W4A16 oracle."""
from fractions import Fraction

import numpy as np
import pytest

import synth
from oracle import formats as F
from oracle import layer as Ly
from oracle import moe as Mo
from oracle import quant as Q
from oracle import w4a16 as W


def _bits(a):
    return synth.bf16_bits_from_f32(np.asarray(a, np.float32))


def test_route_by_hand():
    # logits of the one token: 1, 3, 3, -2
    X, Wr = _bits([[1.0, 1.0]]), _bits([[1, 0], [1, 2], [2, 1], [-1, -1]])
    ids, w = Mo.route(X, Wr, 3)
    assert ids.tolist() == [[1, 2, 0]]                               # equal: the lower index first
    e = np.exp([3.0, 3.0, 1.0])
    np.testing.assert_allclose(w[0], e / e.sum(), rtol=1e-15)
    ids, w = Mo.route(X, Wr, 2, sigmoid=True, renorm=False, scale=2.0, bias=np.array([0.9, 0, 0, 0], np.float32))
    assert ids.tolist() == [[0, 1]]                                  # the bias chooses, the weights lack it
    np.testing.assert_allclose(w[0], 2.0 / (1.0 + np.exp(-np.array([1.0, 3.0]))), rtol=1e-15)


def test_route_nan_and_zero_sum():
    X, Wr = _bits([[np.nan, 0.0]]), _bits([[1, 0], [0, 1], [1, 1]])
    ids, w = Mo.route(X, Wr, 3)
    assert sorted(ids[0].tolist()) == [0, 1, 2] and np.isnan(w).all()
    X = _bits([[2.0 ** 100, 0.0]])
    ids, w = Mo.route(X, _bits([[-2.0 ** 20, 0], [-2.0 ** 20, 0]]), 1, sigmoid=True)
    assert ids.tolist() == [[0]] and w.tolist() == [[0.0]]


@pytest.mark.parametrize("gelu", [False, True])
def test_experts_against_a_plain_loop(gelu):
    rng = np.random.default_rng(5)
    M, H, Fh, N, E = 3, 4, 3, 5, 2
    X = _bits(rng.standard_normal((M, H)))
    wg, wd = rng.standard_normal((E, 2 * Fh, H)), rng.standard_normal((E, N, Fh))
    bg, bd = rng.standard_normal((E, 2 * Fh)), rng.standard_normal((E, N))
    ids = np.array([[0, 1], [1, 1], [-1, 2]], np.int32)
    wt = rng.standard_normal((M, 2))
    Y = Mo.experts(X, ids, wt, wg, bg, wd, bd, gelu)
    x = F.bf16_value(X)
    for m in range(M):
        for n in range(N):
            want = 0.0
            for j in range(2):
                e = ids[m, j]
                if e not in (0, 1):
                    continue
                o = bd[e, n]
                for f in range(Fh):
                    g = sum(x[m, k] * wg[e, f, k] for k in range(H)) + bg[e, f]
                    u = sum(x[m, k] * wg[e, Fh + f, k] for k in range(H)) + bg[e, Fh + f]
                    a = float(Ly.gelu(np.array([g]))[0]) if gelu else g / (1 + np.exp(-g))
                    o += a * u * wd[e, n, f]
                want += wt[m, j] * o
            assert abs(want - Y[m, n]) <= 1e-12 * max(1.0, abs(want))
    assert np.all(Y[2] == 0)                                         # no expert of its own


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
def test_layer_forward_bruteforce_rational(fmt):
    rng = np.random.default_rng(6)
    M, K, N, r = 2, 64, 3, 2
    X = _bits(rng.standard_normal((M, K)))
    lam = np.exp(rng.standard_normal(K)).astype(np.float32)
    L1, L2 = _bits(rng.standard_normal((K, r))), _bits(rng.standard_normal((r, N)))
    R = rng.standard_normal((N, K)).astype(np.float32)
    b = _bits(rng.standard_normal(N))
    o = W.layer_forward(X, lam, L1, L2, R, b, fmt)
    gs = Q.nvfp4_global_scale(R) if fmt == "nvfp4" else 1.0
    w = Q.dequantize(*Q.quantize(R, fmt, gs), fmt, gs)
    xv = F.bf16_value(X)
    for m in range(M):
        xh = [Fraction(float(np.float32(np.float32(xv[m, k]) / lam[k]))) for k in range(K)]
        for n in range(N):
            acc = Fraction(float(F.bf16_value(b)[n]))
            for k in range(K):
                acc += xh[k] * Fraction(float(w[n, k]))
                for i in range(r):
                    acc += xh[k] * Fraction(float(F.bf16_value(L1)[k, i])) * Fraction(float(F.bf16_value(L2)[i, n]))
            assert abs(float(acc) - o["Y"][m, n]) <= 1e-11 * max(1.0, abs(float(acc)))
    # a kernel's sums hold at least the terms themselves
    assert np.all(o["mag"] >= np.abs(w))
