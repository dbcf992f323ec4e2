"""Pins of the router oracle's order (oracle/moe.py): by score + bias, the lower index first among equals."""
import numpy as np
import pytest

import synth
from oracle import moe as Mo


def _bits(a):
    return synth.bf16_bits_from_f32(np.asarray(a, np.float32))


@pytest.mark.parametrize("bias", [None, np.zeros(4, np.float32)])
def test_equal_scores_of_other_logits(bias):
    """1 / (1 + exp(-40)) is 1 in float64, as that of 50 is; exp(-800) and exp(-900) are 0."""
    X = _bits([[1.0]])
    ids, w = Mo.route(X, _bits([[1.0], [40.0], [50.0], [45.0]]), 4, bias, sigmoid=True, renorm=False)
    assert ids.tolist() == [[1, 2, 3, 0]] and w[0, :3].tolist() == [1.0, 1.0, 1.0]
    ids, w = Mo.route(X, _bits([[-800.0], [0.0], [-900.0], [-700.0]]), 4, bias)
    assert ids.tolist() == [[1, 3, 0, 2]] and w[0, 2:].tolist() == [0.0, 0.0]


def test_nan_behind_minus_infinity():
    X, Wr = _bits([[1.0]]), _bits([[0.0], [np.nan], [1.0], [1.0], [np.nan]])
    bias = np.array([0, 0, -np.inf, 0, 0], np.float32)
    assert Mo.route(X, Wr, 5, bias, sigmoid=True)[0].tolist() == [[3, 0, 2, 1, 4]]
