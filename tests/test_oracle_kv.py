"""Pins of oracle/kv.py: library routines, closed forms, brute force."""
import numpy as np
import pytest

from oracle import kv as Kv
from oracle import qkv


def test_hold_values():
    x = np.zeros((2, 64))
    x[0, :4] = [6.0, -3.0, 0.5, np.nan]
    x[1, 0], x[1, 1] = np.inf, -np.inf
    for fmt in ("mxfp4", "int4", "nvfp4"):
        h = Kv.hold(x, fmt)
        assert np.isfinite(h).all() and h[0, 3] == 0 and (h[0, 8:] == 0).all()
    assert list(Kv.hold(x, "mxfp4")[0, :3]) == [6.0, -3.0, 0.5]
    assert list(Kv.hold(x, "nvfp4")[0, :3]) == [6.0, -3.0, 0.5]
    assert Kv.hold(x, "int4")[0, 0] == pytest.approx(6.0, rel=2.0 ** -11)
    assert Kv.hold(x, "mxfp4")[1, 0] == 6 * 2.0 ** 125 and Kv.hold(x, "nvfp4")[1, 1] == -2688


def test_turn_is_a_rotation():
    rng = np.random.default_rng(1)
    x, a = rng.standard_normal((5, 3, 16)), rng.standard_normal((5, 8))
    ref = qkv.rotate_pairs(x, np.cos(a), np.sin(a))
    assert np.allclose(Kv.turn(x, a, False), ref, atol=1e-14)
    order = np.r_[0:16:2, 1:16:2]                      # neighbours' features as halves
    assert np.allclose(Kv.turn(x[..., order], a, True), ref[..., order], atol=1e-14)
    part = Kv.turn(x, a[:, :3], False)
    assert np.array_equal(part[..., 6:], x[..., 6:]) and np.allclose(part[..., :6], ref[..., :6])
    half = Kv.turn(x, a[:, :4], True)
    assert np.array_equal(half[..., 8:], x[..., 8:])
    assert np.allclose(np.linalg.norm(half, axis=-1), np.linalg.norm(x, axis=-1))


def test_several_axes():
    x = np.ones((2, 1, 4))
    pos = np.array([[1, 2], [10, 20]])
    y = Kv.head_rows(x, freq=[0.5, 0.25], axis=np.array([1, 0]), pos=pos)
    want = Kv.turn(x, np.array([[5.0, 0.25], [10.0, 0.5]]), False)
    assert np.array_equal(y, want)
    w = np.array([1.0, 2, 3, 4])
    assert np.allclose(Kv.head_rows(3 * x, norm=w, eps=0.0), np.broadcast_to(w, x.shape))


def test_attend_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((7, 64)), rng.standard_normal((20, 64)), rng.standard_normal((20, 64))
    behind = 14 + np.arange(7)
    O, lse, bo, bl = Kv.attend(q, k, v, np.zeros(7), behind, 0.125, 0.0)
    mask = torch.from_numpy(np.arange(20)[None] < behind[:, None])
    ref = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(t)[None] for t in (q, k, v)), attn_mask=mask[None])
    assert np.allclose(O, ref[0].numpy(), atol=1e-13)
    z = np.where(mask.numpy(), 0.125 * q @ k.T, -np.inf)
    assert np.allclose(lse, np.log(np.exp(z).sum(1)))
    # a score's error is below 2^-24 68 (0.125 sum |q k| < 16) + 2^-22 16 < 2^-13.5 here, a sum's 84 2^-24: an
    # output's below twice these times the largest |v| < 5
    assert (bo > 0).all() and (bo < 2.0 ** -10).all() and (bl < 2.0 ** -12).all()


def test_attend_windows_and_empty_rows():
    k, v = np.zeros((6, 4)), np.arange(24.0).reshape(6, 4)
    O, lse, _, _ = Kv.attend(np.ones((4, 4)), k, v, [2, 0, 5, 6], [4, 0, 9, 6], 1.0, 0.0)
    assert np.array_equal(O[0], (v[2] + v[3]) / 2) and lse[0] == np.log(2)
    assert (O[1] == 0).all() and lse[1] == -np.inf and np.array_equal(O[2], v[5]) and lse[3] == -np.inf


def test_bound_holds_for_float32():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, 64)) * 3 for n in (8, 500, 500))
    O, lse, bo, bl = Kv.attend(q, k, v, np.zeros(8), np.full(8, 500), 0.125, 2.0 ** -8)
    q, k, v = (t.astype(np.float32) for t in (q.astype(np.float32), k, v))
    z = (q @ k.T) * np.float32(0.125)
    e = np.exp(z - z.max(1, keepdims=True))
    p = Kv.F.to_bf16(e.astype(np.float64))
    o = (p @ v.astype(np.float64)) / e.sum(1, dtype=np.float64)[:, None]
    assert (np.abs(o - O) <= bo + 1e-5 * np.abs(O)).all()
    assert (np.abs(np.log(e.sum(1)) + z.max(1) - lse) <= bl + 1e-5).all()
