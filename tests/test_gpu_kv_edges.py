"""The 4-bit key-value cache at its edges: Q heads of any magnitude, rows beside an infinity, windows beyond int32, rows in front
of the sequences."""
import numpy as np
import pytest

import w4a4_quantized_linear_amd as sq
from oracle import kv as Kv

from _kv_helpers import Cache, bits, check_attention, i32

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "int4", "nvfp4"]


@pytest.fixture(scope="module")
def td():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sq.lib()
    assert sq.device_check(), "current device is not gfx950"
    return torch, torch.device("cuda:0")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
@pytest.mark.parametrize("pairs", [0, 16])
def test_append_norm_of_any_magnitude(td, D, eps, pairs):
    """Q heads whose squares leave float32 on either side are normalized as the others, and the others keep their bits
    beside them."""
    torch, dev = td
    kv = sq.KvLayout("mxfp4", 1, D, 16)
    rng = np.random.default_rng(D)
    mags = [2.0 ** e for e in (-133, -126, -100, -80, -66, -45, -41, -40, -39, -20, 0, 20, 58, 61, 62, 64, 80, 100, 125)]
    M, Hq = 5, len(mags)
    x = rng.standard_normal((M, Hq, D)) * np.array(mags)[None, :, None]
    x[0] = np.array(mags)[:, None]                                    # alike values: the largest sums
    x[1, :, 1:] = 0                                                   # one value
    x = np.clip(Kv.F.to_bf16(x), -Kv.BF16_MAX, Kv.BF16_MAX)
    x[:, :, 0] = np.where(np.abs(x).max(-1) == 0, 2.0 ** -133, x[:, :, 0])        # no head of zeros: 0 / 0 with eps 0
    w = Kv.F.to_bf16(1 + 0.2 * rng.standard_normal(D))
    freq = (100.0 ** (-np.arange(pairs) / 16)).astype(np.float32)
    place = np.arange(M)
    bf = lambda t: torch.tensor(np.asarray(t), dtype=torch.float32).bfloat16().to(dev)
    pool = torch.zeros((1, sq.kv_page_bytes(kv)), dtype=torch.uint8, device=dev)
    row, lens, cu = bf(rng.standard_normal((M, D))), i32([M], dev, torch), i32([0, M], dev, torch)
    more = dict(freq=torch.tensor(freq, device=dev)) if pairs else {}
    call = lambda v: sq.kv_append(kv, pool, i32([[0]], dev, torch), lens, row, row, cu=cu, Q=bf(v.reshape(M, -1)), norm_q=bf(w),
                                  eps=eps, **more)
    out = call(x)
    how = dict(freq=freq, pos=place[None]) if pairs else {}
    z = Kv.head_rows(x, w, eps, **how)
    plain = np.abs(Kv.head_rows(x, w, eps))
    # float32: the mean of squares (D / 2 + 8 roundings), root, quotient and products at 2^-24 each, of either feature;
    # bf16's half step, 2^-134 below its normal numbers, and float32's own subnormals on the way
    lim = 2.0 ** -8 * np.abs(z) + (D / 2 + 16) * 2.0 ** -24 * 2 * plain.max(-1, keepdims=True) + 2.0 ** -134 + 2.0 ** -148
    err = np.abs(bits(out).reshape(z.shape) - z)
    assert np.isfinite(bits(out)).all() and (err <= lim).all(), \
        [(m, float((err / lim)[:, i].max())) for i, m in enumerate(mags) if not (err[:, i] <= lim[:, i]).all()]
    ordinary = np.where(np.isin(mags, [2.0 ** -20, 1.0, 2.0 ** 20])[None, :, None], x, 1.0)
    alone = call(ordinary).view(M, Hq, D)
    for i, m in enumerate(mags):
        if m in (2.0 ** -20, 1.0, 2.0 ** 20):
            assert torch.equal(alone[:, i], out.view(M, Hq, D)[:, i])


FORMS = {
    # query rows a sequence, lengths, query heads, heads, columns of the table: each form of the call
    "16 rows": ([1, 1], [700, 900], 4, 1, None),
    "16 rows, ranges": ([1], [9000], 4, 1, None),
    "32 rows": ([6, 5], [700, 900], 4, 1, None),
    "32 rows, ranges": ([6], [9000], 4, 1, None),
    "128 rows": ([768], [2000], 64, 8, None),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", list(FORMS))
def test_attention_rows_beside_an_infinity(td, fmt, name):
    """A row with an infinity, whose scores are lowest at first and highest behind, leaves every bit of the others."""
    torch, dev = td
    q_lens, lens, Hq, H, cols = FORMS[name]
    kv = sq.KvLayout(fmt, H, 64, 32)
    c = Cache(torch, dev, kv, lens, 17, cols=cols, gain=False)
    K = c.K.copy()
    at = np.concatenate([np.arange(n) for n in lens])
    K[:, :, 5] = np.where(at % 700 < 300, -2.0, 2.0)[:, None]
    n32, all32 = i32(lens, dev, torch), i32(c.cu, dev, torch)
    sq.kv_append(kv, c.pool, c.table, n32, c.dev_bf16(K.reshape(len(K), -1)), c.dev_bf16(c.V.reshape(len(K), -1)), cu=all32)
    M = sum(q_lens)
    q = c.dev_bf16(c.rng.standard_normal((M, Hq * 64)) * 1.5)
    cu = None if set(q_lens) == {1} else i32(np.r_[0, np.cumsum(q_lens)], dev, torch)
    for value in (float("inf"), float("nan")):
        bad = q.clone()
        rows = [(m, 0) for m in range(0, M, 7)]
        for m, h in rows:
            bad[m, h * 64 + 5] = value
        a, la = sq.kv_attention(kv, c.pool, c.table, n32, q, cu=cu, lse=True)
        b, lb = sq.kv_attention(kv, c.pool, c.table, n32, bad, cu=cu, lse=True)
        other = torch.ones((M, Hq), dtype=torch.bool, device=dev)
        for m, h in rows:
            other[m, h] = False
        assert torch.equal(la[other], lb[other]), f"{value}: lse of {int((la[other] != lb[other]).sum())} other rows"
        assert torch.equal(a.view(M, Hq, 64)[other], b.view(M, Hq, 64)[other]), f"{value}: other rows"


def test_attention_window_beyond_int32(td):
    torch, dev = td
    kv = sq.KvLayout("mxfp4", 1, 64, 16)
    c = Cache(torch, dev, kv, [40], 3)
    q, n32 = torch.zeros((1, 64), device=dev).bfloat16(), i32([40], dev, torch)
    for window in (1 << 31, (1 << 32) + 5, -(1 << 32) + 5, -(1 << 31) - 1, -(1 << 33)):
        with pytest.raises(ValueError):
            sq.kv_attention(kv, c.pool, c.table, n32, q, window=window)
    for window in (-1, -(1 << 31)):
        with pytest.raises(sq.SvdqError):
            sq.kv_attention(kv, c.pool, c.table, n32, q, window=window)


@pytest.mark.parametrize("q_lens,Hq,H", [([8] * 90, 8, 1), ([0, 3, 24, 0, 8, 1, 40] * 11, 4, 1), ([1] * 130, 40, 1)])
@pytest.mark.parametrize("before", [4, 32, 100])
def test_attention_many_rows_in_front(td, q_lens, Hq, H, before):
    """Rows of no sequence that would be tiles, in front of more than 64 sequences."""
    torch, dev = td
    rng = np.random.default_rng(4)
    lens = [int(q + x) for q, x in zip(q_lens, rng.integers(0, 20, len(q_lens)))]
    kv = sq.KvLayout("mxfp4", H, 64, 16)
    c = Cache(torch, dev, kv, lens, 18)
    M = sum(q_lens)
    Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)))
    q = torch.cat([torch.zeros((before, Hq * 64), device=dev).bfloat16(), c.dev_bf16(Qv.reshape(M, -1))])
    out, lse = torch.full_like(q, 7.0), torch.full((len(q), Hq), 7.0, device=dev)
    sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), q, cu=i32(before + np.r_[0, np.cumsum(q_lens)], dev, torch),
                    out=out, lse=lse)
    check_attention(c, Qv, out[before:], lse[before:], q_lens, lens, Hq, 0.125, True, 0, "rows in front", "few")
    assert (out[:before] == 7.0).all() and (lse[:before] == 7.0).all()
