"""The 4-bit key-value cache at its edges: Q heads of any magnitude, rows beside an infinity, windows beyond int32, rows in front
of the sequences, lengths behind the table, tiles of 32 rows held to their own precision, compaction by parts of the heads."""
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


def _precision(fmt, q_lens, Hq, H):
    """How P is rounded, as the header has it: once, to bf16, in prompts of many and long rows."""
    M = sum(q_lens)
    long = M * Hq >= 384 * 128 and M * (Hq // H) >= 128 * len(q_lens)
    return "nvfp4" if fmt == "nvfp4" else "many" if long else "few"


BEHIND = {
    # query rows, lengths, query heads, heads, columns of 64 tokens
    "16 rows": ([1, 1, 1], [1024 + 50, 700, 1024], 4, 1, 16),
    "16 rows, ranges": ([1, 1, 1], [2048 + 50, 700, 2048], 4, 1, 32),
    "32 rows": ([6, 9, 30], [512 + 3, 200, 512 + 40], 4, 1, 8),
    "32 rows, ranges": ([6, 9, 30], [2048 + 3, 700, 2048 + 40], 4, 1, 32),
    "128 rows": ([580, 190], [512 + 200, 512 + 189], 64, 8, 8),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", list(BEHIND))
def test_attention_lengths_behind_the_table(td, fmt, name):
    """Tokens behind the table are not there; the rows' own places, masks and windows are as the lengths say."""
    torch, dev = td
    q_lens, lens, Hq, H, cols = BEHIND[name]
    kv = sq.KvLayout(fmt, H, 64, 64)
    c = Cache(torch, dev, kv, [min(n, cols * 64) for n in lens], 19, cols=cols)
    M = sum(q_lens)
    Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)) * 1.5)
    q, cu = c.dev_bf16(Qv.reshape(M, -1)), None if set(q_lens) == {1} else i32(np.r_[0, np.cumsum(q_lens)], dev, torch)
    for causal, window in ((True, 0), (False, 0), (True, 45), (False, 45)):
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), q, cu=cu, causal=causal, window=window, lse=True)
        check_attention(c, Qv, out, lse, q_lens, lens, Hq, 0.125, causal, window, f"{fmt} {name} {causal} {window}",
                        _precision(fmt, q_lens, Hq, H))


ROWS32 = {
    "many heads": ([2, 5], [400, 77], 40, 2, 128),
    "prompt": ([130, 70, 1, 257], [130, 300, 5, 600], 4, 2, 32),
    "own heads": ([300], [1100], 2, 2, 64),
    "few tiles": ([764], [800], 64, 8, 64),                       # 4 rows of 64 heads short of the 128-row form
    "short": ([15] * 52, [60] * 52, 64, 8, 16),                   # rows enough, but 120 a sequence
}


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("name,D,table", [(n, D, t) for n in list(ROWS32)[:3] for D in (64, 128) for t in ("own", "long")] +
                         [(n, 64, "own") for n in list(ROWS32)[3:]])
def test_attention_32_rows_keep_two_planes(td, fmt, name, D, table):
    """Tiles of 32 rows round P to 2^-16 of itself, whatever a sequence's rows."""
    torch, dev = td
    q_lens, lens, Hq, H, page = ROWS32[name]
    assert _precision(fmt, q_lens, Hq, H) == "few" and sum(q_lens) * (Hq // H) > 16 * len(q_lens)
    kv = sq.KvLayout(fmt, H, D, page)
    c = Cache(torch, dev, kv, lens, 20 + D, cols=4096 // page if table == "long" else None)
    M = sum(q_lens)
    Qv = c.bf16(c.rng.standard_normal((M, Hq, D)) * 1.5)
    for causal, window in ((True, 0), (True, 40)):
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(M, -1)),
                                   cu=i32(np.r_[0, np.cumsum(q_lens)], dev, torch), causal=causal, window=window, lse=True)
        check_attention(c, Qv, out, lse, q_lens, lens, Hq, D ** -0.5, causal, window, f"{fmt} {name} {window}", "few")


@pytest.mark.parametrize("fmt,B,L,most,planes", [("mxfp4", 1, 6000, 5000, 24), ("int4", 2, 7000, 6000, 12), ("nvfp4", 1, 6000, 5000, 24),
                                                 ("mxfp4", 1, 24000, 20000, 23)])
def test_compact_by_parts_of_the_heads(td, fmt, B, L, most, planes):
    """Long lists in place whose workspace holds a part of the heads and layers at a time, the last part shorter: every
    layer has the tokens that the same list gives in other pages; nothing else changes, also beside the workspace."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 8, 128, 64)
    per, rng = sq.kv_page_bytes(kv), np.random.default_rng(most)
    cols, cols_to = -(-L // 64), -(-most // 64)
    pages = B * (cols + cols_to) + 2
    g = torch.Generator(device=dev)
    g.manual_seed(L)
    pool = torch.randint(256, (planes, pages, per), dtype=torch.uint8, generator=g, device=dev)
    order = rng.permutation(pages)
    table, to = i32(order[:B * cols].reshape(B, cols), dev, torch), i32(order[B * cols:B * (cols + cols_to)].reshape(B, cols_to), dev, torch)
    counts = [most - 37 * b for b in range(B)]
    keep = np.zeros((B, most), int)
    for b, n in enumerate(counts):
        keep[b, :n] = np.sort(rng.choice(L, n, replace=False))
    args = (i32(keep, dev, torch), i32(counts, dev, torch))
    n = sq.kv_compact_bytes(kv, planes, B, most)
    every = B * planes * 8 * (most // 16) * 16 * (per // (8 * 64))           # bytes of the list's tokens in all
    assert 0 < n < every
    space = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=dev)
    before = pool.clone()
    sq.kv_compact(kv, pool, table, *args, workspace=space[256:256 + n])
    assert int((space[:256] != 0xA5).sum()) == 0 and int((space[256 + n:] != 0xA5).sum()) == 0
    want = before.clone()
    sq.kv_compact(kv, want, table, *args, to=to)
    cu, M = i32(np.r_[0, np.cumsum(counts)], dev, torch), sum(counts)
    for layer in range(planes):
        got = sq.kv_read(kv, pool[layer], table, args[1], M, cu=cu, f32=True)
        ref = sq.kv_read(kv, want[layer], to, args[1], M, cu=cu, f32=True)
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), layer
    used = torch.zeros(pages, dtype=torch.bool, device=dev)
    for b, m in enumerate(counts):
        used[table[b, :-(-m // 64)].long()] = True
    assert torch.equal(pool[:, ~used], before[:, ~used])
    behind = [torch.arange(m, -(-m // 64) * 64) for m in counts]             # places behind the last kept token
    for b, places in enumerate(behind):
        if len(places):
            end = i32([int(places[-1]) + 1], dev, torch)
            rows = i32([0, len(places)], dev, torch)
            for layer in (0, planes - 1):
                x, y = (sq.kv_read(kv, p[layer], table[b:b + 1], end, len(places), cu=rows, f32=True) for p in (pool, before))
                assert all(torch.equal(s.view(torch.int32), t.view(torch.int32)) for s, t in zip(x, y))
