"""The 4-bit key-value cache on the GPU against oracle/kv.py: rows in (codes bit for bit), attention (each element
within a bound on float32's rounding and bf16's), pages and tokens that move."""
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


# ---- rows in and back ----

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page,H", [(64, 16, 3), (128, 64, 2), (128, 16, 1), (64, 1024, 1)])
def test_append_and_read(td, fmt, D, page, H):
    """K and V without norm or rotation: the oracle's codes for every element; only the rows' places change."""
    torch, dev = td
    kv = sq.KvLayout(fmt, H, D, page)
    lens = [1, 15, 16, 17, 0, 33, 100]
    c = Cache(torch, dev, kv, lens, 1)
    M = sum(lens)
    for f32 in (True, False):
        k, v = sq.kv_read(kv, c.pool, c.table, i32(lens, dev, torch), M, cu=i32(c.cu, dev, torch), f32=f32)
        kh, vh = c.kh.reshape(M, -1), c.vh.reshape(M, -1)
        if f32:
            assert np.array_equal(k.cpu().numpy(), kh.astype(np.float32)) and np.array_equal(v.cpu().numpy(), vh.astype(np.float32))
        else:
            assert np.array_equal(bits(k), c.bf16(kh)) and np.array_equal(bits(v), c.bf16(vh))
    # bytes written: one code byte per two features, and the scales, of M tokens
    per = sq.kv_page_bytes(kv) // page
    touched = torch.full_like(c.pool, 0)
    again = Cache.__new__(Cache)
    again.__dict__.update(c.__dict__)
    sq.kv_append(kv, touched, c.table, i32(lens, dev, torch), c.dev_bf16(c.K.reshape(M, -1)), c.dev_bf16(c.V.reshape(M, -1)),
                 cu=i32(c.cu, dev, torch))
    same = int((touched == c.pool).sum())
    assert same >= M * per and int(((touched != 0) & (touched != c.pool)).sum()) == 0
    assert int(((c.pool != 255) & (touched != c.pool)).sum()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_append_edge_values(td, fmt):
    """Zeros and signed zeros, subnormals, the largest magnitudes, ties, NaN and infinities."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 1, 128, 16)
    rng = np.random.default_rng(5)
    u = rng.integers(0, 1 << 16, (48, 128)).astype(np.uint16)              # any bf16, NaN and infinities among them
    u[0] = 0
    u[1] = 0x8000
    u[2] &= 0x807F                                                         # subnormals
    u[3] = (u[3] & 0x807F) | 0x7F00                                        # the largest
    u[4] = np.where(rng.random(128) < 0.5, 0x7F80, 0xFF80)                 # infinities
    u[5] = 0x7FC0                                                          # NaN
    u[6, 1:] = 0
    u[6, 0] = 0xFF81
    for i, e in enumerate(range(7, 30)):                                   # rows near one exponent each
        u[e] = (u[e] & 0x807F) | ((110 + i * 2) << 7)
    for e in range(30, 40):                                                # small whole numbers: ties
        v = torch.tensor(rng.integers(-12, 13, 128) * 0.25).bfloat16()
        u[e] = v.view(torch.int16).numpy().view(np.uint16)
    x = torch.from_numpy(u.view(np.int16)).to(dev)
    lens = i32([48], dev, torch)
    pool = torch.zeros((3, sq.kv_page_bytes(kv)), dtype=torch.uint8, device=dev)
    table, cu = i32([[2, 0, 1]], dev, torch), i32([0, 48], dev, torch)
    sq.kv_append(kv, pool, table, lens, x, x.flip(0).contiguous(), cu=cu)
    k, v = sq.kv_read(kv, pool, table, lens, 48, cu=cu, f32=True)
    val = bits(x.view(torch.bfloat16))
    want = Kv.hold(val, fmt).astype(np.float32)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want[::-1])


def _heads(rng, M, H, D):
    return Kv.F.to_bf16(rng.standard_normal((M, H, D)) * 3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,pairs,axes,halves,norm,far", [
    (128, 64, 1, True, True, False), (128, 64, 3, False, True, False), (64, 32, 2, True, False, False),
    (64, 16, 1, False, True, False), (128, 32, 4, True, True, True), (64, 24, 1, True, False, True), (64, 6, 1, False, False, True), (128, 0, 0, False, True, False)])
def test_append_norm_and_rotation(td, fmt, D, pairs, axes, halves, norm, far):
    """K's codes equal the oracle's; Q is within bf16's half step and fp32's rounding of a norm and a rotation."""
    torch, dev = td
    rng = np.random.default_rng(D + pairs + axes)
    H, Hq = 3, 5
    kv = sq.KvLayout(fmt, H, D, 16)
    q_lens, lens = [3, 1, 20, 0, 9], [10, 1, 20, 7, 300]
    M = sum(q_lens)
    Qx, Kx, Vx = _heads(rng, M, Hq, D), _heads(rng, M, H, D), _heads(rng, M, H, D)
    wq, wk = (Kv.F.to_bf16(1 + 0.2 * rng.standard_normal(D)) for _ in range(2))
    freq = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    axis = rng.integers(0, max(axes, 1), pairs)
    pos = rng.integers(-2000000 if far else 0, 2000000 if far else 5000, (axes, M)) if axes > 1 else None
    place = np.concatenate([n - q + np.arange(q) for q, n in zip(q_lens, lens)])
    c = Cache(torch, dev, kv, lens, 2)
    t = lambda x: c.dev_bf16(x.reshape(len(x), -1) if x.ndim > 1 else x)
    row = torch.cat([t(Qx), t(Kx), t(Vx)], 1)                              # parts of one projection's rows
    q, k, v = row[:, :Hq * D], row[:, Hq * D:(Hq + H) * D], row[:, (Hq + H) * D:]
    args = dict(cu=i32(np.r_[0, np.cumsum(q_lens)], dev, torch))
    if norm:
        args.update(norm_q=t(wq), norm_k=t(wk), eps=1e-5)
    if pairs:
        args.update(freq=torch.tensor(freq, device=dev), axis=i32(axis, dev, torch), halves=halves)
        if pos is not None:
            args.update(pos=i32(pos, dev, torch))
    n32 = i32(lens, dev, torch)
    out = sq.kv_append(kv, c.pool, c.table, n32, k, v, Q=q, **args)
    how = dict(freq=freq, axis=axis if pos is not None else None, pos=place[None] if pos is None else pos, halves=halves)
    kz = Kv.bf16_of(Kv.head_rows(Kx, wk if norm else None, 1e-5, **how))
    rk, rv = sq.kv_read(kv, c.pool, c.table, n32, M, cu=args["cu"], f32=True)
    assert np.array_equal(rk.cpu().numpy(), Kv.hold(kz, fmt).reshape(M, -1).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), Kv.hold(Vx, fmt).reshape(M, -1).astype(np.float32))
    qz = Kv.head_rows(Qx, wq if norm else None, 1e-5, **how)
    plain = np.abs(Kv.head_rows(Qx, wq if norm else None, 1e-5))
    # fp32: the mean of squares (D / 2 + 8 roundings), root, quotient and products, at 2^-24 each, of either feature
    lim = 2.0 ** -8 * np.abs(qz) + (D / 2 + 16) * 2.0 ** -24 * 2 * plain.max(-1, keepdims=True)
    err = np.abs(bits(out).reshape(qz.shape) - qz)
    assert (err <= lim).all(), np.max(err / lim)
    # in place, and without Q
    inplace = q.clone()
    assert sq.kv_append(kv, c.pool, c.table, n32, k, v, Q=inplace, q_out=inplace, **args) is inplace
    assert torch.equal(inplace, out)
    before = c.pool.clone()
    args.pop("norm_q", None)
    assert sq.kv_append(kv, c.pool, c.table, n32, k, v, **args) is None and torch.equal(before, c.pool)


def test_rows_without_a_place(td):
    """Rows before cu[0], behind cu[batch], of too short a length, behind the table, on pages outside the pool: the
    pool stays as it was; Q is written for a sequence's rows alone."""
    torch, dev = td
    kv = sq.KvLayout("int4", 2, 64, 16)
    pool = torch.full((4, sq.kv_page_bytes(kv)), 7, dtype=torch.uint8, device=dev)
    x = torch.randn((12, 128), device=dev).bfloat16()
    table = i32([[0, -1], [4, 1 << 30], [-5, 2]], dev, torch)
    lens, cu = i32([17, 32, 40], dev, torch), i32([1, 2, 5, 10], dev, torch)    # places 16; 29..31; 35..39
    q = torch.full((12, 64), 3.0, device=dev).bfloat16()
    out = torch.zeros_like(q)
    sq.kv_append(kv, pool, table, lens, x, x, cu=cu, Q=q, q_out=out)
    assert int((pool != 7).sum()) == 0
    assert torch.equal(out[1:10], q[1:10]) and int((out[0] != 0).sum()) == 0 and int((out[10:] != 0).sum()) == 0
    k, v = sq.kv_read(kv, pool, table, lens, 12, cu=cu)
    assert int((k[1:10] != 0).sum()) == 0 and int((v[1:10] != 0).sum()) == 0
    short = i32([-3, 1, 0], dev, torch)                                          # rows at places below 0
    sq.kv_append(kv, pool, i32([[0, 1], [2, 3], [1, 0]], dev, torch), short, x, x, cu=cu)
    assert int((pool[0] != 7).sum()) == 0 and int((pool[1] != 7).sum()) == 0 and int((pool[3] != 7).sum()) == 0
    k, _ = sq.kv_read(kv, pool, i32([[0, 1], [2, 3], [1, 0]], dev, torch), short, 12, cu=cu, f32=True)
    want = Kv.hold(bits(x[4]).reshape(2, 64), "int4").reshape(-1)
    assert np.array_equal(k[4].cpu().numpy(), want.astype(np.float32)) and int((k[2:4] != 0).sum()) == 0
    assert sq.kv_append(kv, pool, table[:0], lens[:0], x[:0], x[:0]) is None


# ---- attention ----

SHAPES = {
    # name: query rows, lengths, query heads, heads, page
    "one query": ([1] * 14, [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 127, 128, 129, 1000], 8, 2, 16),
    "own heads": ([1] * 5, [700, 3, 64, 65, 250], 3, 3, 32),
    "sixteen": ([1] * 3, [90, 33, 513], 32, 2, 64),
    "seventeen": ([1] * 3, [90, 33, 513], 17, 1, 16),
    "drafts": ([1, 3, 7, 0, 5, 4], [50, 3, 300, 9, 1025, 2], 8, 2, 16),
    "few rows many heads": ([2, 5], [400, 77], 40, 2, 128),
    "prompt": ([130, 70, 1, 257], [130, 300, 5, 600], 4, 2, 32),
    "prompt own heads": ([300], [1100], 2, 2, 64),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("table", ["own", "long"])
def test_attention(td, fmt, D, name, table):
    """Tables as long as the longest sequence, and long ones, whose calls are cut into ranges that are joined."""
    torch, dev = td
    q_lens, lens, Hq, H, page = SHAPES[name]
    kv = sq.KvLayout(fmt, H, D, page)
    c = Cache(torch, dev, kv, lens, len(name) + D, cols=4096 // page if table == "long" else None)
    M = sum(q_lens)
    Qv = c.bf16(c.rng.standard_normal((M, Hq, D)) * 1.5)
    q = c.dev_bf16(Qv.reshape(M, -1))
    cu = None if set(q_lens) == {1} else i32(np.r_[0, np.cumsum(q_lens)], dev, torch)
    few = M * (Hq // H) <= 32 * len(lens)
    precision = "nvfp4" if fmt == "nvfp4" else "few" if few else "many"
    for causal, window in ((True, 0), (False, 0), (True, 1), (True, 40), (False, 200)):
        what = f"{fmt} D{D} {name} causal {causal} window {window}"
        print(what, flush=True)
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), q, cu=cu, causal=causal, window=window, lse=True)
        check_attention(c, Qv, out, lse, q_lens, lens, Hq, D ** -0.5, causal, window, what, precision)
        again = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), q, cu=cu, causal=causal, window=window)
        assert torch.equal(again, out), f"{what}: other bits"


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_long(td, fmt):
    """One long sequence over many ranges, its join, and a batch beyond one scan's 256."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 1, 64, 64)
    short = [int(n) for n in np.random.default_rng(3).integers(0, 50, 600)]
    for lens, Hq, cols in (([70001], 2, None), ([3, 40000, 5], 1, None), (short, 2, None), (short, 2, 100), (short[:200], 2, 100), (short[:200] + [5000], 2, 100)):
        c = Cache(torch, dev, kv, lens, 9, cols=cols)
        Qv = c.bf16(c.rng.standard_normal((len(lens), Hq, 64)))
        for window in (0, 1500, 37777, 500):                           # the last is no longer split
            out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(len(lens), -1)),
                                       window=window, lse=True)
            check_attention(c, Qv, out, lse, [1] * len(lens), lens, Hq, 0.125, True, window, f"{fmt} {len(lens)} {window}",
                            "nvfp4" if fmt == "nvfp4" else "few")


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_many_sequences_of_rows(td, fmt):
    """More than 256 sequences of several rows (the scan's chunks), prompts among them, in both kinds of plan."""
    torch, dev = td
    rng = np.random.default_rng(8)
    for B, most, H, Hq, cols in ((300, 3, 1, 2, None), (300, 3, 1, 2, 300), (270, 90, 2, 4, None), (270, 90, 1, 4, 300)):
        q_lens = [int(x) for x in rng.integers(0, most + 1, B)]
        lens = [int(x + y) for x, y in zip(q_lens, rng.integers(0, 40, B))]
        kv = sq.KvLayout(fmt, H, 64, 16)
        c = Cache(torch, dev, kv, lens, B, cols=cols)
        M = sum(q_lens)
        Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)))
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(M, -1)),
                                   cu=i32(np.r_[0, np.cumsum(q_lens)], dev, torch), lse=True)
        few = M * (Hq // H) <= 32 * B
        check_attention(c, Qv, out, lse, q_lens, lens, Hq, 0.125, True, 0, f"{fmt} {B}",
                        "nvfp4" if fmt == "nvfp4" else "few" if few else "many")


PROMPTS = {
    # the same, of 128-row tiles: 128 rows a sequence on average, M x q_heads >= 384 x 128; the last sequence of "groups"
    # has more rows than tokens
    "groups": ([200, 1, 129, 0, 333, 140], [200, 700, 500, 9, 400, 100], 64, 8, 16),
    "own heads": ([900, 100, 600], [1000, 100, 601], 32, 32, 64),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name,D,masks", [("groups", 64, ((True, 2 ** 31 - 1), (True, 40))), ("groups", 128, ((True, 0), (False, 200))),
                                          ("own heads", 64, ((True, 0), (False, 200)))])
def test_attention_prompts(td, fmt, name, D, masks):
    torch, dev = td
    q_lens, lens, Hq, H, page = PROMPTS[name]
    M = sum(q_lens)
    assert M * Hq >= 384 * 128 and M * (Hq // H) >= 128 * len(lens)
    kv = sq.KvLayout(fmt, H, D, page)
    c = Cache(torch, dev, kv, lens, 5 + D)
    Qv = c.bf16(c.rng.standard_normal((M, Hq, D)) * 1.5)
    q, cu, n = c.dev_bf16(Qv.reshape(M, -1)), i32(np.r_[0, np.cumsum(q_lens)], dev, torch), i32(lens, dev, torch)
    for causal, window in masks:
        what = f"{fmt} D{D} {name} causal {causal} window {window}"
        print(what, flush=True)
        out, lse = sq.kv_attention(kv, c.pool, c.table, n, q, cu=cu, causal=causal, window=window, lse=True)
        check_attention(c, Qv, out, lse, q_lens, lens, Hq, D ** -0.5, causal, window, what,
                        "nvfp4" if fmt == "nvfp4" else "many")
        assert torch.equal(sq.kv_attention(kv, c.pool, c.table, n, q, cu=cu, causal=causal, window=window), out), what


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_drafts_of_a_large_batch(td, fmt):
    """Few rows of many sequences: 32-row tiles and P to 2^-16, however many there are; whole and split."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 8, 64, 16)
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(5, 60, 200)]
    q_lens = [4] * 200
    for cols in (None, 300):
        c = Cache(torch, dev, kv, lens, 6, cols=cols)
        Qv = c.bf16(c.rng.standard_normal((800, 64, 64)))
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(800, -1)),
                                   cu=i32(np.arange(201) * 4, dev, torch), lse=True)
        check_attention(c, Qv, out, lse, q_lens, lens, 64, 0.125, True, 0, f"{fmt} {cols}", "nvfp4" if fmt == "nvfp4" else "few")


@pytest.mark.parametrize("q_lens,Hq,H", [
    ([8] * 90, 8, 1), ([8] * 90, 16, 2), ([0, 0, 24, 0, 8, 1, 0, 40, 0] * 11, 4, 1), ([0] * 70 + [33] + [0] * 70, 8, 8), ([1] * 130, 40, 1),
    ([2] * 5000, 8, 1)])
def test_attention_tiles_of_many_sequences(td, q_lens, Hq, H):
    """Every tile of every sequence is done once: whole tiles, a row more, sequences without rows, rows of none."""
    torch, dev = td
    rng = np.random.default_rng(3)
    lens = [int(q + x) for q, x in zip(q_lens, rng.integers(0, 20, len(q_lens)))]
    kv = sq.KvLayout("mxfp4", H, 64, 16)
    c = Cache(torch, dev, kv, lens, 8)
    M, before, behind = sum(q_lens), 3, 70
    Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)))
    q = torch.cat([torch.zeros((before, Hq * 64), device=dev).bfloat16(), c.dev_bf16(Qv.reshape(M, -1)),
                   torch.zeros((behind, Hq * 64), device=dev).bfloat16()])
    out, lse = torch.full_like(q, 7.0), torch.full((len(q), Hq), 7.0, device=dev)
    sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), q, cu=i32(before + np.r_[0, np.cumsum(q_lens)], dev, torch),
                    out=out, lse=lse)
    check_attention(c, Qv, out[before:before + M], lse[before:before + M], q_lens, lens, Hq, 0.125, True, 0, "tiles", "few")
    for x in (out, lse):
        assert (x[:before] == 7.0).all() and (x[before + M:] == 7.0).all()


@pytest.mark.parametrize("cols", [None, 200])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_widest_windows(td, cols, causal):
    """A window of every size up to the largest int32, with more rows than tokens: it ends before the first place."""
    torch, dev = td
    kv = sq.KvLayout("mxfp4", 1, 64, 16)
    lens, q_lens = [0, 1, 5, 40, 2], [2, 4, 5, 3, 1]
    c = Cache(torch, dev, kv, lens, 2, cols=cols)
    M = sum(q_lens)
    for Hq in (1, 8):                                                  # 16 rows a tile, 32 rows
        Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)))
        for window in (2 ** 30, 2 ** 31 - 8, 2 ** 31 - 2, 2 ** 31 - 1):
            out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(M, -1)),
                                       cu=i32(np.r_[0, np.cumsum(q_lens)], dev, torch), causal=causal, window=window, lse=True)
            check_attention(c, Qv, out, lse, q_lens, lens, Hq, 0.125, causal, window, f"window {window}", "few")


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_scales_and_magnitudes(td, fmt):
    """Peaked and flat softmaxes, tiny and large K, V and Q; a rising running maximum; lengths beyond the table."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 1, 128, 32)
    for mag, scale in ((1.0, 5.0), (1.0, 1e-4), (2.0 ** -9, 2.0 ** 14), (64.0, 2.0 ** -14)):
        lens = [300, 77]
        c = Cache(torch, dev, kv, lens, 4, scale=mag)
        Qv = c.bf16(c.rng.standard_normal((2, 4, 128)) * mag)
        Qv[:, 1] *= 2.0 ** -60                                             # rows of very different size
        Qv[:, 2, 1:] *= 2.0 ** -20
        out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(2, -1)), scale=scale, lse=True)
        check_attention(c, Qv, out, lse, [1, 1], lens, 4, float(np.float32(scale)), True, 0, f"{fmt} {mag} {scale}",
                        "nvfp4" if fmt == "nvfp4" else "few")
    # scores that rise with the place, so that the maximum moves in every step
    lens = [600]
    c = Cache(torch, dev, kv, lens, 4, gain=False)
    K = np.zeros((600, 1, 128))
    K[:, 0, :] = np.linspace(-1, 1, 600)[:, None]
    c.K = c.bf16(K)
    sq.kv_append(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(c.K.reshape(600, -1)), c.dev_bf16(c.V.reshape(600, -1)),
                 cu=i32([0, 600], dev, torch))
    c.kh = Kv.hold(c.K, fmt)
    Qv = c.bf16(np.ones((1, 2, 128)) * [[[8.0], [-8.0]]])
    out, lse = sq.kv_attention(kv, c.pool, c.table, i32(lens, dev, torch), c.dev_bf16(Qv.reshape(1, -1)), lse=True)
    check_attention(c, Qv, out, lse, [1], lens, 2, 128 ** -0.5, True, 0, f"{fmt} rising", "nvfp4" if fmt == "nvfp4" else "few")
    # a length beyond the table: the tokens that are there
    out2, lse2 = sq.kv_attention(kv, c.pool, c.table, i32([c.cols * 32 + 50], dev, torch), c.dev_bf16(Qv.reshape(1, -1)), lse=True)
    full = sq.kv_attention(kv, c.pool, c.table, i32([c.cols * 32], dev, torch), c.dev_bf16(Qv.reshape(1, -1)), lse=True)
    if c.cols * 32 == 600:
        assert torch.equal(out2, full[0]) and torch.equal(lse2, full[1])


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_pages_that_are_not_there(td, fmt):
    """Pages of -1 and beyond the pool inside a sequence hold no token, whatever page 0 holds; a window whose earlier
    pages were given back; garbage on either side of the tokens that are seen."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 2, 64, 16)
    lens = [200, 90]
    c = Cache(torch, dev, kv, lens, 6)
    holes = c.tab.copy()
    holes[0, 2], holes[0, 7], holes[1, 0] = -1, c.pool.shape[0], -7
    Qv = c.bf16(c.rng.standard_normal((2, 4, 64)))
    q = c.dev_bf16(Qv.reshape(2, -1))
    out, lse = sq.kv_attention(kv, c.pool, i32(holes, dev, torch), i32(lens, dev, torch), q, lse=True)
    seen = [np.delete(np.arange(200), np.r_[32:48, 112:128]), np.arange(16, 90)]
    values = lambda b: tuple(t[seen[b]] for t in c.values(b))
    check_attention(c, Qv, out, lse, [1, 1], [len(s) for s in seen], 4, 0.125, True, 0, f"{fmt} holes",
                    "nvfp4" if fmt == "nvfp4" else "few", values=values)
    w = 50                                                             # sees 150 .. 199 and 40 .. 89
    gone = c.tab.copy()
    gone[0, :150 // 16], gone[1, :40 // 16] = c.free[0], c.free[1]     # pages whose bytes are all ones
    out, lse = sq.kv_attention(kv, c.pool, i32(gone, dev, torch), i32(lens, dev, torch), q, window=w, lse=True)
    check_attention(c, Qv, out, lse, [1, 1], lens, 4, 0.125, True, w, f"{fmt} window", "nvfp4" if fmt == "nvfp4" else "few")
    pool = c.pool.clone()                                              # a tile's tokens before the window as well
    small = sq.KvLayout(fmt, 2, 64, 16)
    n = i32([150 // 16 * 16 + 16], dev, torch)
    assert small == kv and int(n[0]) == 160
    k, v = sq.kv_read(kv, pool, c.table[:1], n, 160, cu=i32([0, 160], dev, torch), f32=True)
    fresh = torch.full_like(pool, 255)
    sq.kv_append(kv, fresh, c.table, i32(lens, dev, torch), c.dev_bf16(np.concatenate([c.K[150:200], c.K[240:290]]).reshape(100, -1)),
                 c.dev_bf16(np.concatenate([c.V[150:200], c.V[240:290]]).reshape(100, -1)), cu=i32([0, 50, 100], dev, torch))
    out2, lse2 = sq.kv_attention(kv, fresh, c.table, i32(lens, dev, torch), q, window=w, lse=True)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_strides_and_rows_outside(td, fmt):
    """Rows of a wider matrix, an output with a stride, rows in front of and behind the sequences left alone, a
    workspace of exactly the stated size between guards, NaN in one row."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 2, 64, 32)
    q_lens, lens, Hq = [2, 1, 40], [70, 33, 900], 4
    for q_lens, cols in (([2, 1, 4], None), ([2, 1, 4], 200), ([2, 1, 130], None)):
        c = Cache(torch, dev, kv, lens, 7, cols=cols)
        M = sum(q_lens) + 5
        Qv = c.bf16(c.rng.standard_normal((M, Hq, 64)))
        wide = torch.full((M, Hq * 64 + 24), float("nan"), device=dev).bfloat16()
        q = wide[:, 8:8 + Hq * 64]
        q.copy_(c.dev_bf16(Qv.reshape(M, -1)))
        cu = i32(2 + np.r_[0, np.cumsum(q_lens)], dev, torch)
        n = sq.kv_attention_bytes(kv, c.cols, 3, M, Hq)
        space = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=dev)
        out = torch.full((M, Hq * 64 + 16), 5.0, device=dev).bfloat16()
        y = out[:, 8:8 + Hq * 64]
        ws = space[256:256 + n] if n else None
        lse = torch.full((M, Hq), 9.0, device=dev)
        n32 = i32(lens, dev, torch)
        got = sq.kv_attention(kv, c.pool, c.table, n32, q, cu=cu, out=y, lse=lse, workspace=ws)
        assert got[0] is y and int((space[:256] != 0xA5).sum()) == 0 and int((space[256 + n:] != 0xA5).sum()) == 0
        few = M * 2 <= 32 * 3
        check_attention(c, Qv[2:-3], y[2:-3], lse[2:-3], q_lens, lens, Hq, 0.125, True, 0, f"{fmt} strides",
                        "nvfp4" if fmt == "nvfp4" else "few" if few else "many")
        assert bool((out[:, :8] == 5).all()) and bool((out[:, 8 + Hq * 64:] == 5).all())
        for edge in (out[:2], out[-3:]):
            assert bool((edge == 5).all())
        assert bool((lse[:2] == 9).all()) and bool((lse[-3:] == 9).all())
        # the same bits whatever the workspace held, and NaN in one row of one head stays there
        kept = y.clone()
        bad = q.clone()
        bad[3, 64 + 5] = float("nan")
        other = sq.kv_attention(kv, c.pool, c.table, n32, bad.contiguous(), cu=cu)
        diff = (other[2:-3] != kept[2:-3]).view(-1, Hq, 64)
        assert bool(diff[1, 1].all()) and int(diff.sum()) == 64


def test_attention_refusals(td):
    torch, dev = td
    kv = sq.KvLayout("mxfp4", 2, 64, 16)
    c = Cache(torch, dev, kv, [20, 30], 3, cols=100)
    n32, q = i32([20, 30], dev, torch), torch.zeros((2, 256), device=dev).bfloat16()
    ok = lambda **kw: sq.kv_attention(kv, c.pool, c.table, n32, **{"Q": q, **kw})
    ok()
    for kw in (dict(Q=q[:, :100]), dict(Q=q.float()), dict(Q=q.cpu()), dict(Q=q[:1]), dict(out=q[:, :128]), dict(out=q.float()),
               dict(lse=torch.zeros((2, 3), device=dev)), dict(workspace=q), dict(cu=n32), dict(Q=q.t().contiguous().t()),
               dict(workspace=torch.zeros(4, dtype=torch.uint8)), dict(window=1 << 32)):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(scale=0.0), dict(window=-1), dict(Q=q[:, :192]), dict(workspace=torch.zeros(256, dtype=torch.uint8, device=dev))):
        with pytest.raises(sq.SvdqError):
            ok(**kw)
    for bad in (dict(pool=c.pool[:, :-1]), dict(table=c.table.long()), dict(lens=n32.long()), dict(table=c.table[:1]),
                dict(pool=c.pool.view(torch.int8)), dict(lens=n32[::2])):
        a = dict(pool=c.pool, table=c.table, lens=n32)
        a.update(bad)
        with pytest.raises(ValueError):
            sq.kv_attention(kv, a["pool"], a["table"], a["lens"], q)
        with pytest.raises(ValueError):
            sq.kv_append(kv, a["pool"], a["table"], a["lens"], q[:, :128], q[:, 128:])
        with pytest.raises(ValueError):
            sq.kv_read(kv, a["pool"], a["table"], a["lens"], 2)
    for kw in (dict(Q=q, q_out=q[:, :128]), dict(q_out=q), dict(norm_k=q[0, :32]), dict(axis=n32), dict(pos=n32),
               dict(freq=q[0, :4]), dict(freq=torch.zeros(4, device=dev), pos=n32[None]), dict(Q=q[:1])):
        with pytest.raises(ValueError):
            if kw.get("pos") is not None and kw["pos"].dim() == 2:
                kw["pos"] = kw["pos"][:, :1]
            sq.kv_append(kv, c.pool, c.table, n32, q[:, :128], q[:, 128:], **kw)
    with pytest.raises(sq.SvdqError):
        sq.kv_append(kv, c.pool, c.table, n32, q[:, :128], q[:, 128:], freq=torch.zeros(3, device=dev))
    with pytest.raises(sq.SvdqError):
        sq.kv_copy(kv, c.pool, [0, 1], [2, 0])
    with pytest.raises(ValueError):
        sq.kv_copy(kv, c.pool, [0, 1], [2])
    for bad in ([1 << 32], [0.5], None, torch.zeros(1, device=dev)):
        with pytest.raises(ValueError):
            sq.kv_copy(kv, c.pool, bad, [2])
    with pytest.raises(ValueError):
        sq.kv_compact(kv, c.pool, c.table, n32, n32)
