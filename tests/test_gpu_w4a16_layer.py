"""svdq_linear_w4a16 (a whole packed layer with 16-bit activations) against the float64 oracle.

Bound, from the arithmetic, per output: a term of the 4-bit product passes at most 20 fp32
roundings for each 128 of K it shares a sum with (four or eight MFMAs of at most 5, when one
wave took all of K) and 40 more (the group scale, the waves', the planes' and the bias' sums),
each 2^-24 of a partial sum that B bounds; x_hat is held to 2^-18 (bf16 output, two planes) or
2^-26 (float32, three).  The low-rank terms pass two such products.  GELU has a slope below
1.13 and is computed to 1e-6.  A bf16 output is off by half a step more, 2^-8 relative."""
import numpy as np
import pytest

import synth
import w4a4_quantized_linear_amd as sq
from oracle import formats as F
from oracle import w4a16 as W

from _gpu_helpers import bf16_to_np, dev_tensor, pack

pytestmark = pytest.mark.gpu
EPI = sq.EPI_LOWRANK | sq.EPI_BIAS
FMTS = ["mxfp4", "int4", "nvfp4"]

# (M, K, N, rank): single tokens, the last M that shares a pass and the first that does not (float32
# and bf16 output), blocks of 16 tokens and their ends, K of one superfragment and odd multiples,
# N of one tile, ends inside and at a padded 256 rows, every kind of rank
CASES = [(1, 512, 16, 0), (1, 1024, 1040, 16), (1, 4096, 256, 32), (2, 1536, 48, 8), (5, 2048, 272, 64),
         (6, 2560, 528, 40), (8, 512, 512, 128), (9, 1024, 144, 16), (16, 512, 64, 256), (17, 1536, 32, 24),
         (33, 2048, 784, 48), (3, 512, 16400, 32), (8, 4096, 64, 64), (2, 20480, 32, 16), (100, 1024, 112, 32), (300, 512, 16, 16),
         (40, 8192, 64, 32), (12, 6144, 16, 16), (25, 4096, 272, 64), (48, 3584, 80, 0)]


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sq.lib()
    assert sq.device_check(), "current device is not gfx950"
    return torch, torch.device("cuda:0")


def _draw(fmt, M, K, N, rank, seed):
    spec = synth.layer_spec("qkv", M=M, K=K, N=N, rank=rank, fmt=fmt, x_outliers=max(1, K // 100),
                            w_outliers=max(1, K // 100), lora_rank=0)
    return synth.draw_layer(spec, seed=seed)


def _oracle(L, fmt, rank, gelu=False):
    return W.layer_forward(L["X"], L["lam"], L["L1"] if rank else None, L["L2"] if rank else None, L["R"], L["b"], fmt,
                           gelu)


def _bound(o, K, f32, gelu):
    n = 2.0 ** -24 * (20 * (K // 128) + 40)
    planes = 2.0 ** -26 if f32 else 2.0 ** -18
    lim = (n + planes) * (o["B"] + 3 * o["B_lr"] + np.abs(o["pre"]))
    if gelu:
        lim = 1.13 * lim + 1e-6
    return lim + (0 if f32 else 2.0 ** -8 * (np.abs(o["Y"]) + lim))


def _check(y, o, K, f32, gelu, what):
    err, lim = np.abs(y - o["Y"]), _bound(o, K, f32, gelu)
    assert np.all(err <= lim), f"{what}: {int((err > lim).sum())} outputs beyond the bound, worst {np.max(err / lim):.2f}"


def _np(torch, t):
    return t.cpu().numpy().astype(np.float64) if t.dtype == torch.float32 else bf16_to_np(t)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", CASES, ids=[f"M{c[0]}-K{c[1]}-N{c[2]}-r{c[3]}" for c in CASES])
def test_matches_oracle(torch_dev, fmt, case):
    torch, dev = torch_dev
    M, K, N, rank = case
    L = _draw(fmt, M, K, N, rank, 900 + M)
    layer = sq.Layer(fmt, K, N, rank)
    w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
    for gelu in (False, True):
        o = _oracle(L, fmt, rank, gelu)
        for f32 in (True, False):
            epi = EPI | (sq.EPI_GELU if gelu else 0) | (sq.EPI_OUT_F32 if f32 else 0)
            y = _np(torch, sq.linear_w4a16(layer, w, X, epi))
            _check(y, o, K, f32, gelu, f"{fmt} {case} gelu={gelu} f32={f32}")
            if f32 and not gelu:      # no error shared by all outputs
                assert np.abs(y - o["Y"]).sum() <= 1e-5 * np.abs(o["Y"]).sum() + 1e-12


def test_flags(torch_dev):
    """Without the low-rank and bias flags those terms are absent; rank 0 ignores the flag."""
    torch, dev = torch_dev
    M, K, N, rank = 3, 1024, 256, 16
    L = _draw("mxfp4", M, K, N, rank, 31)
    layer = sq.Layer("mxfp4", K, N, rank)
    w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
    for epi, r, b in ((0, 0, None), (sq.EPI_LOWRANK, rank, None), (sq.EPI_BIAS, 0, L["b"])):
        o = W.layer_forward(L["X"], L["lam"], L["L1"] if r else None, L["L2"] if r else None, L["R"], b, "mxfp4")
        _check(_np(torch, sq.linear_w4a16(layer, w, X, epi | sq.EPI_OUT_F32)), o, K, True, False, f"epi {epi}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 5, 20])
def test_exact_integers(torch_dev, fmt, M):
    """Integer X and lambda 1, R integers of every code with an exact scale: all sums are whole
    numbers below 2^24, so the float32 output equals the oracle bit for bit."""
    torch, dev = torch_dev
    rng = np.random.default_rng(M)
    K, N = 1024, 48
    vals = np.arange(-7, 8) if fmt == "int4" else np.array([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6])
    R = rng.choice(vals, (N, K)).astype(np.float32)
    R[:, ::16] = 7 if fmt == "int4" else 6                 # every group's largest: scale 1 (NVFP4: 448 2^k / 2688 below)
    if fmt == "nvfp4":
        R *= 448.0                                         # tensor scale 1, group scales 448
    X = synth.bf16_bits_from_f32(rng.integers(-2, 3, (M, K)).astype(np.float32))
    L = dict(R=R, lam=np.ones(K, np.float32), L1=np.zeros((K, 0), np.uint16), L2=np.zeros((0, N), np.uint16),
             b=synth.bf16_bits_from_f32(rng.integers(-64, 65, N).astype(np.float32)), X=X)
    layer = sq.Layer(fmt, K, N, 0)
    o = W.layer_forward(X, L["lam"], None, None, R, L["b"], fmt)
    assert np.abs(o["B"]).max() < 2 ** 24 * (448 if fmt == "nvfp4" else 1)
    y = sq.linear_w4a16(layer, pack(layer, L, torch, dev), dev_tensor(X, torch, dev), EPI | sq.EPI_OUT_F32)
    np.testing.assert_array_equal(y.cpu().numpy().astype(np.float64), o["Y"])


def test_strides_and_rows_behind(torch_dev):
    """Strided X and Y: only the M x N outputs are written, a single row's stride is free."""
    torch, dev = torch_dev
    K, N, rank = 1024, 144, 16
    for M in (1, 7, 19):
        L = _draw("int4", M, K, N, rank, 41 + M)
        layer = sq.Layer("int4", K, N, rank)
        w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
        want = sq.linear_w4a16(layer, w, X, EPI)
        wide = torch.full((M + 2, K + 24), 0x7FC0, dtype=torch.int16, device=dev)      # NaN around X
        wide[:M, 8:8 + K] = X
        out = torch.full((M + 2, N + 16), 7.0, dtype=torch.bfloat16, device=dev)
        sq.linear_w4a16(layer, w, wide[:M, 8:8 + K], EPI, out=out[:M, 8:8 + N])
        assert torch.equal(out[:M, 8:8 + N].view(torch.int16), want.view(torch.int16))
        out[:M, 8:8 + N] = 7.0
        assert bool((out == 7.0).all())
    assert sq.linear_w4a16(layer, w, X[:0], EPI).shape == (0, N)
    # a row whose own stride means nothing
    one = X[:1].t().contiguous().t()
    assert torch.equal(sq.linear_w4a16(layer, w, one, EPI).view(torch.int16),
                       sq.linear_w4a16(layer, w, X[:1], EPI).view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [4, 18])
def test_non_finite_rows_stay_alone(torch_dev, fmt, M):
    torch, dev = torch_dev
    K, N, rank = 1024, 64, 16
    L = _draw(fmt, M, K, N, rank, 51)
    layer = sq.Layer(fmt, K, N, rank)
    w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
    for epi in (EPI, EPI | sq.EPI_OUT_F32):
        want = sq.linear_w4a16(layer, w, X, epi)
        for bits in (0x7FC0, 0x7F80, -128):                  # NaN, inf, -inf
            bad = X.clone()
            bad[1, 77] = bits
            y = sq.linear_w4a16(layer, w, bad, epi)
            keep = [m for m in range(M) if m != 1]
            assert torch.equal(y[keep], want[keep]) and not bool(torch.isfinite(y[1]).any())


def test_streams_graphs_and_repeats(torch_dev):
    """The same bits on another stream, on repeats and in replays of a captured graph, with
    eager calls between the replays."""
    torch, dev = torch_dev
    M, K, N, rank = 3, 2048, 512, 32
    L = _draw("mxfp4", M, K, N, rank, 61)
    layer = sq.Layer("mxfp4", K, N, rank)
    w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
    want = sq.linear_w4a16(layer, w, X, EPI)
    for r in (128, 32):                                  # with a workspace (its contents never matter) and without
        Lr = _draw("mxfp4", M, K, N, r, 61)
        lr = sq.Layer("mxfp4", K, N, r)
        wr = pack(lr, Lr, torch, dev)
        ws = torch.full((sq.w4a16_bytes(lr, M) or 256,), 0xFF, dtype=torch.uint8, device=dev)
        assert torch.equal(sq.linear_w4a16(lr, wr, X, EPI, workspace=ws), sq.linear_w4a16(lr, wr, X, EPI))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = sq.linear_w4a16(layer, w, X, EPI, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    sx = X.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sy = sq.linear_w4a16(layer, w, sx, EPI)
    for k in range(4):
        other = torch.roll(X, k, 0).contiguous()
        sx.copy_(other)
        g.replay()
        eager = sq.linear_w4a16(layer, w, other, EPI)
        torch.cuda.synchronize()
        assert torch.equal(sy, eager), f"replay {k}"


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
def test_largest_layer(torch_dev, fmt):
    """65536 x 65536 (codes of 2 GiB): its first and last rows against layers of those rows alone,
    whose groups of weights are the same.  64 features are not zero, so a sum has at most 80 roundings
    whatever its order, each 2^-24 of at most sum |w x| <= 64 x 5 x 5 (INT4: of (24 + |q|) s |x|
    twice, s <= 5 / 7, q <= 7, which is below 54 x 5 x 64)."""
    torch, dev = torch_dev
    K = N = 65536
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    R, one = torch.randn((N, K), generator=g, device=dev).clamp_(-5, 5), torch.ones(K, device=dev)
    X = torch.zeros((20, K), device=dev).bfloat16()
    at = torch.linspace(0, K - 1, 64, device=dev).long()
    X[:, at] = torch.randn((20, 64), generator=g, device=dev).clamp(-5, 5).bfloat16()
    big, rows = sq.Layer(fmt, K, N, 0), sq.Layer(fmt, K, 32, 0)
    w = sq.pack_weight(big, R, None, None, one, None)
    ends = [(slice(i, i + 32), sq.pack_weight(rows, R[i:i + 32].contiguous(), None, None, one, None))
            for i in (0, 32768, N - 32)]
    del R
    for M in (1, 20):
        y = sq.linear_w4a16(big, w, X[:M].contiguous(), sq.EPI_OUT_F32)
        for at, we in ends:
            z = sq.linear_w4a16(rows, we, X[:M].contiguous(), sq.EPI_OUT_F32)
            lim = 2 * 80 * 2.0 ** -24 * 64 * 5 * (54 if fmt == "int4" else 5)
            assert float((y[:, at] - z).abs().max()) <= lim and float(z.abs().max()) > 4


def test_refusals(torch_dev):
    torch, dev = torch_dev
    layer = sq.Layer("mxfp4", 1024, 64, 16)
    w = torch.zeros(sq.weight_bytes(layer), dtype=torch.uint8, device=dev)
    X = torch.zeros((4, 1024), dtype=torch.bfloat16, device=dev)
    for bad in (X.float(), X[:, :512], X.cpu(), X.t(), X[0], torch.zeros((4, 2048), dtype=X.dtype, device=dev)[:, ::2]):
        with pytest.raises(ValueError):
            sq.linear_w4a16(layer, w, bad)
    with pytest.raises(ValueError):
        sq.linear_w4a16(layer, w[:-256], X)
    for out in (torch.zeros((4, 64), device=dev), torch.zeros((3, 64), dtype=X.dtype, device=dev),
                torch.zeros((4, 64), dtype=X.dtype)):
        with pytest.raises(ValueError):
            sq.linear_w4a16(layer, w, X, out=out)
    many = torch.zeros((40, 1024), dtype=torch.bfloat16, device=dev)
    for x, kw, status in ((many, dict(workspace=w[:256]), 5), (X, dict(epi=64), 3),
                          (X, dict(out=torch.zeros((4, 68), dtype=X.dtype, device=dev)[:, :64]), 4)):
        with pytest.raises(sq.SvdqError) as e:
            sq.linear_w4a16(layer, w, x, **kw)
        assert e.value.status == status
