"""Corners of the few-token entry points on the GPU: the same bits from the same call where experts'
blocks take different forms, equal and missing scores, the smallest magnitudes, precision that does
not hang on the number of tokens."""
import numpy as np
import pytest

import synth
import w4a4_quantized_linear_amd as sq
from oracle import formats as F
from oracle import moe as Mo
from oracle import quant as Q
from oracle import w4a16 as W

from _gpu_helpers import dev_tensor, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sq.lib()
    assert sq.device_check(), "current device is not gfx950"
    return torch, torch.device("cuda:0")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,k", [(33, 2), (70, 1), (200, 2), (900, 2), (1100, 2)])
def test_nvfp4_experts_same_bits(torch_dev, M, k, f32):
    """More than 64 pairs of NVFP4 experts at widths where a full block of pairs passes through the LDS
    in parts and a shorter one whole (in fp16): repeats and replays of a graph equal the first call."""
    torch, dev = torch_dev
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    E, H, Fh, N = 5, 2560, 4096, 64
    gu, dn = sq.Layer("nvfp4", H, 2 * Fh, 0), sq.Layer("nvfp4", Fh, N, 0)
    pg, pd = (sq.pack_experts(l, torch.randn((E, l.N, l.K), generator=g, device=dev) * l.K ** -0.5) for l in (gu, dn))
    # magnitudes over 32 octaves: some lie below what fp16 holds beside the row's largest
    X = torch.randn((M, H), generator=g, device=dev) * torch.exp2(-32 * torch.rand((M, H), generator=g, device=dev))
    X, wt = X.bfloat16(), torch.rand((M, k), generator=g, device=dev)
    ids = torch.rand((M, E), generator=g, device=dev).topk(k, 1)[1].int()

    def call():
        return sq.moe(gu, pg, dn, pd, X, ids, wt, sq.EPI_OUT_F32 if f32 else 0)

    want = call()
    assert bool(torch.isfinite(want).all()) and bool((want != 0).any())
    for i in range(40):
        assert torch.equal(call(), want), f"repeat {i}"
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = call()
    for i in range(10):
        graph.replay()
        other = call()
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(other, want), f"replay {i}"


def _bf16(torch, dev, rows):
    """Rows of a few leading features, the others zero, 8 wide."""
    t = torch.zeros((len(rows), 8), dtype=torch.float32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = torch.tensor(r)
    return t.bfloat16().to(dev)


@pytest.mark.parametrize("M,E", [(1, 4), (1, 400), (300, 4), (300, 130)])
def test_route_equal_scores_of_other_logits(torch_dev, M, E):
    """The choice is by score (1 for the sigmoid of 40 and of 50, 0 for exp(-800) and exp(-900)), the
    lower index first, with a bias of zeros as without one; one kernel (few tokens) and two."""
    torch, dev = torch_dev
    X = _bf16(torch, dev, [[1.0]] * M)
    for sigmoid, logits, want in ((True, [1.0, 40.0, 50.0, 45.0], [1, 2, 3, 0]),
                                  (False, [-800.0, 0.0, -900.0, -700.0], [1, 3, 0, 2])):
        router = _bf16(torch, dev, [[-1000.0]] * (E - 4) + [[l] for l in logits])
        if E > 4 and not sigmoid:
            want = [E - 4 + 1, E - 4 + 3, 0, 1]              # every other score is 0: the lowest indices
        elif E > 4:
            want = [E - 4 + i for i in want]
        for bias in (None, torch.zeros(E, device=dev)):
            ids, w = sq.moe_route(X, router, 4, bias=bias, sigmoid=sigmoid, renorm=False)
            assert ids.tolist() == [want] * M
            assert w[:, :2].tolist() == [[1.0, 1.0 if sigmoid else 0.0]] * M


@pytest.mark.parametrize("M,E", [(1, 5), (1, 300), (300, 5), (300, 130)])
def test_route_nan_behind_minus_infinity(torch_dev, M, E):
    """An expert whose score is NaN stands behind one that a bias of -infinity masks."""
    torch, dev = torch_dev
    X = _bf16(torch, dev, [[1.0]] * M)
    nan, inf = float("nan"), float("inf")
    router = _bf16(torch, dev, [[nan]] * (E - 5) + [[0.0], [nan], [1.0], [1.0], [nan]])
    bias = torch.zeros(E, device=dev)
    bias[E - 5 + 2] = -inf
    want = [E - 5 + i for i in (3, 0, 2)] + ([1, 4] if E == 5 else [0, 1])
    ids, w = sq.moe_route(X, router, 5, bias=bias, sigmoid=True, renorm=False)
    assert ids.tolist() == [want] * M
    assert bool(torch.isfinite(w[:, :3]).all()) and bool(torch.isnan(w[:, 3:]).all())


def _bits(a):
    return synth.bf16_bits_from_f32(np.asarray(a, np.float32))


def _values(R, fmt):
    """Experts' dequantized weights and their magnitudes as they enter the kernels' sums."""
    w, mag = np.empty(R.shape), np.empty(R.shape)
    for e in range(len(R)):
        gs = Q.nvfp4_global_scale(R[e]) if fmt == "nvfp4" else np.float32(1.0)
        c, s = Q.quantize(R[e], fmt, gs)
        w[e] = Q.dequantize(c, s, fmt, gs)
        mag[e] = np.abs(w[e])
        if fmt == "int4":
            mag[e] = (np.abs(24 + c.astype(np.float64)) + 24) * np.repeat(F.fp16_value(s), 64, axis=1)
    return w, mag


def _sum_eps(K):
    """Relative rounding of a product's sums: 5 roundings an MFMA, four MFMAs a 128 of K, and 40 more."""
    return 2.0 ** -24 * (20 * (K // 128) + 40)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
@pytest.mark.parametrize("M,k", [(1, 1), (9, 2), (70, 1)])
@pytest.mark.parametrize("up", [9, 0])
def test_experts_smallest_rows(torch_dev, fmt, M, k, up):
    """Tokens of subnormal features, which gate biases and large weights (2^up of gate/up, 2^9 of down)
    keep visible; with up = 0 h is subnormal too.  The experts' bound, 8 roundings of 2^-149, a
    subnormal's, for each element of u and h, and 2^-134 for each of h: its bf16 planes' last place is
    2^-133 however many there are, and the last plane rounds to the nearest."""
    torch, dev = torch_dev
    E, H, Fh, N = 3, 512, 512, 48
    rng = np.random.default_rng(M + up)
    Rg = (rng.standard_normal((E, 2 * Fh, H)) / np.sqrt(H) * 2.0 ** up).astype(np.float32)
    Rd = (rng.standard_normal((E, N, Fh)) / np.sqrt(Fh) * 2.0 ** 9).astype(np.float32)
    bg, bd = np.zeros((E, 2 * Fh), np.float32), np.zeros((E, N), np.float32)
    bg[:, :Fh] = 4.0
    gu, dn = sq.Layer(fmt, H, 2 * Fh, 0), sq.Layer(fmt, Fh, N, 0)
    pg, pd = (sq.pack_experts(l, dev_tensor(R, torch, dev), dev_tensor(_bits(b), torch, dev))
              for l, R, b in ((gu, Rg, bg), (dn, Rd, bd)))
    # the largest are below 2^-126; multiples of 2^-133, bf16's last place there
    X = rng.integers(-100, 101, (M, H)) * 2.0 ** -133
    X[:, 7] = 2.0 ** -127
    ids = np.argsort(rng.random((M, E)), axis=1)[:, :k].astype(np.int32)
    wt = rng.random((M, k)).astype(np.float32)
    (wg, mg), (wd, md) = _values(Rg, fmt), _values(Rd, fmt)
    o, lim = Mo.experts(_bits(X), ids, wt, wg, bg, wd, bd, False, (mg, md), (_sum_eps(H), _sum_eps(Fh) + 2.0 ** -26))
    least = (8 * 2.0 ** -149 * 4.0 + 2.0 ** -134) * np.abs(wd).sum(axis=2).max() * k
    lim = lim * (1 + 2.0 ** -20) + 2.0 ** -24 * (k + 1) * (np.abs(o) + lim) + least
    y = sq.moe(gu, pg, dn, pd, dev_tensor(_bits(X), torch, dev), dev_tensor(ids, torch, dev), dev_tensor(wt, torch, dev),
               sq.EPI_BIAS | sq.EPI_OUT_F32).cpu().numpy().astype(np.float64)
    assert np.abs(o).max() > 2.0 ** -126 and np.all(np.abs(o) + lim > 0)
    assert np.median(lim) < 0.5 * np.median(np.abs(o))                # zeros would be beyond the bound
    assert np.all(np.abs(y - o) <= lim), f"worst {np.max(np.abs(y - o) / lim):.2f}"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,rank", [(1, 2), (5, 64), (8, 2), (8, 100), (9, 2), (40, 64)])
def test_down_projection_keeps_its_bits(torch_dev, M, rank, f32):
    """D = (1 + 2^-9 + 2^-20, 2^-9) exactly, and Y = D0 - D1 - 1 = 2^-20: every sum is exact in fp32, and
    what is left needs more of D than two bf16 parts hold.  For few tokens, more, and either output."""
    torch, dev = torch_dev
    K, N = 512, 48
    X, L1, L2 = np.zeros((M, K)), np.zeros((K, rank)), np.zeros((rank, N))
    X[:, :3] = 1.0, 2.0 ** -9, 2.0 ** -20
    L1[:3, 0], L1[1, 1] = 1.0, 1.0
    L2[0], L2[1] = 1.0, -1.0
    layer = sq.Layer("mxfp4", K, N, rank)
    L1, L2, b = (dev_tensor(_bits(a), torch, dev) for a in (L1, L2, np.full(N, -1.0)))
    w = sq.pack_weight(layer, torch.zeros((N, K), device=dev), L1, L2, torch.ones(K, device=dev), b)
    y = sq.linear_w4a16(layer, w, dev_tensor(_bits(X), torch, dev),
                        sq.EPI_LOWRANK | sq.EPI_BIAS | (sq.EPI_OUT_F32 if f32 else 0))
    assert bool((y == 2.0 ** -20).all())


@pytest.mark.parametrize("M", [1, 300])
def test_route_infinite_features(torch_dev, M):
    """Softmax scores are NaN, sigmoid scores 1, 0 and NaN (infinity times a router weight of 0)."""
    torch, dev = torch_dev
    X, router = _bf16(torch, dev, [[float("inf")]] * M), _bf16(torch, dev, [[-1.0], [0.0], [2.0], [-2.0], [1.0]])
    ids, w = sq.moe_route(X, router, 5, sigmoid=True, renorm=False)
    assert ids.tolist() == [[2, 4, 0, 3, 1]] * M
    assert w[:, :4].tolist() == [[1.0, 1.0, 0.0, 0.0]] * M and bool(torch.isnan(w[:, 4]).all())
    ids, w = sq.moe_route(X, router, 5)
    assert ids.tolist() == [[0, 1, 2, 3, 4]] * M and bool(torch.isnan(w).all())


@pytest.mark.parametrize("fg,fd", [("mxfp4", "int4"), ("int4", "nvfp4"), ("nvfp4", "mxfp4")])
def test_experts_in_parts_within_the_bound(torch_dev, fg, fd):
    """Wide experts of 37 and 39 pairs, whose full blocks pass through the LDS in parts and whose last ones
    whole, against the oracle's bound for each element (76 pairs: 38 tokens, one with the same expert twice)."""
    torch, dev = torch_dev
    E, H, Fh, N, M, k = 2, 2560, 2560, 48, 38, 2
    rng = np.random.default_rng(17)
    Rg = (rng.standard_normal((E, 2 * Fh, H)) / np.sqrt(H)).astype(np.float32)
    Rd = (rng.standard_normal((E, N, Fh)) / np.sqrt(Fh)).astype(np.float32)
    bg, bd = _bits(rng.standard_normal((E, 2 * Fh)) * 0.1), _bits(rng.standard_normal((E, N)) * 0.1)
    gu, dn = sq.Layer(fg, H, 2 * Fh, 0), sq.Layer(fd, Fh, N, 0)
    pg, pd = (sq.pack_experts(l, dev_tensor(R, torch, dev), dev_tensor(b, torch, dev)) for l, R, b in ((gu, Rg, bg), (dn, Rd, bd)))
    X = _bits(rng.standard_normal((M, H)))
    ids = np.array([[0, 1]] * (M - 1) + [[1, 1]], np.int32)
    wt = rng.random((M, k)).astype(np.float32)
    (wg, mg), (wd, md) = _values(Rg, fg), _values(Rd, fd)
    for f32 in (True, False):
        o, lim = Mo.experts(X, ids, wt, wg, F.bf16_value(bg), wd, F.bf16_value(bd), False, (mg, md),
                            (_sum_eps(H), _sum_eps(Fh) + (2.0 ** -26 if f32 else 2.0 ** -18)))
        lim = lim * (1 + 2.0 ** -20) + 2.0 ** -24 * (k + 1) * (np.abs(o) + lim)
        if not f32:
            lim = lim + 2.0 ** -8 * (np.abs(o) + lim)
        y = sq.moe(gu, pg, dn, pd, dev_tensor(X, torch, dev), dev_tensor(ids, torch, dev), dev_tensor(wt, torch, dev),
                   sq.EPI_BIAS | (sq.EPI_OUT_F32 if f32 else 0)).float().cpu().numpy().astype(np.float64)
        err = np.abs(y - o)
        assert np.all(err <= lim), f"f32={f32}: worst {np.max(err / lim):.2f}"
        if f32:                                              # no error shared by all outputs
            assert err.sum() <= 1e-5 * np.abs(o).sum()


@pytest.mark.parametrize("M,K,E,k", [(3, 2560, 64, 4), (3, 2568, 64, 4), (2, 4096, 8, 2), (2, 4104, 8, 2), (2, 1280, 128, 9),
                                     (2, 1288, 128, 9), (256, 512, 160, 3), (257, 512, 160, 3), (1, 8192, 4, 4)])
def test_route_on_both_sides_of_its_forms(torch_dev, M, K, E, k):
    torch, dev = torch_dev
    rng = np.random.default_rng(K + E)
    X, Wr = _bits(rng.standard_normal((M, K))), _bits(rng.standard_normal((E, K)) * 2 / np.sqrt(K))
    ids, w = sq.moe_route(dev_tensor(X, torch, dev), dev_tensor(Wr, torch, dev), k)
    want, ww = Mo.route(X, Wr, k)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2.0 ** -23)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
@pytest.mark.parametrize("M,k,E", [(5, 3, 7), (50, 2, 4), (100, 2, 8), (112, 2, 8)])
def test_experts_down_forms(torch_dev, fmt, M, k, E):
    """The down product with h in LDS, with h too large for it, and either side of where pairs' products go
    through memory (at 200 pairs for one output only): within the oracle's bound, with a workspace of just
    the stated bytes inside a larger buffer that stays as it was."""
    torch, dev = torch_dev
    H, Fh, N = 512, 512, 80
    rng = np.random.default_rng(M)
    Rg = (rng.standard_normal((E, 2 * Fh, H)) / np.sqrt(H)).astype(np.float32)
    Rd = (rng.standard_normal((E, N, Fh)) / np.sqrt(Fh)).astype(np.float32)
    gu, dn = sq.Layer(fmt, H, 2 * Fh, 0), sq.Layer(fmt, Fh, N, 0)
    pg, pd = (sq.pack_experts(l, dev_tensor(R, torch, dev)) for l, R in ((gu, Rg), (dn, Rd)))
    X = _bits(rng.standard_normal((M, H)))
    ids = np.argsort(rng.random((M, E)), axis=1)[:, :k].astype(np.int32)
    wt = rng.random((M, k)).astype(np.float32)
    (wg, mg), (wd, md) = _values(Rg, fmt), _values(Rd, fmt)
    need = sq.moe_bytes(gu, dn, M, k)
    for f32 in (True, False):
        o, lim = Mo.experts(X, ids, wt, wg, None, wd, None, False, (mg, md),
                            (_sum_eps(H), _sum_eps(Fh) + (2.0 ** -26 if f32 else 2.0 ** -18)))
        lim = lim * (1 + 2.0 ** -20) + 2.0 ** -24 * (k + 1) * (np.abs(o) + lim)
        if not f32:
            lim = lim + 2.0 ** -8 * (np.abs(o) + lim)
        around = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=dev)
        y = sq.moe(gu, pg, dn, pd, dev_tensor(X, torch, dev), dev_tensor(ids, torch, dev), dev_tensor(wt, torch, dev),
                   sq.EPI_OUT_F32 if f32 else 0, workspace=around[4096:4096 + need])
        err = np.abs(y.float().cpu().numpy().astype(np.float64) - o)
        assert np.all(err <= lim), f"f32={f32}: worst {np.max(err / lim):.2f}"
        assert bool((around[:4096] == 0xA5).all()) and bool((around[4096 + need:] == 0xA5).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
@pytest.mark.parametrize("M,K,N,rank", [(1, 8192, 48, 32), (2, 8704, 48, 32), (1, 4096, 4112, 64), (3, 4608, 272, 50),
                                        (2, 1024, 8208, 20), (1, 1024, 8208, 0), (4, 512, 16400, 64)])
def test_linear_few_tokens_both_sides_of_its_forms(torch_dev, fmt, M, K, N, rank):
    """Down projections that the kernel forms itself and that a launch prepares, one and more row tiles a
    workgroup, against the oracle with the bound of the layer's tests."""
    torch, dev = torch_dev
    spec = synth.layer_spec("qkv", M=M, K=K, N=N, rank=rank, fmt=fmt, x_outliers=K // 100, w_outliers=K // 100, lora_rank=0)
    L = synth.draw_layer(spec, seed=70 + M)
    layer = sq.Layer(fmt, K, N, rank)
    w, X = pack(layer, L, torch, dev), dev_tensor(L["X"], torch, dev)
    o = W.layer_forward(L["X"], L["lam"], L["L1"] if rank else None, L["L2"] if rank else None, L["R"], L["b"], fmt)
    for f32 in (True, False):
        lim = (_sum_eps(K) + (2.0 ** -26 if f32 else 2.0 ** -18)) * (o["B"] + 3 * o["B_lr"] + np.abs(o["pre"]))
        if not f32:
            lim = lim + 2.0 ** -8 * (np.abs(o["Y"]) + lim)
        y = sq.linear_w4a16(layer, w, X, sq.EPI_LOWRANK | sq.EPI_BIAS | (sq.EPI_OUT_F32 if f32 else 0))
        err = np.abs(y.float().cpu().numpy().astype(np.float64) - o["Y"])
        assert np.all(err <= lim), f"f32={f32}: worst {np.max(err / lim):.2f}"
        if f32:                                              # no error shared by all outputs
            assert err.sum() <= 1e-5 * np.abs(o["Y"]).sum()
