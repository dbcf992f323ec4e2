"""svdq_moe_route and svdq_moe against the float64 oracle (oracle/moe.py), and their run together
with svdq_linear_w4a16.

Router: ids equal the oracle's; a weight is rounded to float32 once (2^-24 relative) from
float64 arithmetic.  Experts: the bound of oracle/moe.py's `experts` with the relative rounding
of each product's sums, 2^-24 (20 (K / 128) + 40) (at most 5 roundings an MFMA, eight MFMAs a
128 of K, and the sums across waves, planes and chunks), h held to 2^-18 (2^-26 with float32
output); the sum over a token's experts adds 2^-24 for each, a bf16 output half a step, 2^-8."""
import numpy as np
import pytest

import synth
import w4a4_quantized_linear_amd as sq
from oracle import formats as F
from oracle import moe as Mo
from oracle import quant as Q
from oracle import w4a16 as W

from _gpu_helpers import bf16_to_np, dev_tensor, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sq.lib()
    assert sq.device_check(), "current device is not gfx950"
    return torch, torch.device("cuda:0")


def _bits(a):
    return synth.bf16_bits_from_f32(np.asarray(a, np.float32))


# ------------------------------------------------------------------ router

ROUTE = [(1, 8, 1, 1), (1, 2048, 64, 8), (2, 520, 5, 5), (3, 4096, 100, 7), (4, 1000, 129, 4), (37, 2888, 160, 10),
         (64, 512, 512, 32), (300, 264, 31, 6), (5, 65536, 16, 2)]


@pytest.mark.parametrize("case", ROUTE, ids=[f"M{c[0]}-K{c[1]}-E{c[2]}-k{c[3]}" for c in ROUTE])
@pytest.mark.parametrize("sigmoid,renorm,biased", [(False, True, False), (False, False, True), (True, True, True),
                                                   (True, False, False)])
def test_route(torch_dev, case, sigmoid, renorm, biased):
    torch, dev = torch_dev
    M, K, E, k = case
    rng = np.random.default_rng(M * 7 + E)
    X, Wr = _bits(rng.standard_normal((M, K))), _bits(rng.standard_normal((E, K)) * 2 / np.sqrt(K))
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32) if biased else None
    ids, w = sq.moe_route(dev_tensor(X, torch, dev), dev_tensor(Wr, torch, dev), k,
                          bias=None if bias is None else dev_tensor(bias, torch, dev), sigmoid=sigmoid, renorm=renorm,
                          scale=1.5)
    want, ww = Mo.route(X, Wr, k, bias, sigmoid, renorm, 1.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2.0 ** -23, atol=2.0 ** -149)


def test_route_ties_strides_and_non_finite(torch_dev):
    torch, dev = torch_dev
    rng = np.random.default_rng(3)
    M, K, E, k = 9, 776, 70, 6
    Wr = rng.standard_normal((E, K)) * 2 / np.sqrt(K)
    Wr[40:70] = Wr[0:30]                                            # equal logits, to the last bit
    X, Wr = _bits(rng.standard_normal((M, K))), _bits(Wr)
    want, ww = Mo.route(X, Wr, k)
    wide = torch.full((M, K + 40), 0x7FC0, dtype=torch.int16, device=dev)
    wide[:, 16:16 + K] = dev_tensor(X, torch, dev)
    router = dev_tensor(Wr, torch, dev)
    i, w = torch.full((M + 1, k), -7, dtype=torch.int32, device=dev), torch.full((M + 1, k), -7.0, device=dev)
    sq.moe_route(wide[:, 16:16 + K], router, k, ids=i[:M], weights=w[:M])
    np.testing.assert_array_equal(i[:M].cpu().numpy(), want)
    np.testing.assert_allclose(w[:M].cpu().numpy(), ww, rtol=2.0 ** -23)
    assert bool((i[M] == -7).all()) and bool((w[M] == -7).all())
    for bits in (0x7FC0, 0x7F80, 0xFF80):
        bad = X.copy()
        bad[4, 5] = bits
        for kw in (dict(), dict(sigmoid=True), dict(bias=torch.zeros(E, device=dev))):
            i, w = (t.cpu().numpy() for t in sq.moe_route(dev_tensor(bad, torch, dev), router, k, **kw))
            ok = [m for m in range(M) if m != 4]
            np.testing.assert_array_equal(i[ok], Mo.route(X, Wr, k, sigmoid="sigmoid" in kw)[0][ok])
            assert len(set(i[4].tolist())) == k and i[4].min() >= 0 and i[4].max() < E
            assert np.isfinite(w[ok]).all()
            if bits == 0x7FC0:
                assert i[4].tolist() == list(range(k)) and np.isnan(w[4]).all()
    i, w = sq.moe_route(dev_tensor(X[:0], torch, dev), router, k)
    assert i.shape == (0, k) and w.shape == (0, k)


def test_route_zero_sum(torch_dev):
    torch, dev = torch_dev
    X = np.zeros((1, 8))
    X[0, 0] = 2.0 ** 100
    Wr = np.zeros((3, 8))
    Wr[:, 0] = -1.0
    ids, w = sq.moe_route(dev_tensor(_bits(X), torch, dev), dev_tensor(_bits(Wr), torch, dev), 2, sigmoid=True)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


# ------------------------------------------------------------------ experts


def _experts(E, fmt, N, K, rng, bias=True):
    R = (rng.standard_normal((E, N, K)) / np.sqrt(K)).astype(np.float32)
    b = _bits(rng.standard_normal((E, N)) * 0.1) if bias else None
    w, mag = np.empty((E, N, K)), np.empty((E, N, K))
    for e in range(E):
        gs = Q.nvfp4_global_scale(R[e]) if fmt == "nvfp4" else np.float32(1.0)
        c, s = Q.quantize(R[e], fmt, gs)
        w[e] = Q.dequantize(c, s, fmt, gs)
        mag[e] = np.abs(w[e])
        if fmt == "int4":
            mag[e] = (np.abs(24 + c.astype(np.float64)) + 24) * np.repeat(F.fp16_value(s), 64, axis=1)
    return R, b, w, mag


class Mixture:
    def __init__(self, torch, dev, E, H, Fh, N, fg, fd, seed, bias=True):
        rng = np.random.default_rng(seed)
        self.rng, self.E, self.H, self.F, self.N, self.bias = rng, E, H, Fh, N, bias
        self.gu, self.dn = sq.Layer(fg, H, 2 * Fh, 0), sq.Layer(fd, Fh, N, 0)
        Rg, bg, self.wg, self.mg = _experts(E, fg, 2 * Fh, H, rng, bias)
        Rd, bd, self.wd, self.md = _experts(E, fd, N, Fh, rng, bias)
        self.bg, self.bd = (None, None) if not bias else (F.bf16_value(bg), F.bf16_value(bd))
        self.pg = sq.pack_experts(self.gu, dev_tensor(Rg, torch, dev), dev_tensor(bg, torch, dev) if bias else None)
        self.pd = sq.pack_experts(self.dn, dev_tensor(Rd, torch, dev), dev_tensor(bd, torch, dev) if bias else None)

    def run(self, X, ids, w, epi, **kw):
        epi |= sq.EPI_BIAS if self.bias else 0
        return sq.moe(self.gu, self.pg, self.dn, self.pd, X, ids, w, epi, **kw)

    def check(self, torch, dev, X, ids, wt, what, gelu=False):
        wt = np.asarray(wt, np.float32)
        Xd, idd, wd = (dev_tensor(a, torch, dev) for a in (X, np.asarray(ids, np.int32), wt))
        for f32 in (True, False):
            n, planes = 2.0 ** -24, 2.0 ** -26 if f32 else 2.0 ** -18
            eps = (n * (20 * (self.H // 128) + 40), n * (20 * (self.F // 128) + 40) + planes)
            o, lim = Mo.experts(X, ids, wt, self.wg, self.bg, self.wd, self.bd, gelu, (self.mg, self.md), eps)
            lim = lim * (1 + 2.0 ** -20) + 2.0 ** -24 * (ids.shape[1] + 1) * (np.abs(o) + lim)
            if not f32:
                lim = lim + 2.0 ** -8 * (np.abs(o) + lim)
            y = self.run(Xd, idd, wd, (sq.EPI_GELU if gelu else 0) | (sq.EPI_OUT_F32 if f32 else 0))
            y = y.cpu().numpy().astype(np.float64) if f32 else bf16_to_np(y)
            err = np.abs(y - o)
            assert np.all(err <= lim), f"{what} f32={f32}: {int((err > lim).sum())} beyond the bound"
            if f32:
                assert err.sum() <= 1e-5 * np.abs(o).sum() + 1e-12, what

    def route(self, M, k, skew=0.0):
        l = self.rng.standard_normal((M, self.E)) + skew * np.arange(self.E)[::-1] / max(1, self.E)
        ids = np.argsort(-l, axis=1)[:, :k].astype(np.int32)
        return ids, self.rng.random((M, k)).astype(np.float32)


# (M, top_k, E, H, F, N, gate/up format, down format, skew): one token; one expert; every format
# and a mixed pair; experts with more than a block of pairs (8, 16, 32); N of one tile and not a
# multiple of 32; more experts than pairs and fewer; more pairs than waves
MOE = [(1, 1, 1, 512, 512, 16, "mxfp4", "mxfp4", 0), (1, 4, 9, 1024, 512, 528, "int4", "int4", 0),
       (1, 8, 16, 512, 1024, 272, "nvfp4", "nvfp4", 0), (5, 3, 4, 1536, 512, 144, "int4", "mxfp4", 0),
       (9, 2, 2, 512, 512, 256, "mxfp4", "nvfp4", 0), (33, 4, 6, 512, 512, 96, "nvfp4", "int4", 9),
       (64, 6, 40, 512, 512, 64, "mxfp4", "mxfp4", 0), (70, 1, 1, 512, 1024, 48, "int4", "nvfp4", 0),
       (3, 32, 64, 512, 512, 32, "mxfp4", "int4", 0),
       # pairs' products through memory (many pairs): N that ends inside a 32-row tile, every format
       (200, 10, 10, 512, 512, 16, "mxfp4", "mxfp4", 0), (220, 10, 11, 512, 512, 80, "int4", "int4", 0),
       (210, 10, 12, 512, 512, 48, "nvfp4", "nvfp4", 4)]


@pytest.mark.parametrize("case", MOE, ids=["-".join(map(str, c)) for c in MOE])
def test_experts(torch_dev, case):
    torch, dev = torch_dev
    M, k, E, H, Fh, N, fg, fd, skew = case
    mix = Mixture(torch, dev, E, H, Fh, N, fg, fd, seed=M + E)
    ids, wt = mix.route(M, k, skew)
    X = _bits(mix.rng.standard_normal((M, H)))
    mix.check(torch, dev, X, ids, wt, f"moe {case}", gelu=M % 2 == 0)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
@pytest.mark.parametrize("M,k,E,H,Fh,N", [(12, 4, 36, 512, 2048, 4144), (24, 8, 40, 1536, 2048, 4096),
                                           (6, 5, 24, 4096, 512, 512), (3, 2, 2, 11264, 512, 64),
                                           (40, 4, 6, 4608, 5632, 96), (64, 1, 1, 10240, 4608, 160)])
def test_experts_large(torch_dev, fmt, M, k, E, H, Fh, N):
    """Sizes that take the other forms (pairs' products through memory for at most 64 pairs and for
    more, few rows in LDS, many, and rows that come in parts), against float64 on the GPU from the packed weights' own codes
    and scales."""
    torch, dev = torch_dev
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    gu, dn = sq.Layer(fmt, H, 2 * Fh, 0), sq.Layer(fmt, Fh, N, 0)
    packed, deq = [], []
    for layer in (gu, dn):
        R = torch.randn((E, layer.N, layer.K), generator=g, device=dev) * layer.K ** -0.5
        packed.append(sq.pack_experts(layer, R))
        deq.append([])
        for e in range(E):
            u = sq.unpack_weight(layer, packed[-1][e])
            c = torch.stack([u["codes"] & 15, u["codes"] >> 4], 2).reshape(layer.N, layer.K).long()
            if fmt == "int4":
                v, s = ((c ^ 8) - 8).double(), u["scales"].view(torch.float16).double()
            else:
                t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                                 device=dev)
                v = t[c]
                s = torch.exp2(u["scales"].double() - 127) if fmt == "mxfp4" else \
                    u["scales"].view(torch.float8_e4m3fn).double() * (R[e].abs().amax() / 2688).double()
            deq[-1].append(v * s.repeat_interleave(layer.group, 1))
        del R
    ids = torch.rand((M, E), generator=g, device=dev).topk(k, 1)[1].int()
    wt = torch.rand((M, k), generator=g, device=dev)
    X = torch.randn((M, H), generator=g, device=dev).bfloat16()
    y = sq.moe(gu, packed[0], dn, packed[1], X, ids, wt, sq.EPI_OUT_F32).double()
    yb = sq.moe(gu, packed[0], dn, packed[1], X, ids, wt).double()
    want, size = torch.zeros((M, N), dtype=torch.float64, device=dev), torch.zeros((M, 1), dtype=torch.float64, device=dev)
    for m in range(M):
        for j in range(k):
            e = int(ids[m, j])
            z = deq[0][e] @ X[m].double()
            h = z[:Fh] * torch.sigmoid(z[:Fh]) * z[Fh:]
            want[m] += wt[m, j].double() * (deq[1][e] @ h)
            size[m] += wt[m, j].double() * h.abs().norm() * deq[1][e].norm(dim=1).max()
    # an error of 2^-17 of the products' size (Cauchy-Schwarz) would be 2^-24 for each of 128
    # roundings in a row; bf16 output rounds once more
    assert bool(((y - want).abs() <= 2.0 ** -17 * size).all())
    assert bool(((yb - want).abs() <= 2.0 ** -16 * size + 2.0 ** -8 * want.abs()).all())


def test_experts_without_bias_in_parts_and_odd_choices(torch_dev):
    """More than 2048 pairs (parts of 682 tokens), experts with hundreds of pairs; ids outside the
    experts, the same expert twice, zero and negative weights, a token without any expert."""
    torch, dev = torch_dev
    mix = Mixture(torch, dev, 5, 512, 512, 32, "mxfp4", "int4", seed=8, bias=False)
    M, k = 1400, 3
    ids, wt = mix.route(M, k, 6)
    mix.check(torch, dev, _bits(mix.rng.standard_normal((M, 512))), ids, wt, "parts")
    ids = np.array([[0, 0, 4], [-1, 5, 2], [-1, -1, 99], [1, 1, 1], [2 ** 31 - 1, -2 ** 31, 3]], np.int32)
    wt = np.array([[0.5, -0.25, 0.0], [9.0, 9.0, 1.0], [1.0, 1.0, 1.0], [1.0, -1.0, 2.0], [1.0, 1.0, 1.0]], np.float32)
    X = _bits(mix.rng.standard_normal((5, 512)))
    mix.check(torch, dev, X, ids, wt, "odd choices")
    y = mix.run(dev_tensor(X, torch, dev), dev_tensor(ids, torch, dev), dev_tensor(wt, torch, dev), 0)
    assert bool((y[2] == 0).all())
    assert mix.run(dev_tensor(X[:0], torch, dev), dev_tensor(ids[:0], torch, dev), dev_tensor(wt[:0], torch, dev),
                   0).shape == (0, 32)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
def test_experts_strides_non_finite_and_repeats(torch_dev, fmt):
    torch, dev = torch_dev
    M, k, H, N = 11, 3, 512, 48
    mix = Mixture(torch, dev, 4, H, 512, N, fmt, fmt, seed=9)
    ids, wt = mix.route(M, k)
    X = dev_tensor(_bits(mix.rng.standard_normal((M, H))), torch, dev)
    ids, wt = dev_tensor(ids, torch, dev), dev_tensor(wt, torch, dev)
    want = mix.run(X, ids, wt, 0)
    wide = torch.full((M, H + 16), 0x7FC0, dtype=torch.int16, device=dev)
    wide[:, 8:8 + H] = X
    out = torch.full((M + 1, N + 8), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.full((sq.moe_bytes(mix.gu, mix.dn, M, k),), 0xFF, dtype=torch.uint8, device=dev)
    for _ in range(3):
        mix.run(wide[:, 8:8 + H], ids, wt, 0, out=out[:M, :N], workspace=ws)
        assert torch.equal(out[:M, :N], want)
    assert bool((out[M] == 7).all()) and bool((out[:, N:] == 7).all())
    for bits in (0x7FC0, 0x7F80, -128):
        bad = X.clone()
        bad[6, 100] = bits
        y = mix.run(bad, ids, wt, 0)
        ok = [m for m in range(M) if m != 6]
        assert torch.equal(y[ok], want[ok]) and not bool(torch.isfinite(y[6]).any())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mix.run(X, ids, wt, 0, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 12])
def test_block_as_used(torch_dev, M):
    """Router, experts and a following projection as a decoding step runs them: against the oracle
    stage by stage, and captured in a graph whose replays, on new tokens, equal eager calls."""
    torch, dev = torch_dev
    k, H = 2, 512
    mix = Mixture(torch, dev, 6, H, 512, H, "mxfp4", "mxfp4", seed=M)
    spec = synth.layer_spec("qkv", M=M, K=H, N=144, rank=16, fmt="mxfp4", x_outliers=5, w_outliers=5, lora_rank=0)
    L = synth.draw_layer(spec, seed=4)
    layer = sq.Layer("mxfp4", H, 144, 16)
    w = pack(layer, L, torch, dev)
    Wr = _bits(mix.rng.standard_normal((6, H)) * 2 / np.sqrt(H))
    router = dev_tensor(Wr, torch, dev)

    def step(x):
        ids, wt = sq.moe_route(x, router, k)
        y = mix.run(x, ids, wt, 0)
        return ids, wt, y, sq.linear_w4a16(layer, w, y, sq.EPI_LOWRANK | sq.EPI_BIAS)

    X = _bits(mix.rng.standard_normal((M, H)))
    ids, wt, y, z = step(dev_tensor(X, torch, dev))
    want_ids, _ = Mo.route(X, Wr, k)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    mix.check(torch, dev, X, want_ids, wt.cpu().numpy(), "block")
    yb = y.view(torch.int16).cpu().numpy().view(np.uint16)
    o = W.layer_forward(yb, L["lam"], L["L1"], L["L2"], L["R"], L["b"], "mxfp4")
    lim = (2.0 ** -24 * 120 + 2.0 ** -18) * (o["B"] + 3 * o["B_lr"] + np.abs(o["Y"]))
    assert np.all(np.abs(bf16_to_np(z) - o["Y"]) <= lim + 2.0 ** -8 * (np.abs(o["Y"]) + lim))

    sx = dev_tensor(X, torch, dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step(sx)
    for r in range(4):
        new = dev_tensor(_bits(mix.rng.standard_normal((M, H))), torch, dev)
        sx.copy_(new)
        g.replay()
        eager = step(new)
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b), f"replay {r}"


def test_experts_most(torch_dev):
    """The most experts and choices, in two parts (64 tokens of 2048 pairs, and 6): four experts' weights,
    each 128 times."""
    torch, dev = torch_dev
    mix = Mixture(torch, dev, 4, 512, 512, 32, "nvfp4", "int4", seed=12)
    of = np.arange(512) % 4
    M, k, many = 70, 32, torch.from_numpy(of).to(dev)
    mix.E, mix.pg, mix.pd = 512, mix.pg[many], mix.pd[many]
    for name in ("wg", "mg", "wd", "md", "bg", "bd"):
        setattr(mix, name, getattr(mix, name)[of])
    ids, wt = mix.route(M, k)
    mix.check(torch, dev, _bits(mix.rng.standard_normal((M, 512))), ids, wt, "most")


def test_experts_beyond_4_gib(torch_dev):
    """Experts whose bytes lie behind 32-bit offsets give the bits that the same experts do at the front."""
    torch, dev = torch_dev
    gu, dn = sq.Layer("mxfp4", 4096, 4096, 0), sq.Layer("mxfp4", 2048, 512, 0)
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    pg, pd = (sq.pack_experts(l, torch.randn((2, l.N, l.K), generator=g, device=dev) * l.K ** -0.5)
              for l in (gu, dn))
    of = torch.arange(512, device=dev) % 2
    pg, pd = pg[of], pd[of]
    assert pg.numel() > 2 ** 32
    for M in (3, 70):
        X = torch.randn((M, 4096), generator=g, device=dev).bfloat16()
        ids = torch.tensor([[0, 1]], dtype=torch.int32, device=dev).repeat(M, 1)
        wt = torch.rand((M, 2), generator=g, device=dev)
        a, b = (sq.moe(gu, pg, dn, pd, X, i, wt) for i in (ids, ids + 510))
        assert torch.equal(a, b) and bool((a != 0).any())


@pytest.mark.parametrize("fmt", ["mxfp4", "int4", "nvfp4"])
def test_long_calls(torch_dev, fmt):
    """Calls that go through the plan and the pairs' products in memory: a router whose logits take a
    kernel of their own and the experts in a graph, replayed on new tokens (new choices) between eager
    calls; two calls at once on two streams; non-finite tokens; a call that no expert has a token of."""
    torch, dev = torch_dev
    M, k, H, N, E = 96, 8, 512, 48, 400
    mix = Mixture(torch, dev, 6, H, 512, N, fmt, fmt, seed=21)
    router = dev_tensor(_bits(mix.rng.standard_normal((E, H)) * 2 / np.sqrt(H)), torch, dev)
    assert sq.moe_route_bytes(M, H, E) > 0

    def step(x, **kw):
        ids, wt = sq.moe_route(x, router, k)
        return ids, wt, mix.run(x, ids % 7, wt, 0, **kw)       # 6 is no expert

    sx = dev_tensor(_bits(mix.rng.standard_normal((M, H))), torch, dev)
    step(sx)
    torch.cuda.synchronize()
    ws = torch.zeros(sq.moe_bytes(mix.gu, mix.dn, M, k), dtype=torch.uint8, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step(sx, workspace=ws)
    for r in range(4):
        new = dev_tensor(_bits(mix.rng.standard_normal((M, H))), torch, dev)
        sx.copy_(new)
        g.replay()
        eager = step(new)
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b), f"replay {r}"
        ws.fill_(0xFF)
    ids, wt, want = eager[0] % 7, eager[1], eager[2]
    mix.check(torch, dev, new.cpu().numpy(), ids.cpu().numpy(), wt.cpu().numpy(), f"long {fmt}")

    half = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    both = []
    for _ in range(5):
        both += [mix.run(new, ids, wt, 0, stream=s) for s in half]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in both)

    for bits in (0x7FC0, 0x7F80, -128):
        bad = new.clone()
        bad[60, 100] = bits
        y = mix.run(bad, ids, wt, 0)
        ok = [m for m in range(M) if m != 60]
        assert torch.equal(y[ok], want[ok]) and not bool(torch.isfinite(y[60]).any())
    y = mix.run(new, torch.full_like(ids, -1), torch.full_like(wt, float("nan")), 0)
    assert bool((y == 0).all())


def test_refusals(torch_dev):
    torch, dev = torch_dev
    mix = Mixture(torch, dev, 2, 512, 512, 32, "mxfp4", "mxfp4", seed=1)
    X = torch.zeros((3, 512), dtype=torch.bfloat16, device=dev)
    ids, wt = torch.zeros((3, 2), dtype=torch.int32, device=dev), torch.zeros((3, 2), device=dev)
    for a in ((X.float(), ids, wt), (X[:, :256], ids, wt), (X, ids.long(), wt), (X, ids[:2], wt), (X, ids, wt.double()),
              (X, ids, wt[:, :1]), (X, ids.cpu(), wt), (X, ids[0], wt), (X, ids.t().contiguous().t(), wt)):
        with pytest.raises(ValueError):
            mix.run(*a, 0)
    for kw in (dict(out=torch.zeros((3, 32), device=dev)), dict(out=torch.zeros((2, 32), dtype=X.dtype, device=dev)),
               dict(workspace=torch.zeros(4096, device=dev))):
        with pytest.raises(ValueError):
            mix.run(X, ids, wt, 0, **kw)
    with pytest.raises(ValueError):
        sq.moe(mix.gu, mix.pg, mix.dn, mix.pd[:1], X, ids, wt)
    for kw, status in ((dict(epi=sq.EPI_LOWRANK), 3), (dict(epi=0, workspace=mix.pd[0][:256]), 5)):
        with pytest.raises(sq.SvdqError) as e:
            mix.run(X, ids, wt, **kw)
        assert e.value.status == status
    for n in (0, 33):
        with pytest.raises(sq.SvdqError) as e:
            mix.run(X, torch.zeros((3, n), dtype=torch.int32, device=dev), torch.zeros((3, n), device=dev), 0)
        assert e.value.status == 2 or n == 0               # no choices: no ids either
    router = torch.zeros((4, 512), dtype=torch.bfloat16, device=dev)
    for a, kw in (((X, router[:, :256], 2), {}), ((X, router.float(), 2), {}), ((X, router, 2), dict(bias=wt[0])),
                  ((X, router, 2), dict(ids=ids[:2])), ((X, router, 2), dict(weights=wt.double())),
                  ((X.cpu(), router, 2), {})):
        with pytest.raises(ValueError):
            sq.moe_route(*a, **kw)
    for k in (0, 5, 33, -1):
        with pytest.raises(sq.SvdqError) as e:
            sq.moe_route(X, router, k)
        assert e.value.status == 2
    with pytest.raises(ValueError):
        sq.pack_experts(mix.gu, torch.zeros((2, 32, 512), device=dev))
