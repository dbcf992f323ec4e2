"""Operators of 4-bit language-model layers for few tokens: cases, plain forms and exact values.

Three operators, in the weight formats of the W4A4 layer (MXFP4, INT4 with groups of 64, NVFP4):

* linear: Y = act(X_hat deQ(R)^T + (X_hat L1) L2 + b), X_hat = fp32(X / lambda), the 4-bit layer with
  16-bit activations;
* route: the router of a mixture of experts, logits X Wr^T, the top experts of each token and their weights;
* moe: the experts' products, Y[m] = sum_j w[m, j] (h Wd_e^T + bd_e), h = act(X Wg_e^T + bg_e) (X Wu_e^T + bu_e),
  e = ids[m, j].

`run` computes an operator in its plain form, from elementary torch operations on the canonical codes and scales,
or, where `own` is true, through w4a4_quantized_linear_amd on the packed weights.
"""
import functools
import math

import torch

own = False

DEV = "cuda"
GROUP = {"mxfp4": 32, "int4": 64, "nvfp4": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token through a small projection: the call's latency
        dict(name="linear mxfp4 M1 1024-1024", op="linear", fmt="mxfp4", M=1, K=1024, N=1024, rank=16, gelu=False,
             f32=False),
        # one token through a square projection of a 4096-wide model
        dict(name="linear int4 M1 4096-4096", op="linear", fmt="int4", M=1, K=4096, N=4096, rank=32, gelu=False,
             f32=False),
        # a few tokens into an MLP whose width ends inside a 32-row pair of tiles
        dict(name="linear nvfp4 M5 2048-8208", op="linear", fmt="nvfp4", M=5, K=2048, N=8208, rank=64, gelu=True,
             f32=False),
        # a head without a low-rank branch, float32 results
        dict(name="linear int4 M8 4096-16384 f32", op="linear", fmt="int4", M=8, K=4096, N=16384, rank=0, gelu=False,
             f32=True),
        # a batch of streams through an MLP's second projection
        dict(name="linear mxfp4 M33 12288-4096", op="linear", fmt="mxfp4", M=33, K=12288, N=4096, rank=32,
             gelu=False, f32=False),
        # one token's routing: latency
        dict(name="route M1 2048-64", op="route", M=1, K=2048, E=64, top_k=8, sigmoid=False, renorm=True),
        # a decoding batch over many experts, scores by a sigmoid with a balancing bias
        dict(name="route M61 4096-256", op="route", M=61, K=4096, E=256, top_k=8, sigmoid=True, renorm=True),
        # a short prompt; a model width that is no power of two
        dict(name="route M1000 2888-128", op="route", M=1000, K=2888, E=128, top_k=4, sigmoid=False, renorm=False),
        # one token through large experts
        dict(name="moe mxfp4 M1 E32k4", op="moe", fmt="mxfp4", M=1, H=2048, F=2048, E=32, top_k=4, gelu=False),
        # one token through many small experts
        dict(name="moe int4 M1 E64k8", op="moe", fmt="int4", M=1, H=2048, F=1024, E=64, top_k=8, gelu=False),
        # a small batch, odd counts
        dict(name="moe nvfp4 M7 E60k5", op="moe", fmt="nvfp4", M=7, H=2560, F=1024, E=60, top_k=5, gelu=False),
        # a decoding batch that reaches every expert: the largest
        dict(name="moe mxfp4 M64 E64k6", op="moe", fmt="mxfp4", M=64, H=4096, F=2048, E=64, top_k=6, gelu=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "moe", "moe"])
    if op == "linear":
        return dict(op=op, fmt=rng.choice(["mxfp4", "int4", "nvfp4"]), M=_log(rng, 1, 48), K=512 * _log(rng, 1, 24),
                    N=16 * _log(rng, 16, 1024), rank=rng.choice([0, 8, 16, 32, 48, 64, 128]),
                    gelu=rng.random() < 0.3, f32=rng.random() < 0.3)
    if op == "route":
        E = _log(rng, 8, 384)
        return dict(op=op, M=_log(rng, 1, 1024), K=8 * _log(rng, 64, 896), E=E, top_k=rng.randint(1, min(10, E)),
                    sigmoid=rng.random() < 0.5, renorm=rng.random() < 0.7)
    E = _log(rng, 8, 96)
    return dict(op=op, fmt=rng.choice(["mxfp4", "int4", "nvfp4"]), M=_log(rng, 1, 48), H=512 * _log(rng, 1, 8),
                F=512 * _log(rng, 1, 4), E=E, top_k=rng.randint(1, 8), gelu=rng.random() < 0.25)


# ---- inputs: weights quantized by the formats' rules, in canonical form and packed ----

def _encode_e2m1(v):
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return torch.bucketize(v.abs(), mid).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _quantize(w, fmt):
    """4-bit fields (N x K, one a byte), scales (N x K / group) and the tensor scale's amax."""
    N, K = w.shape
    g = w.view(N, K // GROUP[fmt], GROUP[fmt])
    top = g.abs().amax(-1)
    amax = w.abs().amax()
    if fmt == "mxfp4":
        e = (torch.frexp(top)[1] - 3).clamp_min(-127)
        f = _encode_e2m1(torch.ldexp(g, -e[..., None]))
        s = (e + 127).to(torch.uint8)
    elif fmt == "int4":
        s = (top / 7).to(torch.float16)
        f = torch.round(g / s.float()[..., None]).clamp(-8, 7).to(torch.int8).view(torch.uint8) & 15
    else:
        gs = amax / 2688
        q = (top / 6 / gs).clamp(max=448).to(torch.float8_e4m3fn)
        f = _encode_e2m1(g / (q.float() * gs)[..., None])
        s = q.view(torch.uint8)
    return f.view(N, K), s, amax


def _up(a, b):
    return (a + b - 1) // b * b


def _pad_rows(t, n):
    return torch.cat([t, t.new_zeros((n - t.shape[0],) + t.shape[1:])]) if n > t.shape[0] else t


def _packed(fields, scales, fmt, amax, L1, L2, lam, bias):
    """A layer's packed weights, in the layout that the library's packing gives them."""
    N, K = fields.shape
    Np, r = _up(N, 256), L1.shape[1]
    rp, R, S = _up(r, 32), Np // 16, K // 128
    f, s = _pad_rows(fields, Np), _pad_rows(scales, Np)
    if fmt == "int4":
        v = f.view(R, 16, S, 2, 4, 2, 2, 4)                       # tile, row, step, group, quarter, dword, nibble, byte
        codes = (v[:, :, :, :, :, :, 0] | (v[:, :, :, :, :, :, 1] << 4)).permute(0, 2, 4, 1, 3, 5, 6)
        sc = s.view(torch.int16).view(Np, S, 2).permute(1, 0, 2)
    else:
        v = f.view(R, 16, S, 4, 16, 2)                            # tile, row, step, block, byte, nibble
        codes = (v[..., 0] | (v[..., 1] << 4)).permute(0, 2, 3, 1, 4)
        sc = s.view(R, 16, S // 4, 4, 4).permute(0, 2, 4, 1, 3) if fmt == "mxfp4" else \
            s.view(R, 16, S, 4, 2).permute(0, 2, 3, 1, 4)
    l1 = torch.zeros((K, rp), dtype=torch.bfloat16, device=f.device)
    l2 = torch.zeros((Np, rp), dtype=torch.bfloat16, device=f.device)
    l1[:, :r] = L1
    l2[:N, :r] = L2.t()
    l1 = l1.view(K // 32, 4, 8, rp // 16, 16).permute(0, 3, 1, 4, 2)
    l2 = l2.view(R, 16, rp // 32, 4, 8).permute(0, 2, 3, 1, 4)
    rl = 1 / lam
    rlo = (torch.addcmul(torch.ones_like(lam, dtype=torch.float64), -rl.double(), lam.double()) * rl.double()).float()
    flags = torch.zeros(1, dtype=torch.int32, device=f.device)
    parts = [codes, sc, l1, l2, lam, rl, rlo, _pad_rows(bias, Np), flags, amax.reshape(1).float()]
    out = []
    for p in parts:
        b = p.contiguous().reshape(-1).view(torch.uint8) if p.numel() else f.new_zeros(0)
        out += [b, b.new_zeros(_up(b.numel(), 256) - b.numel())]
    return torch.cat(out)


def _canonical(fields):
    return fields[:, 0::2] | (fields[:, 1::2] << 4)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "route":
        M, K, E = case["M"], case["K"], case["E"]
        return dict(case=case, X=randn(M, K).bfloat16(), router=(randn(E, K) * K ** -0.5).bfloat16(),
                    bias=randn(E) * 0.05 if case["sigmoid"] else None)
    fmt, M = case["fmt"], case["M"]
    if case["op"] == "linear":
        K, N, r = case["K"], case["N"], case["rank"]
        gain = torch.ones(K, device=DEV)
        gain[torch.randperm(K, generator=g, device=DEV)[: max(1, K // 100)]] = 40.0     # outlier channels
        lam = gain.sqrt() * torch.exp(0.2 * randn(K))
        f, s, amax = _quantize(randn(N, K) * K ** -0.5, fmt)
        L1, L2 = (randn(K, r) * K ** -0.5).bfloat16(), (randn(r, N) * max(r, 1) ** -0.5).bfloat16()
        bias = (randn(N) * 0.1).bfloat16()
        return dict(case=case, X=(randn(M, K) * gain).bfloat16(), codes=_canonical(f), scales=s, amax=amax, L1=L1,
                    L2=L2, lam=lam, bias=bias, packed=_packed(f, s, fmt, amax, L1, L2, lam, bias))
    H, F, E, k = case["H"], case["F"], case["E"], case["top_k"]
    state = dict(case=case, X=randn(M, H).bfloat16())
    for name, N, K in (("gu", 2 * F, H), ("dn", H, F)):
        none = torch.zeros((K, 0), dtype=torch.bfloat16, device=DEV)
        one = torch.ones(K, device=DEV)
        codes, scales, amaxes, biases, packed = [], [], [], [], []
        for _ in range(E):
            f, s, amax = _quantize(randn(N, K) * K ** -0.5, fmt)
            b = (randn(N) * 0.05).bfloat16()
            codes.append(_canonical(f))
            scales.append(s)
            amaxes.append(amax)
            biases.append(b)
            packed.append(_packed(f, s, fmt, amax, none, none.new_zeros((0, N)), one, b))
        state[name] = dict(codes=torch.stack(codes), scales=torch.stack(scales), amax=torch.stack(amaxes),
                           bias=torch.stack(biases), packed=torch.stack(packed))
    logits = randn(M, E) + 0.5 * randn(E)                         # some experts are asked for more often
    top, ids = logits.topk(k, dim=1)
    state.update(ids=ids.int(), weights=torch.softmax(top, 1))
    return state


# ---- the plain forms ----

def _dequantized(codes, scales, amax, fmt):
    """Float32 values of canonical codes (..., N, K / 2) and scales (..., N, K / group)."""
    if fmt == "int4":
        v = torch.arange(16, device=codes.device)
        v = ((v ^ 8) - 8).float()
    else:
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    both = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)                    # a byte's two values
    w = both[codes.int()].reshape(scales.shape + (GROUP[fmt],))
    if fmt == "mxfp4":
        s = torch.exp2(scales.float() - 127)
    elif fmt == "int4":
        s = scales.float()
    else:
        s = scales.view(torch.float8_e4m3fn).float() * (amax / 2688)[..., None, None]
    return (w * s[..., None]).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))


def _gelu(y):
    return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))


def _linear(s):
    c = s["case"]
    x = s["X"].float() / s["lam"]
    y = x @ _dequantized(s["codes"], s["scales"], s["amax"], c["fmt"]).t()
    if c["rank"]:
        y = y + (x @ s["L1"].float()) @ s["L2"].float()
    y = y + s["bias"].float()
    if c["gelu"]:
        y = _gelu(y)
    return y if c["f32"] else y.bfloat16()


def _scores(logits, sigmoid):
    if sigmoid:
        return 1 / (1 + torch.exp(-logits))
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _route(s):
    c = s["case"]
    p = _scores(s["X"].double() @ s["router"].double().t(), c["sigmoid"])             # 64 bits: the choice is a whole number
    key = p + s["bias"].double() if s["bias"] is not None else p
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : c["top_k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), w.float()


def _moe(s):
    c = s["case"]
    M, H, F, E, k, fmt = c["M"], c["H"], c["F"], c["E"], c["top_k"], c["fmt"]
    x, ids, gu, dn = s["X"].float(), s["ids"].long(), s["gu"], s["dn"]
    if M * k <= E:                                                # fewer pairs than experts: each pair's weights
        e = ids.reshape(-1)
        wg = _dequantized(gu["codes"][e], gu["scales"][e], gu["amax"][e], fmt)
        z = torch.bmm(wg, x.repeat_interleave(k, 0)[:, :, None])[:, :, 0] + gu["bias"][e].float()
    else:                                                         # every expert on every token
        wg = _dequantized(gu["codes"], gu["scales"], gu["amax"], fmt)
        z = (x @ wg.reshape(E * 2 * F, H).t()).view(M, E, 2 * F) + gu["bias"].float()
    a, u = z[..., :F], z[..., F:]
    h = (_gelu(a) if c["gelu"] else a / (1 + torch.exp(-a))) * u
    if M * k <= E:
        wd = _dequantized(dn["codes"][e], dn["scales"][e], dn["amax"][e], fmt)
        o = (torch.bmm(wd, h[:, :, None])[:, :, 0] + dn["bias"][e].float()).view(M, k, H)
    else:
        wd = _dequantized(dn["codes"], dn["scales"], dn["amax"], fmt)
        o = torch.bmm(wd, h.permute(1, 2, 0).contiguous()).permute(2, 0, 1) + dn["bias"].float()
        o = o.gather(1, ids[:, :, None].expand(M, k, H))
    return (o * s["weights"][:, :, None]).sum(1).bfloat16()


# ---- the framework's calls ----

@functools.lru_cache(None)
def _layer(fmt, K, N, rank):
    import w4a4_quantized_linear_amd as sq
    return sq.Layer(fmt, K, N, rank)


def _call(s):
    import w4a4_quantized_linear_amd as sq
    c = s["case"]
    if c["op"] == "linear":
        epi = sq.EPI_LOWRANK | sq.EPI_BIAS | (sq.EPI_GELU if c["gelu"] else 0) | (sq.EPI_OUT_F32 if c["f32"] else 0)
        return sq.linear_w4a16(_layer(c["fmt"], c["K"], c["N"], c["rank"]), s["packed"], s["X"], epi)
    if c["op"] == "route":
        return sq.moe_route(s["X"], s["router"], c["top_k"], bias=s["bias"], sigmoid=c["sigmoid"], renorm=c["renorm"])
    epi = sq.EPI_BIAS | (sq.EPI_GELU if c["gelu"] else 0)
    return sq.moe(_layer(c["fmt"], c["H"], 2 * c["F"], 0), s["gu"]["packed"], _layer(c["fmt"], c["F"], c["H"], 0),
                  s["dn"]["packed"], s["X"], s["ids"], s["weights"], epi)


def run(state):
    if own:
        return _call(state)
    return {"linear": _linear, "route": _route, "moe": _moe}[state["case"]["op"]](state)


# ---- what a pass cannot do without ----

def _weight_bytes(fmt, N, K):
    return N * K // 2 + N * K // GROUP[fmt] * (2 if fmt == "int4" else 1)


def work(case):
    M = case["M"]
    if case["op"] == "route":
        K, E, k = case["K"], case["E"], case["top_k"]
        return {"bytes": 2 * K * (M + E) + 8 * M * k, "flops": 2 * M * K * E}
    if case["op"] == "linear":
        K, N, r = case["K"], case["N"], case["rank"]
        return {"bytes": _weight_bytes(case["fmt"], N, K) + 2 * r * (K + N) + 4 * K + 2 * N + 2 * M * K
                + (4 if case["f32"] else 2) * M * N, "flops": 2 * M * (K * N + r * (K + N))}
    H, F, E, k = case["H"], case["F"], case["E"], case["top_k"]
    hit = E * (1 - (1 - min(k, E) / E) ** M)                      # experts that some token asks for, on average
    return {"bytes": hit * (_weight_bytes(case["fmt"], 2 * F, H) + _weight_bytes(case["fmt"], H, F) + 4 * F + 2 * H)
            + 4 * M * H + 8 * M * k, "flops": 6 * M * k * H * F}


# ---- exact values: the definitions in 64 bits ----

def _matrix64(codes, scales, amax, fmt):
    n = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device=codes.device)
    n[:, 0::2], n[:, 1::2] = codes % 16, codes // 16
    if fmt == "int4":
        v, s = torch.where(n > 7, n - 16, n).double(), scales.double()
    else:
        m = n % 8                                                 # E2M1: m / 2 below 2, then (2 + m % 2) 2^(m // 2 - 2)
        v = torch.where(m < 4, m.double() / 2, (2 + m % 2).double() * torch.exp2((m // 2 - 2).double()))
        v = torch.where(n > 7, -v, v)
        b = scales.long()
        if fmt == "mxfp4":
            s = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
        else:
            e, m = b // 8, (b % 8).double()
            s = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double())) * (amax / 2688).double()
    return v * s.repeat_interleave(GROUP[fmt], 1)


def _gelu64(y):
    return y * torch.special.ndtr(y)


def exact(case, seed):
    s = prepare(case, seed)
    X = s["X"].double()
    if case["op"] == "linear":
        x = (s["X"].float() / s["lam"]).double()                  # the definition's float32 quotient
        y = torch.mm(_matrix64(s["codes"], s["scales"], s["amax"], case["fmt"]), x.t()).t()
        y = y + torch.mm(torch.mm(x, s["L1"].double()), s["L2"].double()) + s["bias"].double()
        return _gelu64(y) if case["gelu"] else y
    if case["op"] == "route":
        logits = torch.mm(s["router"].double(), X.t()).t()
        p = torch.sigmoid(logits) if case["sigmoid"] else torch.softmax(logits, 1)
        key = p.clone() if s["bias"] is None else p + s["bias"].double()
        ids = []
        for _ in range(case["top_k"]):                            # the largest, the lowest index first
            at = (key == key.amax(1, keepdim=True)).int().argmax(1)
            ids.append(at)
            key[torch.arange(len(at), device=key.device), at] = -math.inf
        ids = torch.stack(ids, 1)
        w = torch.stack([p[i, r] for i, r in enumerate(ids)])
        return ids.int(), w / w.sum(1, keepdim=True) if case["renorm"] else w
    F, fmt = case["F"], case["fmt"]
    y = torch.zeros((case["M"], case["H"]), dtype=torch.float64, device=DEV)
    for e in s["ids"].unique().tolist():
        m, j = (s["ids"] == e).nonzero(as_tuple=True)
        gu, dn = ({n: t[e] for n, t in s[name].items()} for name in ("gu", "dn"))
        z = X[m] @ _matrix64(gu["codes"], gu["scales"], gu["amax"], fmt).t() + gu["bias"].double()
        a = z[:, :F]
        h = (_gelu64(a) if case["gelu"] else a * torch.sigmoid(a)) * z[:, F:]
        o = h @ _matrix64(dn["codes"], dn["scales"], dn["amax"], fmt).t() + dn["bias"].double()
        y.index_add_(0, m, o * s["weights"][m, j].double()[:, None])   # a token has an expert once
    return y
