"""Operators of a key-value cache held in 4 bits: cases, plain forms and exact values.

A cache is a pool of pages of `page` tokens, for `H` heads of `D` features, in one of the library's formats (MXFP4,
INT4 with groups of 64, NVFP4 with a tensor scale of 1); a table gives each sequence its pages.

* append: new rows of K and V (with an RMS norm of Q's and K's heads and a rotation by positions of up to three axes)
  are quantized into their places in the pool; then the same rows are read back as values;
* attend: softmax(scale Q K^T) V over the cache, one or more queries a sequence, causal, with a window, with the
  logarithm of each row's sum;
* copy: pages to other pages, in every layer of the pool;
* compact: the tokens that are kept move to the front of a sequence, in place or into other pages.

`run` computes an operator in its plain form, from elementary torch operations on the pool's bytes, or, where `own`
is true, through w4a4_quantized_linear_amd.

A page holds, for each head, page / 16 tiles of 16 tokens: K codes (16 rows of D / 2 bytes), V codes (for each 4
tokens, 16 pieces of the 4 tokens' D / 16 features), K scales, V scales.
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
        # one short conversation: the call's latency
        dict(name="attend mxfp4 B1 700", op="attend", fmt="mxfp4", B=1, L=700, q=1, Hq=8, H=2, D=64, page=16, window=0,
             lse=False),
        # a decoding batch of many lengths, grouped heads
        dict(name="attend int4 B16 4000", op="attend", fmt="int4", B=16, L=4000, q=1, Hq=32, H=8, D=128, page=32,
             window=0, lse=False),
        # a few very long contexts
        dict(name="attend nvfp4 B3 131071", op="attend", fmt="nvfp4", B=3, L=131071, q=1, Hq=32, H=4, D=128, page=64,
             window=0, lse=True),
        # a large decoding batch: the most bytes
        dict(name="attend mxfp4 B64 8192", op="attend", fmt="mxfp4", B=64, L=8192, q=1, Hq=64, H=8, D=128, page=64,
             window=0, lse=False),
        # drafts being verified: a few queries a sequence, a sliding window, a head of its own for each query head
        dict(name="attend int4 B12 q7 window", op="attend", fmt="int4", B=12, L=3000, q=7, Hq=16, H=16, D=64, page=16,
             window=1024, lse=True),
        # a piece of a prompt on what came before it: the most operations
        dict(name="attend mxfp4 q2048 8192", op="attend", fmt="mxfp4", B=1, L=8192, q=2048, Hq=32, H=8, D=128,
             page=128, window=0, lse=False),
        # a decoding step's rows, positions of text
        dict(name="append mxfp4 B9", op="append", fmt="mxfp4", B=9, L=2000, q=1, Hq=32, H=8, D=128, page=16, norm=True,
             axes=1, halves=True, lse=False),
        # prompts with images: positions of three axes
        dict(name="append nvfp4 4099", op="append", fmt="nvfp4", B=3, L=4099, q=4099, Hq=32, H=8, D=128, page=64,
             norm=True, axes=3, halves=False, lse=False),
        # sequences that fork: their last pages, one layer
        dict(name="copy int4 5", op="copy", fmt="int4", n=5, pages=64, planes=1, H=8, D=128, page=16),
        # a pool put in order: all layers
        dict(name="copy mxfp4 300x24", op="copy", fmt="mxfp4", n=300, pages=1000, planes=24, H=8, D=128, page=32),
        # accepted drafts move to the front, in place
        dict(name="compact mxfp4 B32 in place", op="compact", fmt="mxfp4", B=32, L=600, start=580, keep=0.3, planes=24,
             H=8, D=128, page=32, inplace=True),
        # tokens evicted from long contexts
        dict(name="compact nvfp4 B3 20000", op="compact", fmt="nvfp4", B=3, L=20000, start=4, keep=0.4, planes=4, H=8,
             D=128, page=64, inplace=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "copy", "compact"])
    c = dict(op=op, fmt=rng.choice(["mxfp4", "int4", "nvfp4"]), H=_log(rng, 1, 16), D=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]))
    H = c["H"]
    if op == "copy":
        planes = _log(rng, 1, 24)
        n = _log(rng, 1, min(400, 2e8 / (planes * _page_bytes(c))))
        return dict(c, n=n, pages=3 * n + 8, planes=planes)
    if op == "compact":
        B, planes = _log(rng, 1, 32), _log(rng, 1, 8)
        return dict(c, B=B, L=_log(rng, 32, max(64, 600000 // (B * planes * H))), start=rng.randint(0, 16),
                    keep=rng.uniform(0.1, 0.9), planes=planes, inplace=rng.random() < 0.5)
    c["Hq"] = Hq = H * rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        M = _log(rng, 1, 160000 // (Hq + 2 * H))
        B = min(M, _log(rng, 1, 24))
        return dict(c, B=B, q=-(-M // B), L=_log(rng, 1, 4000), norm=rng.random() < 0.5, axes=rng.choice([0, 1, 2, 3]),
                    halves=rng.random() < 0.5, lse=False)
    B = _log(rng, 1, 48)
    c.update(B=B, window=0 if rng.random() < 0.7 else _log(rng, 16, 2000), lse=rng.random() < 0.5)
    if rng.random() < 0.6:                                            # one query a sequence
        return dict(c, q=1, L=_log(rng, 1, min(65536, 2000000 // (B * H))))
    q = _log(rng, 2, 1500 // B + 2)                                  # a draft or a piece of a prompt
    return dict(c, q=q, L=_log(rng, q, q + min(12000, 6e10 / (B * q * Hq * c["D"]))))


# ---- shapes, which hang on the case alone ----

def _spread(n, lo, hi):
    """n numbers over lo .. hi, the first of them hi."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _lengths(c):
    """New rows and lengths (with those rows) of a case's sequences; of eight or more one is an unused place."""
    q = _spread(c["B"], max(1, c["q"] // 3), c["q"])
    n = [max(a, b) for a, b in zip(_spread(c["B"], max(1, c["L"] // 10), c["L"]), q)]
    if c["B"] >= 8:
        q[1], n[1] = 1, 0
    return q, n


def _pages(n, page):
    return [-(-x // page) for x in n]


def _scale_bytes(fmt, D):
    return D // GROUP[fmt] * (2 if fmt == "int4" else 1)


def _tile_bytes(c):
    return 16 * (c["D"] + 2 * _scale_bytes(c["fmt"], c["D"]))


def _page_bytes(c):
    return c["H"] * (c["page"] // 16) * _tile_bytes(c)


# ---- the formats, and tiles of 16 tokens ----

def _quantize(x, fmt):
    """4-bit fields (as a pool holds them) of float32 rows x (..., D), and scales (..., D / group)."""
    g = x.unflatten(-1, (-1, GROUP[fmt]))
    top = g.abs().amax(-1)
    if fmt == "int4":
        s = (top / 7).clamp(max=65504).to(torch.float16)
        d = torch.where(s > 0, s.float(), torch.full_like(top, math.inf))
        f = (torch.round(g / d[..., None]).clamp(-8, 7) + 8).to(torch.uint8)
        return f.flatten(-2), s
    if fmt == "mxfp4":
        e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
        v, s = torch.ldexp(g, -e[..., None]), (e + 127).to(torch.uint8)
    else:
        q = (top / 6).clamp(max=448).to(torch.float8_e4m3fn)
        d = torch.where(q.float() > 0, q.float(), torch.full_like(top, math.inf))
        v, s = g / d[..., None], q.view(torch.uint8)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    mid[1::2] = torch.nextafter(mid[1::2], mid.new_zeros(3))         # ties go to the even code
    f = torch.bucketize(v.abs(), mid).to(torch.uint8) | (torch.signbit(g).to(torch.uint8) << 3)
    return f.flatten(-2), s


def _value_order(f, fmt):
    """V's fields of a tile (..., 16, D) in their order in the pool."""
    D = f.shape[-1]
    if fmt == "int4":
        f = f.unflatten(-1, (D // 64, 16, 4)).unflatten(-4, (4, 4))          # .., 4, token, group, piece, element
        return f.movedim(-2, -4)                                             # .., 4, piece, token, group, element
    return f.unflatten(-1, (16, D // 16)).unflatten(-3, (4, 4)).movedim(-2, -3)


def _value_unorder(f, fmt, D):
    """The reverse: fields (..., 16 D) of a tile's V to (..., 16, D)."""
    if fmt == "int4":
        f = f.unflatten(-1, (4, 16, 4, D // 64, 4)).movedim(-4, -2)
        return f.flatten(-3).flatten(-3, -2)
    return f.unflatten(-1, (4, 16, 4, D // 16)).movedim(-3, -2).flatten(-2).flatten(-3, -2)


def _nibbles(f):
    return f[..., 0::2] | (f[..., 1::2] << 4)


def _bytes_of(s):
    return s.contiguous().view(torch.uint8) if s.dtype != torch.uint8 else s


def _tiles(fk, sk, fv, sv, fmt):
    """Bytes of tiles (..., tile bytes) from fields (..., 16, D) and scales (..., 16, D / group)."""
    ks = sk if fmt != "int4" else sk.transpose(-1, -2)
    vs = sv.transpose(-1, -2)
    parts = [_nibbles(fk).flatten(-2), _nibbles(_value_order(fv, fmt)).flatten(fk.dim() - 2),
             _bytes_of(ks.contiguous()).flatten(-2), _bytes_of(vs.contiguous()).flatten(-2)]
    return torch.cat(parts, -1)


def _sections(t, fmt, D):
    """A pool's tiles (..., tile bytes), as views with the token's place as an axis of its own: K codes (.., 16, D / 2),
    V codes (.., 4, 16, 4, D / 32), K scales and V scales with their axis of 16."""
    n, s = 8 * D, 16 * _scale_bytes(fmt, D)
    k, v = t[..., :n].unflatten(-1, (16, D // 2)), t[..., n:2 * n].unflatten(-1, (4, 16, 4, D // 32))
    ks, vs = t[..., 2 * n:2 * n + s], t[..., 2 * n + s:]
    g = D // GROUP[fmt]
    w = 2 if fmt == "int4" else 1
    ks = ks.unflatten(-1, (g, 16, w)) if fmt == "int4" else ks.unflatten(-1, (16, g, 1))
    return k, v, ks, vs.unflatten(-1, (g, 16, w))


def _decode(t, fmt, D):
    """Float32 K and V (..., 16, D) of tiles (..., tile bytes)."""
    g = GROUP[fmt]
    if fmt == "int4":
        table = torch.arange(16, device=t.device).float() - 8
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=t.device)
    k, v, ks, vs = _sections(t, fmt, D)

    def values(codes, scales, order):
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(codes.dim() - 1)
        x = table[(_value_unorder(both.flatten(t.dim() - 1), fmt, D) if order else both).int()]
        if fmt == "int4":
            s = scales.contiguous().view(torch.float16)[..., 0].float()
        elif fmt == "mxfp4":
            s = torch.exp2(scales[..., 0].float() - 127)
        else:
            s = scales[..., 0].contiguous().view(torch.float8_e4m3fn).float()
        s = s if s.shape[-2] == 16 and not order and fmt != "int4" else s.transpose(-1, -2)
        return (x.unflatten(-1, (D // g, g)) * s[..., None]).flatten(-2)

    return values(k, ks, False), values(v, vs, True)


# ---- inputs ----

def _rows(c, cu, n, device):
    """Sequence and place in it of every new row."""
    cu = torch.tensor(cu, device=device)
    q = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(c["B"], device=device), q)
    m = torch.arange(len(b), device=device)
    return b, torch.tensor(n, device=device)[b] - q[b] + m - cu[b]


def _table(pages, order, cols):
    t = torch.full((len(pages), cols), -1, dtype=torch.int32, device=order.device)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def _freq(c):
    """Frequencies of the pairs and the axis of each."""
    D, axes = c["D"], c["axes"]
    if axes <= 1:
        return [10000.0 ** (-2 * i / D) for i in range(D // 2)], [0] * (D // 2)
    sizes = [D // 8] + [(D // 2 - D // 8) // (axes - 1)] * (axes - 1)
    sizes[-1] += D // 2 - sum(sizes)
    f = [10000.0 ** (-i / n) for n in sizes for i in range(n)]
    return f, [a for a, n in enumerate(sizes) for _ in range(n)]


def _inputs(case, seed):
    """A case's inputs; fields and scales of the pool's tokens apart from the pool itself."""
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if c["op"] == "copy":
        order = torch.randperm(c["pages"], generator=g, device=DEV)[: 2 * c["n"]]
        pool = torch.randint(256, (c["planes"], c["pages"], _page_bytes(c)), dtype=torch.uint8, generator=g, device=DEV)
        return dict(case=c, pool=pool, src=order[: c["n"]].tolist(), dst=order[c["n"]:].tolist(), src_t=order[: c["n"]],
                    dst_t=order[c["n"]:])
    if c["op"] == "compact":
        n = [max(x, c["start"] + 1) for x in _spread(c["B"], max(1, c["L"] // 2), c["L"])]
        kept = [max(1, int(c["keep"] * (x - c["start"]))) for x in n]
        p, p2 = _pages(n, c["page"]), _pages([c["start"] + k for k in kept], c["page"])
        order = torch.randperm(sum(p) + sum(p2), generator=g, device=DEV).int()
        pool = torch.randint(256, (c["planes"], len(order), _page_bytes(c)), dtype=torch.uint8, generator=g, device=DEV)
        keep = torch.zeros((c["B"], max(kept)), dtype=torch.int32, device=DEV)
        for b, (x, k) in enumerate(zip(n, kept)):
            at = torch.randperm(x - c["start"], generator=g, device=DEV)[:k]
            keep[b, :k] = c["start"] + at.sort()[0]
        table = _table(p, order, max(p))
        return dict(case=c, pool=pool, table=table, keep=keep,
                    to=table if c["inplace"] else _table(p2, order[sum(p):], max(p2)),
                    start=torch.full((c["B"],), c["start"], dtype=torch.int32, device=DEV),
                    n_keep=torch.tensor(kept, dtype=torch.int32, device=DEV))
    H, Hq, D, fmt, page = c["H"], c["Hq"], c["D"], c["fmt"], c["page"]
    q, n = _lengths(c)
    cu = [0]
    for x in q:
        cu.append(cu[-1] + x)
    p = _pages(n, page)
    order = torch.randperm(max(1, sum(p)), generator=g, device=DEV).int()
    s = dict(case=c, cu=cu, n=n, table=_table(p, order, max(1, max(p))),
             lens=torch.tensor(n, dtype=torch.int32, device=DEV), pages=len(order))
    s["cu_t"] = None if c["q"] == 1 else torch.tensor(cu, dtype=torch.int32, device=DEV)
    gain = 1 + 7 * (torch.rand(H, D, generator=g, device=DEV) < 0.03).float()        # outlier channels of K
    M = cu[-1]
    if c["op"] == "attend":
        s["Q"] = randn(M, Hq * D).bfloat16()
        shape = (len(order), page // 16, 16, H, D)
        s["fk"], s["sk"] = _quantize((randn(*shape) * gain).bfloat16().float(), fmt)
        s["fv"], s["sv"] = _quantize(randn(*shape).bfloat16().float(), fmt)
        return s
    qkv = randn(M, (Hq + 2 * H) * D)                                 # rows [Q | K | V] of one projection
    qkv[:, Hq * D:(Hq + H) * D] *= gain.view(-1)
    s["qkv"] = qkv.bfloat16()
    if c["norm"]:
        s["wq"], s["wk"] = (1 + 0.1 * randn(D)).bfloat16(), (1 + 0.1 * randn(D)).bfloat16()
    if c["axes"]:
        f, a = _freq(c)
        s["freq"], s["axis"] = torch.tensor(f, device=DEV), torch.tensor(a, dtype=torch.int32, device=DEV)
        if c["axes"] > 1:                                            # of a text's one axis the places are the positions
            s["pos"] = torch.randint(4096, (c["axes"], M), dtype=torch.int32, generator=g, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = s["case"]
    if c["op"] == "attend":
        def order(t):
            return t.permute(0, 3, 1, 2, 4)                          # pages, heads, tiles, 16 tokens, features
        t = _tiles(order(s.pop("fk")), order(s.pop("sk")), order(s.pop("fv")), order(s.pop("sv")), c["fmt"])
        s["pool"] = t.reshape(s["pages"], _page_bytes(c))
    if c["op"] == "append":
        s["pool"] = torch.zeros((s["pages"], _page_bytes(c)), dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms ----

def _tiled(pool, c):
    return pool.unflatten(-1, (c["H"], c["page"] // 16, _tile_bytes(c)))


def _attend(s):
    c = s["case"]
    B, H, D, g = c["B"], c["H"], c["D"], c["Hq"] // c["H"]
    cu, n = torch.tensor(s["cu"], device=DEV), s["lens"].long()
    q = cu[1:] - cu[:-1]
    t = _tiled(s["pool"], c)[s["table"].clamp(min=0).long()].transpose(1, 2)         # B, H, pages, tiles, bytes
    k, v = (x.flatten(2, 4) for x in _decode(t, c["fmt"], D))                        # B, H, L, D
    j = torch.arange(c["q"], device=DEV)
    row = (cu[:-1, None] + j).clamp(max=s["cu"][-1] - 1)
    x = s["Q"].float()[row].view(B, c["q"], H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * c["q"], D)
    z = (torch.matmul(x, k.transpose(2, 3)) * D ** -0.5).view(B, H, g, c["q"], -1)
    at, last = torch.arange(z.shape[-1], device=DEV), (n - q)[:, None] + j
    see = (at < n[:, None, None]) & (at <= last[..., None])
    if c["window"]:
        see &= at > last[..., None] - c["window"]
    z = torch.where(see[:, None, None], z, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(z - top)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, g * c["q"], -1), v).view(B, H, g, c["q"], D) / torch.where(l > 0, l, 1)
    there = j < q[:, None]
    o = o.permute(0, 3, 1, 2, 4)[there].reshape(-1, c["Hq"] * D).bfloat16()
    if not c["lse"]:
        return o
    return o, (top + torch.log(l))[..., 0].permute(0, 3, 1, 2)[there].reshape(-1, c["Hq"])


def _turn(x, cos, sin, halves):
    """Pairs of the last axis turned: neighbours, or one of each half."""
    a, b = x.chunk(2, -1) if halves else (x[..., 0::2], x[..., 1::2])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.cat([u, v], -1) if halves else torch.stack([u, v], -1).flatten(-2)


def _append(s):
    c = s["case"]
    H, Hq, D, fmt, page = c["H"], c["Hq"], c["D"], c["fmt"], c["page"]
    b, at = _rows(c, s["cu"], s["n"], DEV)
    qkv = s["qkv"].unflatten(-1, (-1, D))
    q, k, v = qkv[:, :Hq].float(), qkv[:, Hq:Hq + H].double(), qkv[:, Hq + H:].float()   # 64 bits: K's codes are choices
    if c["norm"]:
        q = q / torch.sqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["wq"].float()
        k = k / torch.sqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["wk"].double()
    if c["axes"]:
        pos = s["pos"] if c["axes"] > 1 else at[None]
        angle = (pos.double()[s["axis"].long()].t() * s["freq"].double())[:, None]
        q = _turn(q, torch.cos(angle).float(), torch.sin(angle).float(), c["halves"])
        k = _turn(k, torch.cos(angle), torch.sin(angle), c["halves"])
    q, k = q.bfloat16(), k.float().bfloat16().float()
    (fk, sk), (fv, sv) = _quantize(k, fmt), _quantize(v, fmt)

    def alone(t):                                                    # each row in a tile of its own, at place 0
        return torch.nn.functional.pad(t[:, :, None], (0, 0, 0, 15))

    new = _tiles(alone(fk), alone(sk), alone(fv), alone(sv), fmt)
    ok = at >= 0
    at, new = at.clamp(min=0), torch.where(ok[:, None, None], new, 0)
    pg, tl, tk = s["table"].long()[b, at // page].clamp(min=0), at % page // 16, at % 16
    h = torch.arange(H, device=DEV)
    pk, pv, pks, pvs = _sections(_tiled(s["pool"], c), fmt, D)
    nk, nv, nks, nvs = (t[ok] for t in _sections(new, fmt, D))
    i = (pg[ok, None], h, tl[ok, None])
    tk = tk[ok, None]
    pk[i + (tk,)] = nk[:, :, 0]
    pv[i + (tk // 4, slice(None), tk % 4)] = nv[:, :, 0, :, 0]
    if fmt == "int4":
        pks[i + (slice(None), tk)] = nks[:, :, :, 0]
    else:
        pks[i + (tk,)] = nks[:, :, 0]
    pvs[i + (slice(None), tk)] = nvs[:, :, :, 0]
    k, v = _decode(new, fmt, D)
    k, v = (torch.where(ok[:, None, None], t[:, :, 0], 0) for t in (k, v))
    return q.flatten(1), k.flatten(1), v.flatten(1)


def _copy(s):
    s["pool"][:, s["dst_t"]] = s["pool"][:, s["src_t"]]
    return s["pool"]


def _compact(s):
    c = s["case"]
    i = torch.arange(s["keep"].shape[1], device=DEV)
    b, i = (i < s["n_keep"][:, None]).nonzero(as_tuple=True)
    old, new = s["keep"][b, i].long(), c["start"] + i
    h = torch.arange(c["H"], device=DEV)

    def places(table, at):
        return table.long()[b, at // c["page"]][:, None], h, (at % c["page"] // 16)[:, None], (at % 16)[:, None]

    f, t = places(s["table"], old), places(s["to"], new)
    k, v, ks, vs = _sections(_tiled(s["pool"], c), c["fmt"], c["D"])
    layers = every = (slice(None),)
    groups = every if c["fmt"] == "int4" else ()
    k[layers + t] = k[layers + f]
    v[layers + t[:3] + (t[3] // 4,) + every + (t[3] % 4,)] = v[layers + f[:3] + (f[3] // 4,) + every + (f[3] % 4,)]
    ks[layers + t[:3] + groups + t[3:]] = ks[layers + f[:3] + groups + f[3:]]
    vs[layers + t[:3] + every + t[3:]] = vs[layers + f[:3] + every + f[3:]]
    return s["pool"]


# ---- the framework's calls ----

@functools.lru_cache(None)
def _layout(fmt, H, D, page):
    import w4a4_quantized_linear_amd as sq
    return sq.KvLayout(fmt, H, D, page)


def _call(s):
    import w4a4_quantized_linear_amd as sq
    c = s["case"]
    kv = _layout(c["fmt"], c["H"], c["D"], c["page"])
    if c["op"] == "attend":
        return sq.kv_attention(kv, s["pool"], s["table"], s["lens"], s["Q"], cu=s["cu_t"], window=c["window"],
                               lse=c["lse"])
    if c["op"] == "append":
        a, b = c["Hq"] * c["D"], (c["Hq"] + c["H"]) * c["D"]
        q = sq.kv_append(kv, s["pool"], s["table"], s["lens"], s["qkv"][:, a:b], s["qkv"][:, b:], cu=s["cu_t"],
                         Q=s["qkv"][:, :a], norm_q=s.get("wq"), norm_k=s.get("wk"), freq=s.get("freq"),
                         axis=s.get("axis"), pos=s.get("pos"), halves=c["halves"])
        k, v = sq.kv_read(kv, s["pool"], s["table"], s["lens"], s["cu"][-1], cu=s["cu_t"], f32=True)
        return q, k, v
    if c["op"] == "copy":
        return sq.kv_copy(kv, s["pool"], s["src"], s["dst"])
    return sq.kv_compact(kv, s["pool"], s["table"], s["keep"], s["n_keep"], start=s["start"],
                         to=None if c["inplace"] else s["to"])


def run(state):
    if own:
        return _call(state)
    return {"attend": _attend, "append": _append, "copy": _copy, "compact": _compact}[state["case"]["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    token = c["H"] * _tile_bytes(c) // 16
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * c["planes"] * _page_bytes(c), "flops": 0}
    if c["op"] == "compact":
        n = [max(x, c["start"] + 1) for x in _spread(c["B"], max(1, c["L"] // 2), c["L"])]
        kept = sum(max(1, int(c["keep"] * (x - c["start"]))) for x in n)
        return {"bytes": 2 * kept * c["planes"] * token + 4 * kept, "flops": 0}
    q, n = _lengths(c)
    M, Hq, D = sum(q), c["Hq"], c["D"]
    if c["op"] == "append":                                          # the rows in, Q and the cache out, the values read back
        return {"bytes": 2 * M * D * (2 * Hq + 2 * c["H"]) + 2 * M * token + 8 * M * c["H"] * D, "flops": 0}
    w = c["window"] or max(n) + 1
    pairs = sum(min(w, x - r + j + 1) for r, x in zip(q, n) for j in range(r) if x >= r)
    seen = sum(min(x, w + r - 1) for r, x in zip(q, n))
    return {"bytes": seen * token + 4 * M * Hq * D + (4 * M * Hq if c["lse"] else 0), "flops": 4 * Hq * D * pairs}


# ---- exact values: the definitions in 64 bits ----

def _values64(f, s, fmt):
    f = f.long()
    if fmt == "int4":
        v, s = (f - 8).double(), s.double()
    else:
        m = f % 8                                                    # E2M1: m / 2 below 2, then (2 + m % 2) 2^(m // 2 - 2)
        v = torch.where(m < 4, m.double() / 2, (2 + m % 2).double() * torch.exp2((m // 2 - 2).double()))
        v = torch.where(f > 7, -v, v)
        b = s.long()
        if fmt == "mxfp4":
            s = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
        else:
            s = torch.where(b < 8, (b % 8).double() * 2.0 ** -9, (8 + b % 8).double() * torch.exp2((b // 8 - 10).double()))
    return v * s.repeat_interleave(GROUP[fmt], -1)


def _attend64(s):
    c, fmt, D = s["case"], s["case"]["fmt"], s["case"]["D"]
    g, out, lse = c["Hq"] // c["H"], [], []
    for b in range(c["B"]):
        lo, hi, n = s["cu"][b], s["cu"][b + 1], s["n"][b]
        x = s["Q"][lo:hi].double().view(hi - lo, c["H"], g, D)
        if n == 0:
            out.append(x.new_zeros(hi - lo, c["Hq"] * D))
            lse.append(x.new_full((hi - lo, c["Hq"]), -math.inf))
            continue
        pages = s["table"][b, : -(-n // c["page"])].long()
        k, v = (_values64(s[f][pages].flatten(0, 2)[:n], s[z][pages].flatten(0, 2)[:n], fmt)
                for f, z in (("fk", "sk"), ("fv", "sv")))
        last = n - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)
        hide = (t > last) | (t <= last - (c["window"] or n + 1))
        o, e = torch.empty_like(x), x.new_empty(hi - lo, c["H"], g)
        for h in range(c["H"]):
            for i in range(g):
                z = (torch.mm(x[:, h, i], k[:, h].t()) / math.sqrt(D)).masked_fill(hide, -math.inf)
                e[:, h, i] = torch.logsumexp(z, 1)
                o[:, h, i] = torch.mm(torch.softmax(z, 1), v[:, h])
        out.append(o.flatten(1))
        lse.append(e.flatten(1))
    return (torch.cat(out), torch.cat(lse)) if c["lse"] else torch.cat(out)


def _nearest(x, fmt):
    """The values that 4 bits hold of rows x (64 bits, ..., D), by search among a group's values."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[-1], GROUP[fmt]):
        g = x[..., lo:lo + GROUP[fmt]]
        top = g.abs().amax(-1, keepdim=True)
        if fmt == "int4":
            s = (top.float() / 7).clamp(max=65504).half().double()
            grid = torch.arange(-7, 8, device=x.device).double()
        else:
            grid = torch.tensor([-v for v in E2M1[:0:-1]] + list(E2M1), device=x.device).double()
            if fmt == "mxfp4":
                s = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
            else:
                s = (top.float() / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
        y = torch.where(s > 0, g / s, 0)
        i = torch.searchsorted(grid, y.contiguous()).clamp(1, len(grid) - 1)
        low, high = grid[i - 1], grid[i]
        code = (i - 1 - 7).abs()                                     # magnitude's place in the grid: an even one takes a tie
        up = (high - y < y - low) | ((high - y == y - low) & (code % 2 == 1))
        out[..., lo:lo + GROUP[fmt]] = torch.where(up, high, low) * s
    return out


def _append64(s):
    c = s["case"]
    H, Hq, D, half = c["H"], c["Hq"], c["D"], c["D"] // 2
    x = s["qkv"].double().view(len(s["qkv"]), Hq + 2 * H, D)
    at = torch.tensor([n - (hi - lo) + j for lo, hi, n in zip(s["cu"], s["cu"][1:], s["n"]) for j in range(hi - lo)],
                      device=DEV)
    heads = []
    for h in range(Hq + H):
        y = x[:, h]
        if c["norm"]:
            y = y * (y.pow(2).sum(-1, keepdim=True) / D + 1e-6) ** -0.5 * s["wq" if h < Hq else "wk"].double()
        z = y.clone()
        for p in range(half if c["axes"] else 0):
            a = (s["pos"][s["axis"][p].long()] if c["axes"] > 1 else at).double() * s["freq"][p].double()
            i, j = (p, p + half) if c["halves"] else (2 * p, 2 * p + 1)
            z[:, i] = y[:, i] * torch.cos(a) - y[:, j] * torch.sin(a)
            z[:, j] = y[:, i] * torch.sin(a) + y[:, j] * torch.cos(a)
        heads.append(z)
    q = torch.stack(heads[:Hq], 1)
    k = _nearest(torch.stack(heads[Hq:], 1).float().bfloat16().double(), c["fmt"])   # K is a bf16 before it is quantized
    v = _nearest(x[:, Hq + H:], c["fmt"])
    there = (at >= 0)[:, None, None]
    return q.flatten(1), torch.where(there, k, 0).flatten(1), torch.where(there, v, 0).flatten(1)


def exact(case, seed):
    if case["op"] in ("copy", "compact"):
        return None                                                  # bytes that move
    s = _inputs(case, seed)
    return _attend64(s) if case["op"] == "attend" else _append64(s)
