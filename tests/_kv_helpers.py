"""A cache on the GPU and its model in numpy, shared by the cache's tests."""
from __future__ import annotations

import numpy as np

import w4a4_quantized_linear_amd as sq
from oracle import formats as F
from oracle import kv as Kv
from oracle import quant as Q

P_ROUND = {"nvfp4": 2.0 ** -11, "few": 2.0 ** -16, "many": 2.0 ** -8}   # fp16; two bf16 planes; one


def i32(a, dev, torch):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def bits(t):
    """float64 values of a bf16 tensor."""
    return t.float().cpu().numpy().astype(np.float64)


class Cache:
    """Sequences of given lengths in a pool whose unwritten bytes are all ones (NaN scales)."""

    def __init__(self, torch, dev, kv, lens, seed, cols=None, spare=3, gain=True, scale=1.0, planes=None):
        self.torch, self.dev, self.kv, self.lens = torch, dev, kv, list(lens)
        rng = self.rng = np.random.default_rng(seed)
        n = [-(-x // kv.page) for x in lens]
        self.cols = cols or max(max(n), 1)
        pages = sum(n) + spare
        order = rng.permutation(pages)
        tab = np.full((len(lens), self.cols), -1, np.int64)
        at = 0
        for b, k in enumerate(n):
            tab[b, :k] = order[at:at + k]
            at += k
        self.free = order[at:]
        self.tab = tab
        self.table = i32(tab, dev, torch)
        self.pool = torch.full((pages, sq.kv_page_bytes(kv)), 255, dtype=torch.uint8, device=dev)
        H, D = kv.heads, kv.head_dim
        M = sum(lens)
        g = np.where(rng.random((H, D)) < 0.05, 8.0, 1.0) if gain else 1.0
        self.K = self.bf16(rng.standard_normal((M, H, D)) * g * scale)
        self.V = self.bf16(rng.standard_normal((M, H, D)) * scale)
        self.cu = np.r_[0, np.cumsum(lens)]
        if M:
            sq.kv_append(kv, self.pool, self.table, i32(lens, dev, torch), self.dev_bf16(self.K.reshape(M, -1)),
                         self.dev_bf16(self.V.reshape(M, -1)), cu=i32(self.cu, dev, torch))
        self.kh, self.vh = Kv.hold(self.K, kv.fmt), Kv.hold(self.V, kv.fmt)

    def bf16(self, x):
        return F.to_bf16(np.asarray(x, np.float64))

    def dev_bf16(self, x):
        return self.torch.tensor(np.asarray(x), dtype=self.torch.float32).bfloat16().to(self.dev)

    def values(self, b):
        lo, hi = self.cu[b], self.cu[b + 1]
        return self.kh[lo:hi], self.vh[lo:hi]

    def magnitudes(self, x):
        """|values| as they enter a kernel's sums: INT4 codes enter as q + 8 with 8 times the group's sum taken off."""
        if self.kv.fmt != "int4":
            return np.abs(x)
        flat = x.reshape(-1, x.shape[-1])
        top = np.abs(flat.reshape(len(flat), -1, 64)).max(-1, keepdims=True) / 6.5       # at least the scale
        return (np.repeat(top * 24, 64, -1)).reshape(x.shape)


def query_spans(length, rows, causal, window, there):
    at = length - rows + np.arange(rows)
    behind = np.minimum(at + 1, there) if causal else np.full(rows, there)
    first = np.maximum(at - window + 1, 0) if window else np.zeros(rows, int)
    return first, behind


def check_attention(c, Qv, out, lse, q_lens, lens, Hq, scale, causal, window, what, precision, values=None, there=None):
    """out (M, Hq D) and lse against the oracle, every element within its bound and bf16's rounding."""
    kv = c.kv
    H, D = kv.heads, kv.head_dim
    g = Hq // H
    o, e = bits(out).reshape(-1, Hq, D), None if lse is None else lse.cpu().numpy().astype(np.float64)
    at = 0
    for b, (q, n) in enumerate(zip(q_lens, lens)):
        k, v = (values or c.values)(b)
        k, v = k[:n], v[:n]
        first, behind = query_spans(n, q, causal, window, min(n, len(k)) if there is None else there[b])
        for h in range(Hq):
            kk, vv = k[:, h // g], v[:, h // g]
            O, l, bo, bl = Kv.attend(Qv[at:at + q, h], kk, vv, first, behind, scale, P_ROUND[precision],
                                     c.magnitudes(kk) if len(kk) else None, c.magnitudes(vv) if len(vv) else None)
            err, lim = np.abs(o[at:at + q, h] - O), bo * 1.01 + 2.0 ** -8 * (np.abs(O) + bo) + 2.0 ** -134
            assert np.isfinite(o[at:at + q, h]).all() and (err <= lim).all(), \
                f"{what}: sequence {b} head {h}: {np.max(err / np.maximum(lim, 1e-300)):.2f} of the bound at " \
                f"{np.unravel_index(np.argmax(err - lim), err.shape)}"
            if e is not None:
                el = e[at:at + q, h]
                empty = np.isneginf(l)
                assert (np.isneginf(el) == empty).all(), f"{what}: lse of empty rows"
                assert (np.abs(el - l)[~empty] <= bl[~empty]).all(), f"{what}: lse of sequence {b} head {h}"
        at += q
