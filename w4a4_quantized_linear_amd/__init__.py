"""SVDQuant W4A4 + low-rank linear layer on MI355X (gfx950).

A thin binding over libsvdq.so (include/svdq.h).  Functions take torch tensors
that live on the GPU, pass their addresses and the current HIP stream to the
library, and return torch tensors allocated for the outputs.  All computation
happens in the library's HIP kernels; there is no fallback path, and every
call raises if the library is not built or the device is not gfx950.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

from ._lib import (EPI_BIAS, EPI_GELU, EPI_LOWRANK, EPI_OUT_F32, INT4_G64, MXFP4, NVFP4, LIB_PATH,  # noqa: F401
                   ROUTE_RENORM, ROUTE_SIGMOID, LayerDesc, SvdqError, check, lib)

FORMATS = {"mxfp4": MXFP4, "int4": INT4_G64, "nvfp4": NVFP4}
GROUPS = {"mxfp4": 32, "int4": 64, "nvfp4": 16}


@dataclass(frozen=True)
class Layer:
    """Shape of one layer: 4-bit format, input features K, output features N, rank."""

    fmt: str
    K: int
    N: int
    rank: int

    def desc(self) -> LayerDesc:
        return LayerDesc(FORMATS[self.fmt], self.K, self.N, self.rank)

    @property
    def group(self) -> int:
        return GROUPS[self.fmt]


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _desc_ref(layer: Layer):
    d = layer.desc()
    return d, ctypes.byref(d)


def weight_bytes(layer: Layer) -> int:
    d, p = _desc_ref(layer)
    return int(lib().svdq_weight_bytes(p))


def act_bytes(layer: Layer, M: int) -> int:
    d, p = _desc_ref(layer)
    return int(lib().svdq_act_bytes(p, int(M)))


def _empty_u8(n: int, device):
    torch = _torch()
    # torch's caching allocator returns 256-byte aligned blocks for fresh tensors
    return torch.empty(int(n), dtype=torch.uint8, device=device)


def pack_weight(layer: Layer, R, L1, L2, lam, bias=None, out=None, stream=None):
    """R (N x K fp32), L1 (K x r bf16), L2 (r x N bf16), lam (K fp32), bias (N bf16 or None)."""
    d, p = _desc_ref(layer)
    if out is None:
        out = _empty_u8(lib().svdq_weight_bytes(p), R.device)
    st = lib().svdq_pack_weight(p, _ptr(R), _ptr(L1 if layer.rank else None), _ptr(L2 if layer.rank else None),
                                _ptr(lam), _ptr(bias), _ptr(out), _stream(stream))
    check("svdq_pack_weight", st)
    return out


def quantize_act(layer: Layer, w_packed, X, out=None, stream=None):
    """Launch 1: X (M x K bf16, row stride X.stride(0)) -> activation workspace."""
    d, p = _desc_ref(layer)
    M = X.shape[0]
    if out is None:
        out = _empty_u8(lib().svdq_act_bytes(p, M), X.device)
    st = lib().svdq_quantize_act(p, _ptr(w_packed), _ptr(X), M, X.stride(0), _ptr(out), _stream(stream))
    check("svdq_quantize_act", st)
    return out


def gemm(layer: Layer, w_packed, a_packed, M: int, epi: int, out=None, stream=None):
    """Launch 2: Y (M x N, bf16; fp32 with EPI_OUT_F32)."""
    torch = _torch()
    d, p = _desc_ref(layer)
    if out is None:
        dt = torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
        out = torch.empty((M, layer.N), dtype=dt, device=w_packed.device)
    st = lib().svdq_gemm(p, _ptr(w_packed), _ptr(a_packed), M, _ptr(out), out.stride(0), epi, _stream(stream))
    check("svdq_gemm", st)
    return out


def gemm_quant(layer: Layer, w_packed, a_packed, M: int, epi: int, next_layer: Layer, wn_packed, out=None,
               stream=None):
    """Launch 2 of `layer` with its bf16 output quantized for `next_layer` (fused MLP
    step): returns next_layer's activation workspace, as quantize_act would fill it."""
    d, p = _desc_ref(layer)
    dn, pn = _desc_ref(next_layer)
    if out is None:
        out = _empty_u8(lib().svdq_act_bytes(pn, M), w_packed.device)
    st = lib().svdq_gemm_quant(p, _ptr(w_packed), _ptr(a_packed), M, epi, pn, _ptr(wn_packed), _ptr(out),
                               _stream(stream))
    check("svdq_gemm_quant", st)
    return out


def gemm_qkv(layer: Layer, w_packed, a_packed, M: int, epi: int, norm_q, norm_k, eps: float, rope_cos, rope_sin,
             head_dim: int = 128, out=None, stream=None):
    """Launch 2 of a fused [Q | K | V] layer with the Q/K RMS normalization (weights
    norm_q, norm_k: bf16[head_dim]) and the rotary embedding (rope_cos, rope_sin:
    fp32 M x head_dim/2) in the epilogue; returns Y (M x N bf16)."""
    torch = _torch()
    d, p = _desc_ref(layer)
    if out is None:
        out = torch.empty((M, layer.N), dtype=torch.bfloat16, device=w_packed.device)
    st = lib().svdq_gemm_qkv(p, _ptr(w_packed), _ptr(a_packed), M, epi, head_dim, _ptr(norm_q), _ptr(norm_k),
                             float(eps), _ptr(rope_cos), _ptr(rope_sin), _ptr(out), out.stride(0), _stream(stream))
    check("svdq_gemm_qkv", st)
    return out


def gemm_w4a16(layer: Layer, w_packed, X, epi: int = 0, out=None, stream=None):
    """W4A16: Y = X deQ(Q4(W))^T (+ b) for an INT4 rank-0 blob and bf16 X (M x K);
    returns Y (M x N, bf16, or float32 with EPI_OUT_F32)."""
    torch = _torch()
    d, p = _desc_ref(layer)
    M = X.shape[0]
    if out is None:
        dt = torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
        out = torch.empty((M, layer.N), dtype=dt, device=X.device)
    st = lib().svdq_gemm_w4a16(p, _ptr(w_packed), _ptr(X), M, X.stride(0), _ptr(out), out.stride(0), epi,
                               _stream(stream))
    check("svdq_gemm_w4a16", st)
    return out


def linear(layer: Layer, w_packed, X, epi: int, out=None, workspace=None, stream=None):
    """Both launches: Y = act(deQ(Q(X/lam)) deQ(Q(R))^T + (X/lam L1) L2 + b)."""
    torch = _torch()
    d, p = _desc_ref(layer)
    M = X.shape[0]
    need = lib().svdq_act_bytes(p, M)
    if workspace is None:
        workspace = _empty_u8(need, X.device)
    if out is None:
        dt = torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
        out = torch.empty((M, layer.N), dtype=dt, device=X.device)
    st = lib().svdq_linear(p, _ptr(w_packed), _ptr(X), M, X.stride(0), _ptr(out), out.stride(0), epi,
                           _ptr(workspace), workspace.numel(), _stream(stream))
    check("svdq_linear", st)
    return out


def linear_noalloc(layer: Layer, w_packed, X, epi: int, out=None, stream=None):
    """svdq_linear with the workspace in the library's static scratch (no device
    allocation by the library; `out` is allocated here when not given)."""
    torch = _torch()
    d, p = _desc_ref(layer)
    M = X.shape[0]
    if out is None:
        dt = torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
        out = torch.empty((M, layer.N), dtype=dt, device=X.device)
    st = lib().svdq_linear_noalloc(p, _ptr(w_packed), _ptr(X), M, X.stride(0), _ptr(out), out.stride(0), epi,
                                   _stream(stream))
    check("svdq_linear_noalloc", st)
    return out


# ---- few tokens: 16-bit activations, experts ----
#
# These calls check what the C entry points cannot see of a tensor (type, device, shape,
# inner stride, bytes of a packed weight) and raise ValueError.  `out` shares no elements with X.  They run on the device of
# their tensors, on `stream` or its current stream; what they allocate belongs to that stream.
# A decoding step makes many of them on kernels of a few microseconds, so a call keeps to
# plain attribute reads, raw addresses and one lookup of the layer's descriptor.

@functools.lru_cache(maxsize=4096)
def _kept_desc(layer: Layer):
    d = layer.desc()
    p = ctypes.byref(d)                                   # keeps d alive
    return p, int(lib().svdq_weight_bytes(p))


def _rows(t, name: str, cols: int, device, dtypes) -> int:
    """Row stride of a matrix of `cols` columns; a single row's is cols (its stride says nothing)."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or t.dtype not in dtypes or t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: expected rows x {cols} of {dtypes} on {device}, got {tuple(shape)} of {t.dtype} "
                         f"on {t.device}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return ld if shape[0] > 1 else (cols + 7) // 8 * 8


def _flat(t, name: str, shape, device, dtype):
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {tuple(shape)} of {dtype} on {device}, got {tuple(t.shape)} of "
                         f"{t.dtype} on {t.device}")


def _bytes(t, name: str, nbytes: int, device):
    if t.dtype != _torch().uint8 or t.numel() != nbytes or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected {nbytes} contiguous bytes on {device}, got {tuple(t.shape)} of {t.dtype} on "
                         f"{t.device}")


def _space(t, nbytes: int, device):
    """A caller's workspace, checked, or a new one; None where the call needs none (or is invalid,
    which it then reports itself)."""
    if t is None:
        return _empty_u8(nbytes, device) if nbytes else None
    if t.dtype != _torch().uint8 or t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace: expected contiguous bytes on {device}, got {t.dtype} on {t.device}")
    return t


def _elsewhere(device, stream, call):
    """call() with `device` and, if given, `stream` current."""
    torch = _torch()
    if device.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {device}")
    if stream is None:
        with torch.cuda.device(device):
            return call()
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    with torch.cuda.stream(stream):
        return call()


def w4a16_bytes(layer: Layer, M: int) -> int:
    """Workspace bytes of linear_w4a16 for M tokens (0: none needed, or invalid)."""
    return int(lib().svdq_w4a16_bytes(_kept_desc(layer)[0], int(M)))


def linear_w4a16(layer: Layer, w_packed, X, epi: int = 0, out=None, workspace=None, stream=None):
    """Y = act(X_hat deQ(Q(R))^T + (X_hat L1) L2 + b), X_hat = X / lam not quantized: a packed
    layer of any format for few tokens (X: M x K bf16); returns Y (M x N, bf16, or float32
    with EPI_OUT_F32)."""
    torch, dev = _torch(), X.device
    if stream is not None or dev.index is None or dev.index != torch.cuda.current_device():
        return _elsewhere(dev, stream, lambda: linear_w4a16(layer, w_packed, X, epi, out, workspace))
    p, wb = _kept_desc(layer)
    ldx = _rows(X, "X", layer.K, dev, (torch.bfloat16, torch.int16))
    _bytes(w_packed, "w_packed", wb, dev)
    M, N, dt = X.shape[0], layer.N, torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
    if out is None:
        out, ldy = torch.empty((M, N), dtype=dt, device=dev), N
    else:
        ldy = _rows(out, "out", N, dev, (dt,))
        if out.shape[0] != M:
            raise ValueError(f"out: {out.shape[0]} rows for {M} tokens")
    L = lib()
    ws = _space(workspace, L.svdq_w4a16_bytes(p, M), dev)
    st = L.svdq_linear_w4a16(p, w_packed.data_ptr(), X.data_ptr(), M, ldx, out.data_ptr(), ldy, epi,
                             None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                             torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        check("svdq_linear_w4a16", st)
    return out


def moe_route_bytes(M: int, K: int, E: int) -> int:
    """Workspace bytes of moe_route (0: none needed, or invalid)."""
    return int(lib().svdq_moe_route_bytes(int(M), int(K), int(E)))


def moe_route(X, router, top_k: int, bias=None, sigmoid: bool = False, renorm: bool = True, scale: float = 1.0,
              ids=None, weights=None, workspace=None, stream=None):
    """The router of a mixture of experts: X (M x K bf16), router (E x K bf16, contiguous), bias
    (float32[E] or None, for the choice only).  Returns ids (int32 M x top_k, by falling score)
    and weights (float32 M x top_k): softmax (or sigmoid) scores, divided by a token's sum with
    `renorm`, times `scale`."""
    torch, dev = _torch(), X.device
    if stream is not None or dev.index is None or dev.index != torch.cuda.current_device():
        return _elsewhere(dev, stream, lambda: moe_route(X, router, top_k, bias, sigmoid, renorm, scale, ids, weights,
                                                         workspace))
    shape = router.shape
    if len(shape) != 2 or router.dtype not in (torch.bfloat16, torch.int16):
        raise ValueError(f"router: expected experts x features of bf16, got {tuple(shape)} of {router.dtype}")
    E, K = shape
    ldx = _rows(X, "X", K, dev, (torch.bfloat16, torch.int16))
    _flat(router, "router", shape, dev, router.dtype)
    if bias is not None:
        _flat(bias, "bias", (E,), dev, torch.float32)
    M, top_k = X.shape[0], int(top_k)
    out = (M, max(top_k, 1))                              # an invalid top_k is the call's to report
    if ids is None:
        ids = torch.empty(out, dtype=torch.int32, device=dev)
    else:
        _flat(ids, "ids", out, dev, torch.int32)
    if weights is None:
        weights = torch.empty(out, dtype=torch.float32, device=dev)
    else:
        _flat(weights, "weights", out, dev, torch.float32)
    L = lib()
    ws = _space(workspace, L.svdq_moe_route_bytes(M, K, E), dev)
    st = L.svdq_moe_route(X.data_ptr(), M, ldx, K, router.data_ptr(), E, None if bias is None else bias.data_ptr(),
                          top_k, (ROUTE_SIGMOID if sigmoid else 0) | (ROUTE_RENORM if renorm else 0), scale,
                          ids.data_ptr(), weights.data_ptr(), None if ws is None else ws.data_ptr(),
                          0 if ws is None else ws.numel(), torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        check("svdq_moe_route", st)
    return ids, weights


def pack_experts(layer: Layer, R, bias=None, stream=None):
    """E experts' weights of one layer shape (rank 0, lambda 1): R (E x N x K fp32), bias (E x N
    bf16 or None) -> E x weight_bytes(layer) uint8, as moe takes them."""
    torch, dev = _torch(), R.device
    if stream is not None or dev.index is None or dev.index != torch.cuda.current_device():
        return _elsewhere(dev, stream, lambda: pack_experts(layer, R, bias))
    if layer.rank != 0 or R.dim() != 3 or tuple(R.shape[1:]) != (layer.N, layer.K):
        raise ValueError(f"expected rank 0 and weights E x {layer.N} x {layer.K}, got rank {layer.rank} and {tuple(R.shape)}")
    _flat(R, "R", R.shape, dev, torch.float32)
    if bias is not None:
        _flat(bias, "bias", (R.shape[0], layer.N), dev, bias.dtype if bias.dtype == torch.int16 else torch.bfloat16)
    out = torch.empty((R.shape[0], weight_bytes(layer)), dtype=torch.uint8, device=dev)
    one = torch.ones(layer.K, dtype=torch.float32, device=dev)
    for e in range(R.shape[0]):
        pack_weight(layer, R[e], None, None, one, None if bias is None else bias[e], out=out[e])
    return out


def moe_bytes(gate_up: Layer, down: Layer, M: int, top_k: int) -> int:
    """Workspace bytes of moe (0: invalid)."""
    return int(lib().svdq_moe_bytes(_kept_desc(gate_up)[0], _kept_desc(down)[0], int(M), int(top_k)))


def moe(gate_up: Layer, wg_packed, down: Layer, wd_packed, X, ids, weights, epi: int = 0, out=None, workspace=None,
        stream=None):
    """The experts' products of a mixture of experts for few tokens: X (M x K bf16), ids and
    weights (M x top_k, int32 and float32), wg_packed and wd_packed (E packed experts each,
    pack_experts: gate_up's outputs are [gate | up], twice down.K).  Y = sum_j weights[:, j]
    down(act(gate) * up), act SiLU or, with EPI_GELU, GELU; returns Y (M x down.N, bf16, or
    float32 with EPI_OUT_F32)."""
    torch, dev = _torch(), X.device
    if stream is not None or dev.index is None or dev.index != torch.cuda.current_device():
        return _elsewhere(dev, stream, lambda: moe(gate_up, wg_packed, down, wd_packed, X, ids, weights, epi, out,
                                                   workspace))
    (pg, gb), (pd, db) = _kept_desc(gate_up), _kept_desc(down)
    ldx = _rows(X, "X", gate_up.K, dev, (torch.bfloat16, torch.int16))
    if wg_packed.dim() != 2:
        raise ValueError(f"wg_packed: expected experts x {gb} bytes, got {tuple(wg_packed.shape)}")
    E, M, N = wg_packed.shape[0], X.shape[0], down.N
    _bytes(wg_packed, "wg_packed", E * gb, dev)
    _bytes(wd_packed, "wd_packed", E * db, dev)
    if ids.dim() != 2:
        raise ValueError(f"ids: expected tokens x choices, got {tuple(ids.shape)}")
    top_k = ids.shape[1]
    _flat(ids, "ids", (M, top_k), dev, torch.int32)
    _flat(weights, "weights", (M, top_k), dev, torch.float32)
    dt = torch.float32 if epi & EPI_OUT_F32 else torch.bfloat16
    if out is None:
        out, ldy = torch.empty((M, N), dtype=dt, device=dev), N
    else:
        ldy = _rows(out, "out", N, dev, (dt,))
        if out.shape[0] != M:
            raise ValueError(f"out: {out.shape[0]} rows for {M} tokens")
    L = lib()
    ws = _space(workspace, L.svdq_moe_bytes(pg, pd, M, top_k) or 1, dev)   # 0: invalid, the call's to report
    st = L.svdq_moe(pg, wg_packed.data_ptr(), pd, wd_packed.data_ptr(), E, X.data_ptr(), M, ldx, ids.data_ptr(),
                    weights.data_ptr(), top_k, out.data_ptr(), ldy, epi, None if ws is None else ws.data_ptr(),
                    0 if ws is None else ws.numel(), torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        check("svdq_moe", st)
    return out


def _scales_out(torch, layer: Layer, rows: int, dev):
    """Canonical scales: one byte per group (E8M0 for MXFP4, E4M3 for NVFP4) or fp16 bits (INT4)."""
    dt = torch.int16 if layer.fmt == "int4" else torch.uint8
    return torch.empty((rows, layer.K // layer.group), dtype=dt, device=dev)


def unpack_weight(layer: Layer, w_packed, stream=None) -> dict:
    """Canonical codes (N x K/2), scales, L1, L2, lambda and bias of a packed weight."""
    torch = _torch()
    d, p = _desc_ref(layer)
    dev = w_packed.device
    K, N, r = layer.K, layer.N, layer.rank
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = _scales_out(torch, layer, N, dev)
    L1 = torch.empty((K, r), dtype=torch.int16, device=dev)
    L2 = torch.empty((r, N), dtype=torch.int16, device=dev)
    lam = torch.empty(K, dtype=torch.float32, device=dev)
    bias = torch.empty(N, dtype=torch.int16, device=dev)
    st = lib().svdq_unpack_weight(p, _ptr(w_packed), _ptr(codes), _ptr(scales), _ptr(L1 if r else None),
                                  _ptr(L2 if r else None), _ptr(lam), _ptr(bias), _stream(stream))
    check("svdq_unpack_weight", st)
    return dict(codes=codes, scales=scales, L1=L1, L2=L2, lam=lam, bias=bias)


def unpack_act(layer: Layer, a_packed, M: int, stream=None) -> dict:
    """Canonical codes (M x K/2), scales and D (M x rank fp32) of an activation workspace."""
    torch = _torch()
    d, p = _desc_ref(layer)
    dev = a_packed.device
    K, r = layer.K, layer.rank
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    scales = _scales_out(torch, layer, M, dev)
    D = torch.empty((M, r), dtype=torch.float32, device=dev)
    st = lib().svdq_unpack_act(p, _ptr(a_packed), M, _ptr(codes), _ptr(scales), _ptr(D if r else None),
                               _stream(stream))
    check("svdq_unpack_act", st)
    return dict(codes=codes, scales=scales, D=D)


def device_check() -> bool:
    return lib().svdq_device_check() == 0
