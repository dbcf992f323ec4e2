"""The few-token entry points on the host: size queries and the refusal of every invalid call with
the documented status, before any device is touched (the device-error hook is on)."""
import ctypes

import pytest

import w4a4_quantized_linear_amd as sq
from w4a4_quantized_linear_amd import _lib

P = 0x100000   # a 256-aligned fake device address; never dereferenced (validation fails first)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return sq.lib()


@pytest.fixture
def forced_device_error(L):
    L.svdq_test_force_device_error(1)
    yield
    L.svdq_test_force_device_error(0)


def D(fmt=1, K=1024, N=512, rank=16):
    return ctypes.byref(_lib.LayerDesc(fmt, K, N, rank))


def test_sizes(L):
    assert L.svdq_w4a16_bytes(D(), 1) == 0                                  # one kernel, in LDS
    assert L.svdq_w4a16_bytes(D(rank=256), 1) >= 2 * 256 * 4                # its down projection's sums
    many = L.svdq_w4a16_bytes(D(), 100)
    assert many >= 100 * (1024 * 6 + 2 * 32 * 4) and many % 256 == 0
    assert L.svdq_w4a16_bytes(D(K=1000), 1) == 0
    assert L.svdq_w4a16_bytes(D(), -1) == 0 and L.svdq_w4a16_bytes(None, 1) == 0 and L.svdq_w4a16_bytes(D(fmt=9), 1) == 0
    assert L.svdq_moe_route_bytes(1, 1024, 64) == 0                         # one kernel
    assert L.svdq_moe_route_bytes(700, 1024, 64) >= 700 * 64 * 8
    for bad in ((-1, 1024, 64), (700, 1024, 0), (700, 1024, 513), (700, 0, 64)):
        assert L.svdq_moe_route_bytes(*bad) == 0
    g, d = D(K=1024, N=1024, rank=0), D(K=512, N=256, rank=0)
    assert L.svdq_moe_bytes(g, d, 5, 3) >= 15 * 512 * 6
    assert L.svdq_moe_bytes(g, d, 10 ** 6, 3) <= 2048 * (512 * 6 + 256 * 4) + 150000       # parts share it
    assert L.svdq_moe_bytes(g, D(K=1024, N=256, rank=0), 5, 3) == 0 and L.svdq_moe_bytes(g, d, 5, 0) == 0
    assert L.svdq_moe_bytes(g, d, 5, 33) == 0 and L.svdq_moe_bytes(None, d, 5, 3) == 0


def test_linear_w4a16_validation(L, forced_device_error):
    f, d = L.svdq_linear_w4a16, D()
    n = L.svdq_w4a16_bytes(d, 40)
    ok = [d, P, P, 40, 1024, P, 512, 15, P, n, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call() == 6 and call(_3=0, _2=None, _5=None) == 6                # valid; M = 0 without X and Y
    for i in (0, 1, 2, 5, 8):
        assert call(**{f"_{i}": None}) == 1
    assert call(_0=D(K=1000)) == 2 and call(_0=D(N=24)) == 2 and call(_0=D(rank=257)) == 2
    assert call(_3=-1) == 2 and call(_3=(1 << 26) + 1) == 2 and call(_4=1016) == 2 and call(_6=504) == 2
    assert call(_4=(1 << 24) + 8) == 2
    assert call(_0=D(fmt=0)) == 3 and call(_7=16) == 3
    assert call(_2=P + 8) == 4 and call(_5=P + 8) == 4 and call(_1=P + 16) == 4 and call(_8=P + 16) == 4
    assert call(_4=1028) == 4 and call(_6=516) == 4
    assert call(_9=n - 1) == 5
    for fmt in (1, 2, 3):
        assert call(_0=D(fmt=fmt)) == 6
    # a call that needs no workspace takes NULL
    assert call(_3=1, _8=None, _9=0) == 6 and call(_3=1, _8=None, _9=0, _0=D(rank=256)) == 1
    assert call(_3=1, _8=P, _9=0) == 6 and call(_3=1, _8=P + 8, _9=0) == 4


def test_route_validation(L, forced_device_error):
    f = L.svdq_moe_route
    # X, M, ldx, K, router, E, bias, top_k, flags, scale, ids, weights, workspace, bytes, stream
    ok = [P, 400, 1024, 1024, P, 64, None, 8, 3, 1.0, P, P, P, BIG, None]
    n = L.svdq_moe_route_bytes(400, 1024, 64)

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call() == 6 and call(_6=P) == 6 and call(_1=0, _0=None, _10=None, _11=None) == 6
    for i in (0, 4, 10, 11, 12):
        assert call(**{f"_{i}": None}) == 1
    for kw in (dict(_1=-1), dict(_2=1016), dict(_2=(1 << 24) + 8), dict(_3=0), dict(_3=65544, _2=65544), dict(_5=0),
               dict(_5=513), dict(_7=0), dict(_7=33), dict(_5=4, _7=5), dict(_9=float("nan"))):
        assert call(**kw) == 2, kw
    assert call(_8=4) == 3
    for kw in (dict(_3=1020), dict(_2=1028), dict(_0=P + 8), dict(_4=P + 8), dict(_6=P + 2), dict(_10=P + 2),
               dict(_11=P + 2), dict(_12=P + 64)):
        assert call(**kw) == 4, kw
    assert call(_13=n - 1) == 5 and call(_13=n) == 6
    assert call(_1=4, _12=None, _13=0) == 6                                 # needs none


def test_moe_validation(L, forced_device_error):
    f = L.svdq_moe
    g, d = D(K=1024, N=1024, rank=0), D(K=512, N=256, rank=0)
    n = L.svdq_moe_bytes(g, d, 4, 2)
    # dg, wg, dd, wd, E, X, M, ldx, ids, weights, top_k, Y, ldy, epi, workspace, bytes, stream
    ok = [g, P, d, P, 8, P, 4, 1024, P, P, 2, P, 256, 14, P, n, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call() == 6 and call(_6=0, _5=None, _8=None, _9=None, _11=None) == 6
    for i in (0, 1, 2, 3, 5, 8, 9, 11, 14):
        assert call(**{f"_{i}": None}) == 1
    for kw in (dict(_0=D(K=1024, N=1040, rank=0)), dict(_2=D(K=1024, N=256, rank=0)), dict(_0=D(K=1000, N=1024, rank=0)),
               dict(_4=0), dict(_4=513), dict(_6=-1), dict(_7=1016), dict(_10=0), dict(_10=33), dict(_12=248)):
        assert call(**kw) == 2, kw
    for kw in (dict(_0=D(fmt=4, K=1024, N=1024, rank=0)), dict(_2=D(fmt=0, K=512, N=256, rank=0)),
               dict(_0=D(K=1024, N=1024)), dict(_2=D(K=512, N=256)), dict(_13=1), dict(_13=16)):
        assert call(**kw) == 3, kw
    for kw in (dict(_1=P + 16), dict(_3=P + 16), dict(_14=P + 16), dict(_5=P + 8), dict(_11=P + 8), dict(_8=P + 2),
               dict(_9=P + 2), dict(_7=1028), dict(_12=260)):
        assert call(**kw) == 4, kw
    assert call(_15=n - 1) == 5
    assert call(_0=D(fmt=2, K=1024, N=1024, rank=0), _2=D(fmt=3, K=512, N=256, rank=0)) == 6   # formats may differ
