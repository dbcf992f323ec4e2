"""The cache's entry points on the host: size queries and the refusal of every invalid call with the documented
status, before any device is touched (the device-error hook is on)."""
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


def D(fmt=1, heads=4, dim=128, page=32):
    return ctypes.byref(_lib.KvDesc(fmt, heads, dim, page))


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def caller(f, ok):
    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    return call


BAD_DESC = [dict(heads=0), dict(heads=257), dict(dim=96), dict(dim=256), dict(page=8), dict(page=48), dict(page=2048)]
# pool, pages, table, ldt, cols, lens, cu, batch, M at positions 1 .. 9 of every call on one layer's cache
BAD_CACHE = [dict(_2=0), dict(_2=(1 << 30) + 1), dict(_4=7), dict(_5=0), dict(_5=1 << 26, _4=1 << 26), dict(_8=-1),
             dict(_8=16385), dict(_9=-1), dict(_9=(1 << 22) + 1), dict(_7=None), dict(_8=0)]


def test_sizes(L):
    # heads x tokens x (D / 2 codes + scales) for K and V
    assert L.svdq_kv_page_bytes(D()) == 4 * 32 * 2 * (64 + 4)
    assert L.svdq_kv_page_bytes(D(fmt=2, dim=64, page=16, heads=1)) == 16 * 2 * (32 + 2)
    assert L.svdq_kv_page_bytes(D(fmt=3, page=1024)) == 4 * 1024 * 2 * (64 + 8)
    assert L.svdq_kv_page_bytes(None) == 0 and L.svdq_kv_page_bytes(D(fmt=4)) == 0
    for bad in BAD_DESC:
        assert L.svdq_kv_page_bytes(D(**bad)) == 0
    n = L.svdq_kv_attention_bytes(D(), 100, 3, 3, 16)
    assert n > 0 and n % 256 == 0 and L.svdq_kv_attention_bytes(D(), 5000, 1, 100000, 16) == 0   # enough tiles: not split
    assert L.svdq_kv_attention_bytes(D(), 4, 3, 3, 16) == 0                     # short tables: a job is one workgroup's
    for bad in ((0, 1, 1, 16), (1 << 26, 1, 1, 16), (100, 0, 1, 16), (100, 16385, 1, 16), (100, 1, 0, 16), (100, 1, 1, 6),
                (100, 1, 1, 0), (100, 1, 1 << 23, 16), (100, 1, 1 << 22, 1024)):
        assert L.svdq_kv_attention_bytes(D(), *bad) == 0


def test_append_validation(L, forced_device_error):
    # d, pool, pages, table, ldt, cols, lens, cu, batch, M, K, ldk, V, ldv, Q, ldq, q_heads, Q_out, ldqo, norm_q,
    # norm_k, eps, freq, axis, pairs, pos, axes, flags, stream
    call = caller(L.svdq_kv_append, [D(), P, 100, P, 8, 8, P, P, 5, 40, P, 512, P, 512, P, 1024, 8, P, 1024, P, P, 1e-6, P,
                                     P, 64, P, 3, 1, None])
    assert call() == 6 and call(_9=0, _10=None, _12=None, _14=None, _17=None) == 6
    assert call(_16=0, _14=None, _17=None) == 6 and call(_24=0, _22=None, _23=None, _25=None) == 6
    assert call(_24=12, _27=0) == 6 and call(_24=24) == 6
    assert call(_19=None) == 6 and call(_20=None, _23=None, _25=None) == 6 and call(_7=None, _9=5) == 6
    for i in (0, 1, 3, 6, 10, 12, 14, 17, 22):
        assert call(**{f"_{i}": None}) == 1, i
    for bad in BAD_DESC:
        assert call(_0=D(**bad)) == 2
    for bad in BAD_CACHE + [dict(_11=504), dict(_13=504), dict(_15=1016), dict(_18=1016), dict(_11=(1 << 24) + 8),
                            dict(_16=-1), dict(_24=-2), dict(_24=66), dict(_24=7, _27=0), dict(_24=68), dict(_24=12), dict(_26=0), dict(_26=17),
                            dict(_21=-1.0), dict(_21=2.0), dict(_21=float("nan"))]:
        assert call(**bad) == 2, bad
    assert call(_0=D(fmt=0)) == 3 and call(_27=2) == 3
    for i in (1, 10, 12, 14, 17, 19, 20):
        assert call(**{f"_{i}": P + 8}) == 4, i
    for i in (3, 6, 7, 22, 23, 25):
        assert call(**{f"_{i}": P + 2}) == 4, i
    assert call(_11=516) == 4 and call(_15=1028) == 4


def test_read_validation(L, forced_device_error):
    call = caller(L.svdq_kv_read, [D(), P, 100, P, 8, 8, P, P, 5, 40, P, 512, P, 512, 8, None])
    assert call() == 6 and call(_14=0) == 6 and call(_9=0, _10=None, _12=None) == 6
    for i in (0, 1, 3, 6, 10, 12):
        assert call(**{f"_{i}": None}) == 1, i
    for bad in BAD_CACHE + [dict(_11=504), dict(_13=504)] + [dict(_0=D(**b)) for b in BAD_DESC]:
        assert call(**bad) == 2, bad
    assert call(_14=1) == 3 and call(_0=D(fmt=9)) == 3
    assert call(_10=P + 8) == 4 and call(_13=516) == 4 and call(_1=P + 32) == 4 and call(_1=P + 64) == 6


def test_attention_validation(L, forced_device_error):
    n = L.svdq_kv_attention_bytes(D(), 80, 5, 40, 16)
    # d, pool, pages, table, ldt, cols, lens, cu, batch, M, Q, ldq, q_heads, scale, window, flags, Y, ldy, lse, ws,
    # bytes, stream
    call = caller(L.svdq_kv_attention, [D(), P, 100, P, 80, 80, P, P, 5, 40, P, 2048, 16, 0.1, 0, 0, P, 2048, P, P, n, None])
    assert n > 0 and call() == 6 and call(_15=1, _18=None, _14=7) == 6
    assert call(_9=0, _10=None, _16=None, _19=None, _20=0) == 6
    for i in (0, 1, 3, 6, 10, 16, 19):
        assert call(**{f"_{i}": None}) == 1, i
    for bad in [b for b in BAD_CACHE if b != dict(_4=7)] + [dict(_4=79), dict(_11=2040), dict(_17=2040), dict(_12=6, _20=BIG), dict(_12=0), dict(_13=0.0),
                            dict(_13=-1.0), dict(_13=float("nan")), dict(_13=float("inf")), dict(_13=2.1e38), dict(_14=-1)] + [dict(_0=D(**b)) for b in BAD_DESC]:
        assert call(**bad) == 2, bad
    assert call(_8=16000, _4=1 << 25, _5=1 << 25, _20=BIG) == 6            # more units than 32 bits count: not split
    assert call(_15=2) == 3 and call(_0=D(fmt=0)) == 3
    for bad in (dict(_10=P + 8), dict(_16=P + 8), dict(_18=P + 2), dict(_19=P + 64), dict(_11=2052), dict(_1=P + 16)):
        assert call(**bad) == 4, bad
    assert call(_20=n - 1) == 5


def test_copy_validation(L, forced_device_error):
    per = L.svdq_kv_page_bytes(D())
    call = caller(L.svdq_kv_copy, [D(), P, 100, 3, 100 * per, ints(1, 2, 2), ints(5, 6, 7), 3, None])
    assert call() == 6 and call(_7=0, _5=None, _6=None) == 6 and call(_3=1, _4=0) == 6
    assert call(_5=ints(9, 2, 3), _6=ints(9, 6, 7)) == 6                   # a page onto itself
    for i in (0, 1, 5, 6):
        assert call(**{f"_{i}": None}) == 1
    for bad in [dict(_0=D(**b)) for b in BAD_DESC] + [
            dict(_2=0), dict(_3=0), dict(_3=4097), dict(_4=100 * per - 1), dict(_7=-1), dict(_7=101),
            dict(_5=ints(1, 2, 100)), dict(_5=ints(-1, 2, 3)), dict(_6=ints(5, 6, 100)), dict(_6=ints(5, -1, 7)),
            dict(_6=ints(5, 6, 5)), dict(_6=ints(5, 6, 1))]:
        assert call(**bad) == 2, bad
    many = list(range(200))
    ok = dict(_2=1000, _4=1000 * per, _7=200)
    assert call(_5=ints(*many), _6=ints(*range(500, 700)), **ok) == 6
    assert call(_5=ints(*many), _6=ints(*range(199, 399)), **ok) == 2       # page 199 is both
    assert call(_5=ints(*many), _6=ints(*([500] + list(range(500, 699)))), **ok) == 2
    assert call(_5=ints(*many), _6=ints(*many), **ok) == 6
    for n in (256, 257, 900):                                              # each size of the table they are looked up in
        ok = dict(_2=2000, _4=2000 * per, _7=n)
        src, dst = [7 * i % 1000 for i in range(n)], [1999 - i for i in range(n)]
        assert call(_5=ints(*src), _6=ints(*dst), **ok) == 6
        for i, j in ((0, n - 1), (n - 1, 0), (n // 2, 3)):
            assert call(_5=ints(*src), _6=ints(*[dst[j] if k == i else p for k, p in enumerate(dst)]), **ok) == 2
            assert call(_5=ints(*[dst[j] if k == i else p for k, p in enumerate(src)]), _6=ints(*dst), **ok) == 2
    assert call(_0=D(fmt=7)) == 3
    assert call(_1=P + 16) == 4 and call(_4=100 * per + 32) == 4


def test_compact_validation(L, forced_device_error):
    per = L.svdq_kv_page_bytes(D())
    # d, pool, pages, planes, plane_bytes, table, ldt, cols, to, ldto, cols_to, start, keep, ldkeep, most, n_keep, batch,
    # stream
    call = caller(L.svdq_kv_compact, [D(), P, 100, 2, 100 * per, P, 8, 8, P + 256, 6, 6, P, P, 50, 50, P, 5, None, 0, None])
    assert call() == 6 and call(_8=None, _9=0, _10=0) == 6 and call(_11=None) == 6 and call(_14=0, _12=None) == 6
    assert call(_16=0, _5=None, _15=None, _12=None) == 6
    for i in (0, 1, 5, 12, 15):
        assert call(**{f"_{i}": None}) == 1, i
    for bad in [dict(_0=D(**b)) for b in BAD_DESC] + [
            dict(_2=0), dict(_3=0), dict(_4=100 * per - 64), dict(_6=7), dict(_7=0), dict(_9=5), dict(_10=0),
            dict(_13=49), dict(_14=-1), dict(_16=-1), dict(_16=16385)]:
        assert call(**bad) == 2, bad
    n = L.svdq_kv_compact_bytes(D(), 2, 5, 5000, 1)
    assert n >= 5 * 5000 * 2 * 4 * 2 * 68 and n % 256 == 0 and L.svdq_kv_compact_bytes(D(), 2, 5, 5000, 0) == 0
    assert L.svdq_kv_compact_bytes(D(), 2, 5, 64, 1) == 0 and L.svdq_kv_compact_bytes(D(), 100, 5, 5000, 1) == 0
    for bad in ((None, 2, 5, 500, 1), (D(fmt=0), 2, 5, 500, 1), (D(), 0, 5, 500, 1), (D(), 2, 0, 500, 1), (D(), 2, 5, 0, 1)):
        assert L.svdq_kv_compact_bytes(*bad) == 0
    long = dict(_8=None, _9=0, _10=0, _13=5000, _14=5000)
    assert call(**long) == 1 and call(**long, _17=P) == 5 and call(**long, _17=P, _18=n - 1) == 5
    assert call(**long, _17=P, _18=n) == 6 and call(**long, _17=P + 64, _18=n) == 4 and call(**{**long, "_8": P, "_9": 8, "_10": 8}, _17=P, _18=0) == 5
    assert call(_0=D(fmt=0)) == 3
    for bad in (dict(_1=P + 16), dict(_4=100 * per + 32), dict(_5=P + 2), dict(_8=P + 2), dict(_11=P + 2), dict(_12=P + 2),
                dict(_15=P + 2)):
        assert call(**bad) == 4, bad


def test_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    kv = sq.KvLayout("mxfp4", 2, 64, 16)
    pool = torch.zeros((4, sq.kv_page_bytes(kv)), dtype=torch.uint8)
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    x = torch.zeros((1, 128), dtype=torch.bfloat16)
    for call in (lambda: sq.kv_append(kv, pool, table, lens, x, x), lambda: sq.kv_attention(kv, pool, table, lens, x),
                 lambda: sq.kv_read(kv, pool, table, lens, 1), lambda: sq.kv_copy(kv, pool, [0], [1]),
                 lambda: sq.kv_compact(kv, pool, table, table, lens)):
        with pytest.raises(ValueError):
            call()
    assert sq.kv_page_bytes(sq.KvLayout("mxfp4", 2, 96, 16)) == 0


def test_compact_onto_its_own_table(L, forced_device_error):
    """The same table is in place; a part of it, or its bytes with another stride, is neither form."""
    per = L.svdq_kv_page_bytes(D())
    call = caller(L.svdq_kv_compact, [D(), P, 100, 2, 100 * per, P, 8, 8, P, 8, 8, P, P, 50, 50, P, 5, None, 0, None])
    assert call() == 6 and call(_16=1, _9=20) == 6 and call(_16=0) == 6
    for bad in (dict(_10=6), dict(_9=16), dict(_9=16, _10=16), dict(_10=6, _16=1)):
        assert call(**bad) == 2, bad


@pytest.mark.parametrize("wrap", [1 << 32, -(1 << 32), 1 << 64])
def test_numbers_beyond_int32(wrap):
    """A size whose low 32 bits would be a valid one is invalid."""
    kv = sq.KvLayout("mxfp4", 4, 128, 32)
    for i in range(3):
        a = [4, 128, 32]
        a[i] += wrap
        assert sq.kv_page_bytes(sq.KvLayout("mxfp4", *a)) == 0
    for f, ok in ((sq.kv_attention_bytes, [100, 3, 3, 16]), (sq.kv_compact_bytes, [2, 5, 5000])):
        assert f(kv, *ok) > 0
        for i in range(len(ok)):
            a = list(ok)
            a[i] += wrap
            assert f(kv, *a) == 0, (f.__name__, i)
