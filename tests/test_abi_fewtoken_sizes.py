"""When a few-token call needs a workspace: the size query against the conditions that the header
states, and the refusal of NULL, on the host (the device-error hook is on)."""
import ctypes

import pytest

import w4a4_quantized_linear_amd as sq
from w4a4_quantized_linear_amd import _lib

P = 0x100000   # a 256-aligned fake device address; never dereferenced (validation fails first)


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


# (M, K, rank, whether a workspace is needed): 3 parts of M rows of 2 K + 16 bytes beside 16 KiB of sums
# in 152 KiB; rank and K x rank; more tokens than one MFMA has columns for three parts of
NEEDS = [(1, 22528, 0, False), (1, 23552, 0, True), (5, 4096, 0, False), (5, 4608, 0, False), (5, 5120, 0, True),
         (8, 512, 0, True), (8, 4608, 0, True), (8, 8192, 0, True), (6, 512, 0, True), (1, 8192, 32, False),
         (1, 8704, 32, True), (1, 4096, 64, False), (1, 4608, 64, True), (1, 512, 65, True), (1, 8704, 1, True)]


@pytest.mark.parametrize("M,K,rank,needed", NEEDS)
def test_linear_w4a16_workspace(L, forced_device_error, M, K, rank, needed):
    for fmt in (1, 2, 3):
        d = D(fmt, K, 512, rank)
        n = L.svdq_w4a16_bytes(d, M)
        assert (n > 0) == needed
        for epi in (1, 9):                                   # bf16 and float32 output
            def call(ws, nbytes):
                return L.svdq_linear_w4a16(d, P, P, M, K, P, 512, epi, ws, nbytes, None)
            assert call(None, 0) == (1 if needed else 6) and call(P, n) == 6
            if needed:
                assert call(P, n - 1) == 5


def test_moe_bytes_of_invalid_layers(L):
    """0 for what svdq_moe refuses, as the other size queries."""
    g, d = D(K=1024, N=1024, rank=0), D(K=512, N=256, rank=0)
    assert L.svdq_moe_bytes(g, d, 4, 2) > 0
    for bad_g in (D(fmt=0, K=1024, N=1024, rank=0), D(fmt=4, K=1024, N=1024, rank=0), D(K=1024, N=1024, rank=16)):
        assert L.svdq_moe_bytes(bad_g, d, 4, 2) == 0
    for bad_d in (D(fmt=0, K=512, N=256, rank=0), D(fmt=4, K=512, N=256, rank=0), D(K=512, N=256, rank=16)):
        assert L.svdq_moe_bytes(g, bad_d, 4, 2) == 0


@pytest.mark.parametrize("M,K,E,needed", [(1, 2560, 64, False), (1, 2568, 64, True), (1, 2560, 16, False), (1, 4096, 16, True),
                                          (1, 1280, 128, False), (1, 1288, 128, True), (1, 4096, 8, False), (1, 4104, 8, True),
                                          (256, 512, 160, False), (257, 512, 160, True), (1, 320, 512, False),
                                          (1, 328, 512, True)])
def test_route_workspace(L, forced_device_error, M, K, E, needed):
    n = L.svdq_moe_route_bytes(M, K, E)
    assert (n > 0) == needed and (n == 0 or n >= M * E * 8)

    def call(ws, nbytes):
        return L.svdq_moe_route(P, M, K, K, P, E, None, 4, 0, 1.0, P, P, ws, nbytes, None)

    assert call(None, 0) == (1 if needed else 6) and call(P, n) == 6
    if needed:
        assert call(P, n - 1) == 5
