"""Sizes whose products leave 64 bits are refused like all that are too large, on the
host, before any device is touched (runs without a GPU)."""
import ctypes

import pytest

PTR = ctypes.c_void_p(1 << 20)     # a fake, aligned, never-dereferenced address
BIG = 1 << 44
ESHAPE = 2


@pytest.fixture(scope="module")
def lib():
    import nvfp4_block_scaled_quant_amd as nv
    return nv._lib


# 2^55 * 512 is 0 in 64 bits; the last is the least size that is refused for its product
@pytest.mark.parametrize("T,E,k", [(1 << 55, 512, 8), ((1 << 55) + 1, 512, 8), (1 << 62, 4, 1), ((1 << 63) - 1, 3, 1),
                                   (1 << 31, 1, 1), ((1 << 31) // 3 + 1, 3, 1)])
def test_router_gradient(lib, T, E, k):
    assert lib.nvfp4_route_topk_backward(PTR, PTR, PTR, T, E, k, PTR, None) == ESHAPE


@pytest.mark.parametrize("M,N,K,offsets", [
    (1 << 24, 1 << 48, 1 << 17, None),          # N * pitch_q(K) and the tiles' number wrap to 0
    (0, 1 << 60, 1 << 16, None), (0, 1 << 60, 1 << 16, PTR), (1, 1 << 58, 16, None), (1, 1 << 31, 1 << 20, PTR),
    (4, (1 << 63) - 32, 16, None)])
@pytest.mark.parametrize("flags", [0, 1])
def test_matvec(lib, M, N, K, offsets, flags):
    assert lib.nvfp4_matvec(PTR, 0, PTR, PTR, PTR, offsets, M, N, K, 1, flags, PTR, None) == ESHAPE
