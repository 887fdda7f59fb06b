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


def test_gemm(lib):
    def f(M, N, K):
        return lib.nvfp4_gemm(*[PTR] * 6, M, N, K, PTR, PTR, BIG, None)

    assert f(1 << 40, 64, 1 << 24) == ESHAPE and f(4, 1 << 48, 1 << 17) == ESHAPE and f(0, 1 << 60, 1 << 16) == ESHAPE
    assert f(0, 16, 1 << 62) == ESHAPE and f(1 << 62, 16, 16) == ESHAPE


def test_gemm_lora(lib):
    for M, N, K in ((4, 1 << 48, 1 << 17), (0, 1 << 60, 1 << 16)):
        assert lib.nvfp4_gemm_lora(*[PTR] * 12, M, N, K, 1, 8, PTR, PTR, BIG, None) == ESHAPE
        assert lib.nvfp4_gemm_lora_workspace(M, N, K, 1, 8) == 0


def test_quantize_weights_parts(lib):
    for E, parts in ((1 << 62, 4), (1 << 60, 16), (4, 1 << 62)):
        assert lib.nvfp4_quantize_weights_parts(PTR, E, 16, 128, parts, PTR, PTR, PTR, PTR, BIG, None) == ESHAPE
