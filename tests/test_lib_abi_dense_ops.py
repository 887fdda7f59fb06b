"""Argument checks of nvfp4_gemm_lora and nvfp4_gated_* on the host, before any
device is touched (runs without a GPU)."""
import ctypes

import pytest

A16 = 1 << 20          # a fake, aligned, never-dereferenced address
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    import nvfp4_block_scaled_quant_amd as nv
    return nv._lib


def p(v):
    return ctypes.c_void_p(v)


def test_gemm_lora_argument_errors(lib):
    ws = lib.nvfp4_gemm_lora_workspace

    def call(M=4, N=32, K=64, L=2, R=8, nbytes=BIG, wsp=A16, out=A16, **at):
        names = ("aq", "asf", "a_gs", "bq", "bsf", "b_alpha", "x", "lora_a", "lora_b", "scale", "rank", "ids")
        return lib.nvfp4_gemm_lora(*[p(at.get(n, A16)) for n in names], M, N, K, L, R, p(out), p(wsp), nbytes, None)

    assert call(M=0) == 0
    assert call(M=-1) == 1 and call(N=0) == 1 and call(L=0) == 1 and call(R=0) == 1 and call(K=-16) == 1
    assert call(N=24) == 2 and call(K=24) == 2 and call(R=12) == 2 and call(R=264) == 2 and call(L=8193) == 2
    assert call(M=1 << 23, K=16) == 2 and call(M=1 << 20, K=1 << 13) == 2
    for name in ("aq", "asf", "a_gs", "bq", "bsf", "b_alpha", "x", "lora_a", "lora_b", "scale", "ids"):
        assert call(**{name: 0}) == 1, name
    for name, off in (("aq", 4), ("bq", 8), ("bsf", 4), ("x", 8), ("lora_a", 8), ("lora_b", 8), ("scale", 2),
                      ("rank", 2), ("ids", 2)):
        assert call(**{name: A16 + off}) == 1, name
    assert call(out=A16 + 4) == 1 and call(out=0) == 1
    need = ws(4, 32, 64, 2, 8)
    assert need > 0 and call(nbytes=need - 1) == 3
    assert call(wsp=0) == 3 and call(wsp=A16 + 64) == 3
    assert ws(4, 24, 64, 2, 8) == 0 and ws(4, 32, 64, 2, 4) == 0 and ws(-1, 32, 64, 2, 8) == 0
    # a tiled batch: the shrunk rows come on top of nvfp4_gemm's workspace
    assert ws(4096, 6144, 7168, 8, 64) >= lib.nvfp4_gemm_workspace(4096, 6144, 7168) + 4096 * 64 * 4


def test_gated_argument_errors(lib):
    def fwd(T=4, H=32, I=16, x=A16, w=A16, act=A16, gu=0, wsp=A16, nbytes=BIG):
        return lib.nvfp4_gated_forward(p(x), p(w), T, H, I, p(act), p(gu), p(wsp), nbytes, None)

    assert fwd(T=0, x=0, w=0, act=0) == 0
    assert fwd(T=-1) == 1 and fwd(H=0) == 1 and fwd(I=-16) == 1
    assert fwd(H=24) == 2 and fwd(I=8) == 2 and fwd(T=(1 << 24) + 1) == 2 and fwd(H=(1 << 20) + 16) == 2
    assert fwd(x=0) == 1 and fwd(w=0) == 1 and fwd(act=0) == 1
    assert fwd(x=A16 + 8) == 1 and fwd(w=A16 + 2) == 1 and fwd(act=A16 + 8) == 1 and fwd(gu=A16 + 8) == 1
    need = lib.nvfp4_gated_workspace(4, 1024, 64)
    assert need > 0 and fwd(H=1024, I=64, nbytes=need - 1) == 3 and fwd(wsp=0) == 3 and fwd(wsp=A16 + 16) == 3
    assert lib.nvfp4_gated_workspace(4, 24, 64) == 0 and lib.nvfp4_gated_workspace(-1, 32, 64) == 0


def test_gated_backward_argument_errors(lib):
    def bwd(T=4, H=32, I=16, d=A16, x=A16, w=A16, gu=A16, dx=A16, dw=A16, wsp=A16, nbytes=BIG):
        return lib.nvfp4_gated_backward(p(d), p(x), p(w), p(gu), T, H, I, p(dx), p(dw), p(wsp), nbytes, None)

    assert bwd(T=0, dw=0) == 0                     # nothing to write
    assert bwd(T=-1) == 1 and bwd(H=-16) == 1 and bwd(I=0) == 1
    assert bwd(H=8) == 2 and bwd(I=24) == 2
    assert bwd(dx=0, dw=0) == 1 and bwd(d=0) == 1 and bwd(gu=0) == 1
    assert bwd(w=0) == 1 and bwd(x=0) == 1         # each needed by one of the outputs
    for name in ("d", "x", "w", "gu", "dx", "dw"):
        assert bwd(**{name: A16 + 8}) == 1, name
    need = lib.nvfp4_gated_backward_workspace(4, 32, 16)
    assert need >= 4 * 32 * 2 and bwd(nbytes=need - 1) == 3 and bwd(wsp=A16 + 128) == 3
    assert lib.nvfp4_gated_backward_workspace(4, 24, 16) == 0
