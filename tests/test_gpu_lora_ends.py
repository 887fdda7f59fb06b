"""nvfp4_gemm_lora at the ends of the number range, in each of its kernels.

Tolerances are those of test_gpu_lora.py; infinities are compared exactly."""
import pytest

from test_gpu_lora import check, make, run

pytestmark = pytest.mark.gpu

# M, N, K: the one-launch form; weight streams of one, two and four row blocks and
# of two parts; tiled with K chunks, rows ranked and sorted; tiled with the adapters
# in the GEMM's epilogue (K 144: one chunk), rows ranked and sorted, 128- and
# 256-row tiles
PATHS = [(4, 272, 528), (9, 272, 528), (20, 272, 528), (64, 272, 528), (100, 272, 528), (100, 8224, 528),
         (700, 272, 528), (100, 8224, 144), (700, 272, 144), (1300, 6144, 144)]


@pytest.mark.parametrize("M,N,K", PATHS)
def test_finite_shrunk_rows_stay_finite(nv, M, N, K):
    """v = scale * x A^T between the largest bf16 and the largest float32: finite
    in float32, as products with B far below one are."""
    import torch
    L, R = 3, 8
    s = make(nv, M, N, K, L, R, M + N, ids=torch.arange(M) % (L + 1) - 1)
    s["x"].zero_()
    s["x"][:, 0] = 1.0
    s["lora_a"][:, :, 0] = torch.tensor([1, -1, 0.99609375, 1, 2.0 ** -20, -1, 0, 1]).to(torch.bfloat16).cuda()
    s["lora_scale"] = torch.tensor([3.4e38, -3.4e38, 3.402e38], device="cuda")
    s["lora_b"] *= 2.0 ** -10
    out = run(nv, s)
    assert bool(out.isfinite().all())
    check(s, out)
