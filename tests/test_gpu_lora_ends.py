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


@pytest.mark.parametrize("M,N,K", PATHS)
def test_infinite_values_of_b(nv, M, N, K):
    """An infinity in lora_b times a shrunk row is the infinity of the product's
    sign: for a v that is a bf16 value (what is left of it is zero), for one that
    is not (what is left may have either sign), and for an infinite v. The other
    columns and the other requests' rows keep their bits."""
    import torch
    L, R = 4, 24
    ranks = [24, 9, 17, 1]
    s = make(nv, M, N, K, L, R, 2 * M + N, ids=(torch.arange(M) + 1) % (L + 1) - 1, ranks=ranks)
    ids = s["adapter_ids"]
    s["x"][ids == 2] = 0.0
    s["x"][ids == 2, 3] = 1.0                            # v of adapter 2: bf16 values, scale 1
    s["x"][ids == 3, 0] = 1.0                            # and of adapter 3: one, then infinite
    s["lora_a"][3, 0], s["lora_a"][3, 0, 0] = 0.0, 1.0
    s["lora_a"][2, :, 3] = torch.where(s["lora_a"][2, :, 3] == 0, 1.0, s["lora_a"][2, :, 3])
    s["lora_scale"][2:] = 1.0
    out = run(nv, s).clone()
    check(s, out)
    n = torch.arange(0, N, 3, device="cuda")
    sign = torch.where(n % 2 == 0, 1.0, -1.0)
    s["x"][ids == 3, 0] = float("inf")
    for a, r in enumerate(ranks):
        s["lora_b"][a, n, n % r] = (sign * float("inf")).to(torch.bfloat16)
    again = run(nv, s)
    other = torch.ones((N,), dtype=torch.bool, device="cuda")
    other[n] = False
    assert torch.equal(again[ids == -1], out[ids == -1])
    seen = 0
    for a, r in enumerate(ranks):
        rows = (ids == a).nonzero()[:, 0]
        v = s["lora_scale"][a].double() * (s["x"][rows].double() @ s["lora_a"][a, :r].double().t())
        assert bool((v != 0).all())
        expect = v[:, n % r].sign() * sign * float("inf")
        assert torch.equal(again[rows][:, n].double(), expect), a
        if a != 3:
            assert torch.equal(again[rows][:, other], out[rows][:, other])
        seen += len(rows)
    assert seen > 0
