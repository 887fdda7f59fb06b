"""The one-launch form of nvfp4_gemm_lora (up to four rows of small adapters):
broken adapters and ranks at their ends, each with rows of its own in the batch."""
import pytest

from test_gpu_lora import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [2, 3, 4])
def test_a_broken_adapter_reaches_its_own_rows_only(nv, M):
    import torch
    L, R, N, K = 5, 24, 272, 528                     # M R K <= 2^18 and M R <= 128: one launch
    for broken in range(M):
        s = make(nv, M, N, K, L, R, 10 * M + broken, ids=torch.arange(M), ranks=[24, 9, 16, 24, 1])
        out = run(nv, s).clone()
        check(s, out)
        s["lora_a"][broken, 0], s["lora_b"][broken, ::3, 0] = float("inf"), float("nan")
        again = run(nv, s)
        keep = torch.arange(M, device="cuda") != broken
        assert torch.equal(again[keep], out[keep])
        assert bool(again[broken, ::3].isnan().all())


@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_ranks_at_their_ends(nv, M):
    """Ranks of zero, below zero and beyond R, every adapter with a row; what lies
    beyond a rank is broken and not used."""
    import torch
    L, R, N, K = 6, 24, 272, 528
    ranks = [0, -3, 24, 100, 1, -2 ** 31]
    for first in range(L):
        ids = (first + torch.arange(M)) % L
        s = make(nv, M, N, K, L, R, 7 * M + first, ids=ids, ranks=ranks)
        out = run(nv, s).clone()
        check(s, out)
        for a, r in enumerate(ranks):
            r = max(0, min(R, r))
            s["lora_a"][a, r:] = float("nan")
            s["lora_b"][a, :, r:] = float("inf")
        assert torch.equal(run(nv, s), out)
