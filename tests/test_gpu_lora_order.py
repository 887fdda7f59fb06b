"""nvfp4_gemm_lora beside nvfp4_gemm, which sums the same K chunks: rows without
an adapter have the plain projection's bits."""
import pytest

from test_gpu_lora import check, make, run

pytestmark = pytest.mark.gpu


# 2, 5, 7, 16 and 12 chunks of K (dense_ksplit); the last two are tiled although
# narrow because their adapters are large
@pytest.mark.parametrize("M,N,K,L,R", [(700, 272, 528, 4, 16), (256, 6144, 7168, 6, 16), (200, 4144, 7168, 5, 24),
                                       (256, 512, 4096, 48, 128), (200, 528, 3600, 48, 256)])
def test_rows_without_an_adapter_have_the_plain_projections_bits(nv, M, N, K, L, R):
    import torch
    s = make(nv, M, N, K, L, R, M + K)
    out = run(nv, s)
    check(s, out)
    plain = nv.gemm(s["aq"], s["asf"], s["a_gs"], s["bq"], s["bsf"], s["b_alpha"])
    bare = (s["adapter_ids"] < 0) | (s["adapter_ids"] >= L)
    assert int(bare.sum()) > 0 and torch.equal(out[bare], plain[bare])


def test_chunks_are_added_in_order(nv):
    """Sixteen chunks of 256 K values whose sums in order are 2^24, 2^24 (+ 1 is
    lost), 2^24 (again), 0: any other grouping of the four leaves a one or a two."""
    import torch
    M, N, K, L, R = 256, 512, 4096, 48, 128
    s = make(nv, M, N, K, L, R, 5, ids=torch.where(torch.arange(M) % 2 == 0, -1, torch.arange(M) % L))
    aq, asf = torch.zeros((M, K // 2), dtype=torch.uint8), torch.zeros((M, K // 16), dtype=torch.uint8)
    wq, wsf = torch.zeros((1, K // 2, N), dtype=torch.uint8), torch.zeros((1, K // 16, N), dtype=torch.uint8)
    one, big = 0x38, 0x78                            # E4M3 bits of 1 and 256
    for chunk, sign in ((0, 1), (8, -1)):            # sixteen products (4 x 256)^2 = 2^20
        k = 256 * chunk
        aq[:, k // 2:k // 2 + 8] = 0x66 if sign > 0 else 0xEE       # +-4, +-4
        wq[:, k // 2:k // 2 + 8] = 0x66
        asf[:, k // 16], wsf[:, k // 16] = big, big
    for chunk in (6, 7):                             # one product 1 x 1
        k = 256 * chunk
        aq[:, k // 2], wq[:, k // 2] = 0x02, 0x02
        asf[:, k // 16], wsf[:, k // 16] = one, one
    bq, bsf = nv.prepack_weights(wq.cuda(), wsf.cuda())
    s.update(aq=aq.cuda(), asf=asf.cuda(), a_gs=torch.ones((1,), device="cuda"), bq=bq[0], bsf=bsf[0],
             b_alpha=torch.ones((1,), device="cuda"))
    plain = nv.gemm(s["aq"], s["asf"], s["a_gs"], s["bq"], s["bsf"], s["b_alpha"])
    assert bool((plain == 0).all())
    assert bool((run(nv, s)[::2] == 0).all())
