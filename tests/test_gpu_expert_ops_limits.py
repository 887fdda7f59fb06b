"""The operators around the experts where the other tests do not reach: one GPU's
share of the experts (most sorted rows have none), all rows on one expert, float16
beside bfloat16, the longest rows and the largest numbers of them. Tolerances are
those that tests/test_gpu_matvec.py derives; what is moved is compared exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ("bfloat16", "float16")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,k,held,routed", [(8, 8, 16, 48), (24, 8, 16, 48), (40, 8, 6, 48), (5, 3, 1, 48)])
def test_a_share_of_the_experts(nv, T, k, held, routed, gated, dtype):
    """The router chooses from `routed` experts, of which this GPU holds the first
    `held`: most of the sorted rows lie behind the last one. They hold NaN and are
    neither read into a result nor written."""
    import torch
    from test_gpu_matvec import _randn, _weights, check
    dtype = getattr(torch, dtype)
    K, N = 272, 96
    bq, bsf, w, alpha = _weights(nv, held, K, N, T + held, 2 if gated else 1)
    ids = torch.from_numpy(np.argsort(np.random.RandomState(T).rand(T, routed), 1)[:, :k].astype(np.int32)).cuda()
    x = _randn((T, K), 1.5, T, dtype)
    rows = torch.full((T * k, K), float("nan"), dtype=dtype, device="cuda")
    _, offsets, row = nv.sort_tokens(x, ids, held, rows=rows)
    out = torch.full((T * k, N // 2 if gated else N), 7.0, dtype=dtype, device="cuda")
    nv.matvec(rows, bq, bsf, alpha, offsets=offsets, gated=gated, out=out)
    ends = offsets.tolist()
    assert ends[-1] < T * k
    for e in range(held):
        a, b = ends[e], ends[e + 1]
        if b > a:
            check(rows[a:b], w[e], alpha[e], out[a:b], gated)
    assert bool((out[ends[-1]:] == 7).all())
    y = nv.unsort_tokens(out, row, torch.ones((T, k), device="cuda"))
    assert bool(y.isfinite().all()) and bool((y[(row < 0).all(1)] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,E,at", [(64, 48, 47), (65, 12, 0), (129, 8, 3)])      # tiles of 4, 8 and 16 rows
def test_all_rows_on_one_expert(nv, M, E, at, dtype):
    import torch
    from test_gpu_matvec import _offsets, _randn, _weights, check
    K, N = 528, 64
    bq, bsf, w, alpha = _weights(nv, E, K, N, M)
    x = _randn((M, K), 1.5, M, getattr(torch, dtype))
    counts = [0] * E
    counts[at] = M
    out = nv.matvec(x, bq, bsf, alpha, offsets=_offsets(counts))
    check(x, w[at], alpha[at], out)


@pytest.mark.parametrize("T,E", [(700, 16), (1500, 16), (9000, 64), (2000, 97), (40000, 16)])
def test_all_slots_on_one_expert(nv, T, E):
    """Each way to rank the slots where they are all one expert's (named eight times
    by each token)."""
    import torch
    k, H, e = 8, 40, E - 3
    ids = torch.full((T, k), e, dtype=torch.int32, device="cuda")
    x = torch.arange(T * H, device="cuda", dtype=torch.float32).view(T, H)
    rows, offsets, row = nv.sort_tokens(x, ids, E)
    assert torch.equal(row.view(-1), torch.arange(T * k, device="cuda", dtype=torch.int32))
    assert offsets.tolist() == [0] * (e + 1) + [T * k] * (E - e)
    assert torch.equal(rows, x.repeat_interleave(k, 0))


@pytest.mark.parametrize("M", [1, 5, 16])
def test_longest_rows(nv, M):
    """K = 2^20. (K + 2) 2^-24 of the sum of magnitudes is derived for sums one after
    another and is wide here; that the end of K counts is checked apart."""
    import torch
    from test_gpu_matvec import _randn, _weights, check
    K, N = 1 << 20, 32
    bq, bsf, w, alpha = _weights(nv, 1, K, N, 3)
    x = _randn((M, K), 1.0, M, torch.bfloat16)
    check(x, w[0], alpha, nv.matvec(x, bq[0], bsf[0], alpha))
    x[:, :K - 64] = 0                                         # zeros add no rounding: as 64 values
    check(x[:, K - 64:], w[0, K - 64:], alpha, nv.matvec(x, bq[0], bsf[0], alpha))


def test_many_tiles(nv):
    import torch
    from test_gpu_matvec import _randn, _weights, check
    K, N, M = 16, 48, 1000003
    bq, bsf, w, alpha = _weights(nv, 1, K, N, 4)
    x = _randn((M, K), 1.0, 5, torch.bfloat16)
    check(x, w[0], alpha, nv.matvec(x, bq[0], bsf[0], alpha))


def test_dropout_of_more_elements_than_a_launch_has(nv):
    """2^32 float32 values and a few: the work-groups go round again."""
    import torch
    from test_gpu_dropout import _rng, kept
    n, p = (1 << 32) + 1003, 0.5
    x = torch.ones(n, device="cuda")
    assert nv.dropout(x, p, _rng(9, 0), y=x) is x
    for at in (0, (1 << 32) - 1024, 1 << 32, n - 999):
        m = min(999, n - at)
        lead = at % 4                                         # the first element's word of its counter
        keep = kept(m + lead, p, 9, at // 4)[lead:]
        assert torch.equal(x[at:at + m], 2.0 * torch.from_numpy(keep).cuda().float())


def test_more_pieces_than_a_launch_has(nv):
    """2^24 tokens of 66 pieces each: the moves' work-groups go round again."""
    import torch
    T, H = 1 << 24, 528
    x = torch.randint(-100, 100, (T, H), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    rows, offsets, row = nv.sort_tokens(x, ids, 1)
    assert offsets.tolist() == [0, T]
    assert torch.equal(row.view(-1), torch.arange(T, device="cuda", dtype=torch.int32))
    assert torch.equal(rows, x)
    rows.zero_()
    nv.sort_tokens_backward(x, row, dx=rows)
    assert torch.equal(rows, x)
    rows.zero_()
    nv.unsort_tokens(x, row, torch.ones((T, 1), device="cuda"), y=rows)
    assert torch.equal(rows, x)


def test_too_many_experts_allocate_nothing(nv):
    """A number of experts that the library refuses is refused before outputs of that
    size are allocated."""
    import torch
    x, w = torch.zeros((4, 32), device="cuda"), torch.zeros((4, 2), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for E in (513, 1 << 31, 1 << 42, 1 << 60):
        for call in (lambda: nv.sort_tokens(x, ids, E), lambda: nv.route_topk_backward(w, ids, w, E)):
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            with pytest.raises(nv.Nvfp4Error):
                call()
            assert torch.cuda.max_memory_allocated() - before <= 1 << 20
