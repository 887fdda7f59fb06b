"""Products of a few rows with packed 4-bit weights against the definition in
float64 over the canonical weights (so the packed layout is checked too).

Tolerances, element by element: the products of x and a dequantized weight are
exact in float32's matrix cores; their sum is off by at most (K + 2) 2^-24 of the
sum of magnitudes (alpha included), and the result is one rounding of it. Gated: as
tests/test_gpu_gated.py derives it (|d silu| <= 1.1, |silu(g)| <= |g|, and 16
roundings of float32 in the activation and the product)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
DTYPES = ("bfloat16", "float16")


def _weights(nv, E, K, N, seed, parts=1):
    """Packed weights of E matrices, their float64 values without alpha, alpha."""
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    w = (torch.randn((E, K, N), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    q, sf, alpha = nv.quantize_weights(w) if parts == 1 else nv.quantize_weights_parts(w, parts)
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64).cuda()
    v = torch.stack((e2m1[(q & 15).long()], e2m1[(q >> 4).long()]), 2).view(E, K, N)
    v = v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return nv.prepack_weights(q, sf) + (v, alpha)


def _randn(shape, std, seed, dtype):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def check(x, w, alpha, out, gated=False):
    """alpha: one value, or (gate, up)."""
    import torch
    K = w.shape[0]
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps / 2 + 1e-36
    xd = x.double()
    a = alpha.double().reshape(-1)
    a = a.repeat_interleave(w.shape[1] // a.numel())
    ref, eps = (xd @ w) * a, (K + 2) * F32 * (xd.abs() @ w.abs()) * a.abs()
    if gated:
        g, u = ref.chunk(2, 1)
        eg, eu = eps.chunk(2, 1)
        ref = g * torch.sigmoid(g) * u
        eps = 1.1 * u.abs() * eg + g.abs() * eu + eg * eu + 16 * F32 * ref.abs()
    err = (out.double() - ref).abs()
    tol = half * ref.abs() + eps * (1 + half) + tiny
    assert bool((err <= tol).all()), float((err / tol).max())


# one row, part of a tile, several tiles; K with ends inside a 128-element step
# and inside a group of four, of one to all waves and several groups a wave; odd
# numbers of column blocks
SIZES = [(1, 16, 16), (1, 6144, 7168), (2, 48, 32), (3, 32, 144), (5, 112, 528), (13, 7168, 2048), (15, 16, 4112),
         (16, 64, 512), (17, 144, 640), (16, 528, 1040), (1, 2064, 20000), (33, 272, 784), (100, 512, 1024),
         (7, 4112, 272), (16, 4112, 144), (9, 64, 4096), (8, 4096, 2064)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_one_matrix(nv, M, N, K, dtype):
    import torch
    dtype = getattr(torch, dtype)
    bq, bsf, w, alpha = _weights(nv, 1, K, N, M + N + K)
    x = _randn((M, K), 1.5, M, dtype)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    got = nv.matvec(x, bq[0], bsf[0], alpha, out=out)
    assert got is out
    check(x, w[0], alpha, out)
    # each row alone gives the same bits (at these sizes as many waves share K)
    for m in {0, M // 2, M - 1}:
        assert torch.equal(nv.matvec(x[m:m + 1], bq[0], bsf[0], alpha), out[m:m + 1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,parts", [(1, 32, 16, 1), (1, 4096, 7168, 2), (4, 96, 272, 1), (16, 1376, 528, 2),
                                         (21, 64, 2048, 1)])
def test_gated(nv, M, N, K, parts, dtype):
    import torch
    dtype = getattr(torch, dtype)
    bq, bsf, w, alpha = _weights(nv, 1, K, N, M + N + K, parts)
    x = _randn((M, K), 2.0, M, dtype)
    out = nv.matvec(x, bq[0], bsf[0], alpha.view(-1), gated=True)
    assert out.shape == (M, N // 2) and out.dtype == dtype
    check(x, w[0], alpha, out, gated=True)


def _offsets(counts):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,N,counts,rest", [
    (16, 32, [1], 0), (272, 64, [0, 0, 3, 0, 1, 0], 5), (512, 96, [16, 17, 0, 15, 33, 1], 0), (1040, 64, [0, 0, 0], 7),
    (784, 32, [1 if e % 3 else 0 for e in range(130)], 2), (64, 32, [2] * 512, 1), (7168, 512, [1, 2, 0, 4], 1),
    (528, 96, [8, 5, 0, 9, 7], 1), (1040, 4192, [5, 8, 3, 6], 0)])
def test_each_expert_has_its_rows(nv, K, N, counts, rest, gated):
    """Empty experts, experts of more than a tile, more than 64 experts; rows behind
    the last are left as they were."""
    import torch
    E, M = len(counts), sum(counts) + rest
    bq, bsf, w, alpha = _weights(nv, E, K, N, K + N + E, 2 if gated else 1)
    x = _randn((M, K), 1.5, M, torch.bfloat16)
    n_out = N // 2 if gated else N
    out = torch.full((M, n_out), 7.0, dtype=torch.bfloat16, device="cuda")
    offsets = _offsets(counts)
    nv.matvec(x, bq, bsf, alpha, offsets=offsets, gated=gated, out=out)
    ends = offsets.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if b > a:
            check(x[a:b], w[e], alpha[e], out[a:b], gated)
            one = nv.matvec(x[a:b], bq[e], bsf[e], alpha[e].reshape(-1), gated=gated)
            assert torch.equal(one, out[a:b])
    assert bool((out[ends[-1]:] == 7).all())


def test_offsets_that_leave_the_rows(nv):
    """What offsets name beyond M (or below 0) is ignored; rows in range are there."""
    import torch
    K, N = 272, 32
    bq, bsf, w, alpha = _weights(nv, 3, K, N, 5)
    x = _randn((20, K), 1.0, 1, torch.bfloat16)
    buf = torch.full((40, N), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[10:30]
    off = torch.tensor([-9, 4, 12, 1 << 30], dtype=torch.int32).cuda()
    nv.matvec(x, bq, bsf, alpha, offsets=off, out=out)
    check(x[:4], w[0], alpha[0], out[:4])
    check(x[4:12], w[1], alpha[1], out[4:12])
    check(x[12:], w[2], alpha[2], out[12:])
    assert bool((buf[:10] == 7).all()) and bool((buf[30:] == 7).all())
    out.fill_(7.0)
    nv.matvec(x, bq, bsf, alpha, offsets=torch.tensor([30, 30, 40, 50], dtype=torch.int32).cuda(), out=out)
    assert bool((buf == 7).all())


def test_rows_are_separate(nv):
    import torch
    for M, K, N in ((5, 528, 64), (20, 2048, 48)):
        bq, bsf, w, alpha = _weights(nv, 1, K, N, M)
        x = _randn((M, K), 1.5, M, torch.bfloat16)
        out = nv.matvec(x, bq[0], bsf[0], alpha)
        bad = x.clone()
        bad[M - 2, ::3], bad[M - 2, 1::3] = float("nan"), float("inf")
        got = nv.matvec(bad, bq[0], bsf[0], alpha)
        keep = torch.arange(M, device="cuda") != M - 2
        assert torch.equal(got[keep], out[keep]) and bool(got[M - 2].isnan().all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_scale(nv, dtype):
    """Every nibble under every finite scale byte, one product an output: exact up
    to the result's rounding."""
    import torch
    dtype = getattr(torch, dtype)
    K, N = 16, 128 * 16
    n = torch.arange(N)
    code, byte = (n % 16).to(torch.uint8), (n // 16).to(torch.uint8)
    byte[byte == 0x7F] = 0x7E
    q = torch.zeros((1, K // 2, N), dtype=torch.uint8)
    q[0, 3] = code << 4                                       # k = 7
    bq, bsf = nv.prepack_weights(q.cuda(), byte.view(1, 1, N).contiguous().cuda())
    x = torch.zeros((1, K), dtype=dtype, device="cuda")
    x[0, 7] = 1.25
    alpha = torch.tensor([0.5], device="cuda")
    out = nv.matvec(x, bq[0], bsf[0], alpha)
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    val = mag[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0).double()
    ref = (0.625 * val * byte.view(torch.float8_e4m3fn).double()).cuda()
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    assert bool(((out[0].double() - ref).abs() <= half * ref.abs() + tiny).all())


def test_values_at_the_ends_of_the_types(nv):
    """Rows of very large and very small values: their sums scale with them."""
    import torch
    K, N = 528, 48
    bq, bsf, w, alpha = _weights(nv, 1, K, N, 3)
    base = _randn((3, K), 1.0, 4, torch.bfloat16)
    for power in (-100, 100):
        x = base * 2.0 ** power
        check(x, w[0], alpha, nv.matvec(x, bq[0], bsf[0], alpha))
    x = (base.float() * 2.0 ** -14).to(torch.float16)         # float16 with subnormal numbers
    check(x, w[0], alpha, nv.matvec(x, bq[0], bsf[0], alpha))


def test_streams_and_graph(nv):
    import torch
    K, N, E, M = 1040, 256, 6, 24
    bq, bsf, w, alpha = _weights(nv, E, K, N, 8, 2)
    x, off = _randn((M, K), 1.0, 1, torch.bfloat16), _offsets([3, 0, 8, 1, 4, 5])

    def both():
        return (nv.matvec(x, bq, bsf, alpha, offsets=off, gated=True, out=act),
                nv.matvec(x[:3], bq[1], bsf[1], alpha[1, :1], out=one))

    act = torch.empty((M, N // 2), dtype=torch.bfloat16, device="cuda")
    one = torch.empty((3, N), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed, counts in ((2, [3, 0, 8, 1, 4, 5]), (3, [0, 20, 0, 0, 1, 0]), (4, [24, 0, 0, 0, 0, 0])):
        x.copy_(_randn((M, K), 1.0, seed, torch.bfloat16)), off.copy_(_offsets(counts))
        act.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = act.clone(), one.clone()
        act.fill_(7.0)
        both()
        torch.cuda.synchronize()
        assert torch.equal(got[0], act) and torch.equal(got[1], one)


def test_weights_beyond_4_gib(nv):
    """The last of many experts lies behind more than 4 GiB of packed weights."""
    import torch
    K, N, E = 7168, 4096, 320
    bq1, bsf1, w, alpha1 = _weights(nv, 1, K, N, 1)
    shq, shs = nv.packed_shapes(E, K, N)
    bq = torch.zeros(shq, dtype=torch.uint8, device="cuda")
    bsf = torch.zeros(shs, dtype=torch.uint8, device="cuda")
    assert bq.numel() > 1 << 32
    bq[E - 1], bsf[E - 1] = bq1[0], bsf1[0]
    alpha = torch.ones(E, device="cuda")
    alpha[E - 1] = alpha1[0]
    x = _randn((3, K), 1.0, 2, torch.bfloat16)
    counts = [0] * E
    counts[0], counts[E - 1] = 1, 2
    out = nv.matvec(x, bq, bsf, alpha, offsets=_offsets(counts))
    assert bool((out[0] == 0).all())
    check(x[1:], w[0], alpha1, out[1:])


def test_refusals(nv):
    import torch
    bq, bsf, _, alpha = _weights(nv, 2, 64, 48, 1)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    off = _offsets([2, 2])
    bad = [(TypeError, lambda: nv.matvec(x.float(), bq[0], bsf[0], alpha[:1])),
           (TypeError, lambda: nv.matvec(x.cpu(), bq[0], bsf[0], alpha[:1])),
           (ValueError, lambda: nv.matvec(x[:, :48].contiguous(), bq, bsf, alpha)),               # no offsets
           (ValueError, lambda: nv.matvec(x[:, :40].contiguous(), bq[0], bsf[0], alpha[:1])),     # K % 16
           (ValueError, lambda: nv.matvec(torch.zeros((4, 256), dtype=x.dtype, device="cuda"), bq[0], bsf[0],
                                          alpha[:1])),
           (ValueError, lambda: nv.matvec(x[:, ::2], bq[0], bsf[0], alpha[:1])),
           (ValueError, lambda: nv.matvec(x, bq[0], bsf[0], alpha[:1], gated=True)),              # 48 columns
           (ValueError, lambda: nv.matvec(x, bq[0], bsf[0], alpha)),
           (TypeError, lambda: nv.matvec(x, bq[0], bsf[0], alpha.double())),
           (ValueError, lambda: nv.matvec(x, bq, bsf, alpha[:1], offsets=off)),
           (ValueError, lambda: nv.matvec(x, bq, bsf, alpha, offsets=off[:2])),
           (TypeError, lambda: nv.matvec(x, bq, bsf, alpha, offsets=off.long())),
           (ValueError, lambda: nv.matvec(x, bq, bsf[:1], alpha, offsets=off)),
           (ValueError, lambda: nv.matvec(x, bq[0], bsf[0], alpha[:1], out=x)),
           (nv.Nvfp4Error, lambda: nv.matvec(torch.zeros(4 * 64 + 1, dtype=x.dtype, device="cuda")[1:].view(4, 64),
                                             bq[0], bsf[0], alpha[:1]))]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
    assert nv.matvec(x[:0], bq[0], bsf[0], alpha[:1]).shape == (0, 48)


def test_subnormal_values(nv):
    """bf16 rows of subnormal numbers: 2^-133 steps meet weights up to 2688 and an
    alpha of 2^100, so that neither the sums nor the results are subnormal."""
    import torch
    K, N = 272, 48
    bq, bsf, w, _ = _weights(nv, 1, K, N, 9)
    g = torch.Generator().manual_seed(1)
    bits = torch.randint(-127, 128, (4, K), generator=g)
    x = (bits.double() * 2.0 ** -133).to(torch.bfloat16).cuda()
    assert bool((x.double().cpu() == bits.double() * 2.0 ** -133).all())
    alpha = torch.tensor([2.0 ** 100], device="cuda")
    out = nv.matvec(x, bq[0], bsf[0], alpha)
    ref, mag = (x.double() @ w[0]) * 2.0 ** 100, (x.double().abs() @ w[0].abs()) * 2.0 ** 100
    # (a float32 sum that is subnormal on the way is off by 2^-149 an addition)
    tol = 2.0 ** -8 * ref.abs() + ((K + 2) * F32 * mag + K * 2.0 ** -49) * 1.01
    assert bool(((out.double() - ref).abs() <= tol).all())
