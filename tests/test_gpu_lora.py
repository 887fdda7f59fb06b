"""The shared NVFP4 projection with low-rank adapters (nvfp4_gemm_lora) against
its definition in float64.

Tolerance, per element: half a bf16 step of the result (2^-8 relative), the
float32 sums (n terms: n * 2^-24 of the sum of magnitudes) of the projection and
of both adapter products, and the 2^-17 of the shrunk row's two-term bf16 form."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
F32 = 2.0 ** -24
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def make(nv, M, N, K, L, R, seed, ids=None, ranks=None):
    import torch
    g = torch.Generator().manual_seed(seed)

    def normal(shape, std):
        return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()

    x = normal((M, K), 1.5)
    w = normal((1, K, N), 0.02)
    aq, asf, a_gs = nv.quantize(x)
    wq, wsf, b_alpha = nv.quantize_weights(w)
    bq, bsf = nv.prepack_weights(wq, wsf)
    s = dict(x=x, aq=aq, asf=asf, a_gs=a_gs, wq=wq[0], wsf=wsf[0], b_alpha=b_alpha, bq=bq[0], bsf=bsf[0],
             lora_a=normal((L, R, K), K ** -0.5), lora_b=normal((L, N, R), 0.05),
             lora_scale=(torch.rand((L,), generator=g) * 3 - 1).cuda())
    if ids is None:
        ids = torch.randint(-1, L + 1, (M,), generator=g)    # L: no adapter either
    s["adapter_ids"] = torch.as_tensor(ids).to(torch.int32).cuda()
    s["lora_rank"] = None if ranks is None else torch.as_tensor(ranks).to(torch.int32).cuda()
    return s


def run(nv, s, **kw):
    return nv.gemm_lora(s["aq"], s["asf"], s["a_gs"], s["bq"], s["bsf"], s["b_alpha"], s["x"], s["lora_a"],
                        s["lora_b"], s["lora_scale"], s["adapter_ids"], lora_rank=s["lora_rank"], **kw)


def dequant(q, sf, dim):
    """float64 values of packed codes and scales along dimension `dim`."""
    import torch
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), dim + 1)
    v = v.flatten(dim, dim + 1)
    return v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim)


def check(s, out):
    import torch
    M, N = out.shape
    K = s["x"].shape[1]
    L, R = s["lora_a"].shape[:2]
    a, b = dequant(s["aq"], s["asf"], 1), dequant(s["wq"], s["wsf"], 0)
    alpha = s["a_gs"].double() * s["b_alpha"].double()
    ref, mag = alpha * (a @ b), alpha.abs() * (a.abs() @ b.abs())
    err = (K + 4) * F32 * mag
    ids = s["adapter_ids"]
    for i in range(L):
        rows = (ids == i).nonzero()[:, 0]
        if not len(rows):
            continue
        r = R if s["lora_rank"] is None else max(0, min(R, int(s["lora_rank"][i])))
        la, lb, sc = s["lora_a"][i, :r].double(), s["lora_b"][i, :, :r].double(), s["lora_scale"][i].double()
        x = s["x"][rows].double()
        v, vm = sc * (x @ la.t()), sc.abs() * (x.abs() @ la.abs().t())
        ref[rows] += v @ lb.t()
        err[rows] += ((K + 16) * F32 * vm + 2.0 ** -16 * v.abs()) @ lb.abs().t()
        err[rows] += (2 * R + 4) * F32 * (v.abs() @ lb.abs().t())
    tol = HALF * ref.abs() + err * (1 + HALF) + 4 * F32 * ref.abs() + 1e-37
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


# single rows; every row count around the 16-, 64-, 128- and 256-row tiles;
# K tails (multiples of 16 only); ranks that end inside a 16-rank block and go
# past a 64-rank one; one adapter and more adapters than rows
@pytest.mark.parametrize("M,N,K,L,R", [
    (1, 16, 16, 1, 8), (1, 6144, 7168, 8, 16), (2, 48, 144, 3, 24), (5, 272, 208, 40, 8), (13, 1024, 2048, 16, 64),
    (16, 512, 1040, 4, 16), (17, 256, 512, 17, 32), (33, 784, 272, 5, 72), (61, 1536, 1024, 32, 32),
    (64, 512, 4096, 64, 128), (65, 528, 512, 65, 16), (128, 512, 256, 3, 256), (129, 1040, 528, 9, 40),
    (256, 768, 640, 6, 16), (300, 512, 256, 20, 64), (513, 6144, 512, 2, 16), (1300, 6144, 144, 7, 136),
    (4093, 4096, 128, 300, 8), (31, 1040, 2064, 9, 24), (32, 16, 7168, 2, 256), (8, 528, 144, 8, 64),
    (16, 1296, 12304, 3, 8), (700, 1024, 2048, 48, 32), (5000, 256, 128, 8192, 8),
    # narrow projections of several 64-row parts, and the widths beyond which
    # such batches are tiled instead
    (512, 2048, 528, 4, 16), (449, 2064, 272, 12, 24), (200, 16, 16, 5, 8), (128, 8192, 272, 4, 16), (128, 8224, 272, 4, 16),
    (65, 8224, 272, 65, 16), (129, 5488, 528, 9, 40), (255, 4112, 640, 6, 256), (300, 3296, 512, 20, 64),
    # many adapters of high rank: tiled although narrow
    (256, 512, 2048, 48, 128), (512, 272, 4096, 64, 64), (70, 528, 7168, 80, 80),
    # a few rows in one launch, and just too much for it
    (3, 1040, 2064, 5, 16), (4, 8192, 1040, 6, 24), (4, 4112, 4096, 3, 8), (1, 8192, 16368, 2, 8), (1, 4112, 512, 2, 256),
    (1, 48, 1024, 4, 128), (2, 272, 1024, 4, 64), (1, 8208, 1040, 2, 16), (2, 6144, 7168, 3, 16), (1, 80, 16400, 2, 8), (1, 272, 16400, 2, 16),
    (4, 272, 1024, 4, 40), (3, 528, 2048, 2, 40), (4, 528, 2048, 2, 32), (1, 272, 32752, 1, 8)])
def test_random_ids(nv, M, N, K, L, R):
    import torch
    s = make(nv, M, N, K, L, R, M + N + K + L + R)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    run(nv, s, out=out)
    check(s, out)
    assert torch.equal(run(nv, s), out)


@pytest.mark.parametrize("M,N", [(2, 528), (7, 528), (64, 528), (200, 528), (200, 4144), (1500, 528)])
def test_runs_of_rows(nv, M, N):
    """Requests as runs of rows, some without an adapter; ranks of their own,
    0 and beyond R among them."""
    import torch
    L, R = 6, 48
    cuts = sorted(set([0, M] + [int(M * f) for f in (0.1, 0.33, 0.34, 0.7, 0.95)]))
    ids = torch.full((M,), -1)
    for n, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
        ids[a:b] = (n * 5) % (L + 1) - 1
    s = make(nv, M, N, 1040, L, R, M, ids=ids, ranks=[48, 0, 7, 33, 100, -3])
    check(s, run(nv, s))


@pytest.mark.parametrize("M,N", [(3, 256), (40, 256), (300, 256), (100, 8224), (600, 256)])
def test_no_row_has_an_adapter(nv, M, N):
    """Only the shared projection: what nvfp4_gemm gives up to summation order."""
    import torch
    s = make(nv, M, N, 512, 4, 16, M, ids=torch.tensor([-1, 4, 2 ** 30, -2 ** 31]).repeat(M)[:M])
    check(s, run(nv, s))


@pytest.mark.parametrize("M,N", [(4, 272), (9, 272), (64, 272), (100, 272), (100, 8224), (700, 272)])
def test_broken_requests_stay_alone(nv, M, N):
    """NaN and infinity in one request's adapter, and in what is stored beyond
    the ranks, reach no other row."""
    import torch
    L, R, K = 5, 24, 528
    s = make(nv, M, N, K, L, R, 3 * M, ids=torch.arange(M) % (L + 1) - 1, ranks=[24, 9, 16, 24, 1])
    out = run(nv, s).clone()
    check(s, out)
    for a, r in enumerate([24, 9, 16, 24, 1]):
        s["lora_a"][a, r:] = float("nan")
        s["lora_b"][a, :, r:] = float("inf")
    assert torch.equal(run(nv, s), out)
    s["lora_a"][3, 5], s["lora_b"][3, ::3] = float("inf"), float("nan")
    s["x"][1] = float("nan")                          # aq stays: only the adapter's input is broken
    keep = (s["adapter_ids"] != 3) & (torch.arange(M, device="cuda") != 1)
    again = run(nv, s)
    assert torch.equal(again[keep], out[keep])
    assert bool(again[s["adapter_ids"] == 3][:, ::3].isnan().all())


@pytest.mark.parametrize("M,N", [(4, 272), (9, 272), (64, 272), (100, 272), (100, 8224), (700, 272)])
def test_shrunk_rows_that_overflow_stay_infinite(nv, M, N):
    """v = scale * x A^T beyond float32: the sum with B of one sign is that
    infinity, in rows of the adapter alone."""
    import torch
    K = 528
    s = make(nv, M, N, K, 3, 8, M + 1, ids=torch.arange(M) % 4 - 1)
    out = run(nv, s).clone()
    check(s, out)
    s["lora_a"][1] = s["x"][(s["adapter_ids"] == 1).nonzero()[0, 0]].sign()     # a positive sum in that row
    s["lora_scale"][1] = 3e38
    s["lora_b"][1] = s["lora_b"][1].abs() + 0.01
    s["lora_b"][1, ::2] *= -1
    again = run(nv, s)
    rows = s["adapter_ids"] == 1
    assert torch.equal(again[~rows], out[~rows])
    row = again[rows][0].float()
    assert bool((row[1::2] == float("inf")).all()) and bool((row[::2] == float("-inf")).all())


@pytest.mark.parametrize("M", [33, 47, 48, 49])
def test_row_blocks_of_a_partly_filled_tile(nv, M):
    """Three of four 16-row blocks in use; a workspace of exactly the needed
    size, bytes of NaN patterns before every run."""
    import torch
    N, K, L, R = 160, 1040, 4, 16
    s = make(nv, M, N, K, L, R, M)
    ws = torch.full((nv._lib.nvfp4_gemm_lora_workspace(M, N, K, L, R),), 0xFF, dtype=torch.uint8, device="cuda")
    check(s, run(nv, s, workspace=ws))


def test_a_request_does_not_depend_on_its_batch_mates_ids(nv):
    """The same rows beside other ids: rows whose id did not change keep their
    bits."""
    import torch
    s = make(nv, 50, 256, 1024, 8, 16, 4)
    out = run(nv, s).clone()
    ids = s["adapter_ids"].clone()
    ids[10:30] = torch.flip(ids[10:30], (0,))
    same = ids == s["adapter_ids"]
    s["adapter_ids"] = ids
    assert torch.equal(run(nv, s)[same], out[same])


@pytest.mark.parametrize("M,N", [(1, 512), (20, 512), (150, 512), (150, 5488), (600, 512)])
def test_streams_and_graph(nv, M, N):
    import torch
    K, L, R = 1024, 4, 16
    s = make(nv, M, N, K, L, R, 5)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty((nv._lib.nvfp4_gemm_lora_workspace(M, N, K, L, R),), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(nv, s)
    torch.cuda.current_stream().wait_stream(side)
    check(s, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(nv, s, out=out, workspace=ws)
    for seed in (6, 7, 8):
        t = make(nv, M, N, K, L, R, seed)
        for k in ("x", "aq", "asf", "a_gs", "bq", "bsf", "b_alpha", "lora_a", "lora_b", "lora_scale", "adapter_ids"):
            s[k].copy_(t[k])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(t, out)
        assert torch.equal(run(nv, t), out)


@pytest.mark.parametrize("M,N,K,L,R", [(1, 16, 16, 1, 8), (50, 272, 528, 6, 72), (100, 528, 1040, 6, 24), (100, 8224, 272, 6, 24),
                                       (600, 784, 272, 9, 136), (2100, 4112, 144, 5, 16)])
def test_nothing_beside_the_output_is_written(nv, M, N, K, L, R):
    """The output and a workspace of exactly the asked size inside larger
    buffers: what lies before and behind them stays, and what the workspace
    held does not matter."""
    import torch
    s = make(nv, M, N, K, L, R, 17)
    guard = 4096
    n_ws = nv._lib.nvfp4_gemm_lora_workspace(M, N, K, L, R)
    for fill in (0x5A, 0xFF):                       # 0xFF: NaN in every float type
        out = torch.full((2 * M * N + 2 * guard,), fill, dtype=torch.uint8, device="cuda")
        ws = torch.full((n_ws + 2 * guard,), fill, dtype=torch.uint8, device="cuda")
        y = out[guard:-guard].view(torch.bfloat16).view(M, N)
        run(nv, s, out=y, workspace=ws[guard:-guard])
        check(s, y)
        for buf in (out, ws):
            assert bool((buf[:guard] == fill).all()) and bool((buf[-guard:] == fill).all())


@pytest.mark.parametrize("M", [1, 30, 64, 200, 900])
def test_one_adapter_and_every_row_its_own(nv, M):
    """The two ends: one adapter for all rows, and as many adapters as rows."""
    import torch
    for L, ids in ((1, torch.zeros(M)), (M, torch.randperm(M, generator=torch.Generator().manual_seed(M)))):
        s = make(nv, M, 272, 272, L, 16, M + L, ids=ids)
        check(s, run(nv, s))


def test_two_streams_at_once(nv):
    """Calls in flight together on two streams, each with its own workspace: one
    that streams the weights, one tiled."""
    import torch
    sets = [make(nv, 40, 512, 2048, 6, 32, 51), make(nv, 600, 512, 1024, 4, 16, 52)]
    alone = [run(nv, s).clone() for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                out[k].append(run(nv, sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, alone[k]) for o in out[k])


def test_refusals(nv):
    import torch
    s = make(nv, 4, 32, 64, 2, 8, 1)

    def bad(exc, **kw):
        t = dict(s)
        t.update(kw)
        with pytest.raises(exc):
            run(nv, t)

    bad(TypeError, x=s["x"].float())
    bad(TypeError, lora_a=s["lora_a"].half())
    bad(TypeError, adapter_ids=s["adapter_ids"].long())
    bad(TypeError, lora_scale=s["lora_scale"].cpu())
    bad(ValueError, lora_a=s["lora_a"].transpose(1, 2))
    bad(ValueError, lora_a=s["lora_a"][:, :, :48].contiguous())
    bad(ValueError, lora_a=s["lora_a"][:, :4].contiguous(), lora_b=s["lora_b"][:, :, :4].contiguous())   # R % 8
    bad(ValueError, adapter_ids=s["adapter_ids"][:3].contiguous())
    bad(ValueError, lora_rank=torch.ones((3,), dtype=torch.int32, device="cuda"))
    bad(ValueError, lora_a=s["lora_a"][:0], lora_b=s["lora_b"][:0], lora_scale=s["lora_scale"][:0])
    with pytest.raises(nv.Nvfp4Error):
        run(nv, s, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        run(nv, s, out=torch.empty((4, 48), dtype=torch.bfloat16, device="cuda"))


def test_empty_batch(nv):
    s = make(nv, 4, 32, 64, 2, 8, 1)
    for k in ("x", "aq", "asf", "adapter_ids"):
        s[k] = s[k][:0]
    assert run(nv, s).shape == (0, 32)


@pytest.mark.parametrize("T", [1, 37, 300])
def test_feed_forward_with_adapters(nv, T):
    """The dense feed-forward as it is used: the gated block in bf16, its
    output quantized, the shared NVFP4 down projection with each request's
    adapter, beside the routed experts' own entry points on one stream."""
    import torch
    H, I, L, R = 512, 256, 4, 16
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    w13 = (torch.randn((H, 2 * I), generator=g) * 0.05).to(torch.bfloat16).cuda()
    s = make(nv, T, H, I, L, R, T + 9)
    act = nv.gated_forward(x, w13)
    s["x"] = act
    s["aq"], s["asf"], s["a_gs"] = nv.quantize(act)
    y = run(nv, s)
    check(s, y)
    gu = x.double() @ w13.double()
    ref = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    assert float((act.double() - ref).norm() / ref.norm()) < HALF


def check_rows(s, out, rows):
    """check on some rows of a result."""
    check({**s, "x": s["x"][rows], "aq": s["aq"][rows], "asf": s["asf"][rows], "adapter_ids": s["adapter_ids"][rows]},
          out[rows])


def test_outputs_beyond_32_bits(nv):
    """More than 4 GiB of output: rows of both ends and beside the 4 GiB border."""
    import torch
    M, N, K, L, R = 131100, 16416, 64, 3, 8
    s = make(nv, M, N, K, L, R, 9)
    out = run(nv, s)
    border = 2 ** 31 // N
    check_rows(s, out, torch.tensor([0, 1, border, border + 1, M // 2, M - 2, M - 1], device="cuda"))


@pytest.mark.parametrize("M", [2, 40, 70, 300])
def test_adapters_beyond_32_bits(nv, M):
    """Adapters stored in more than 4 GiB, the last ones in use."""
    import torch
    N, K, L, R = 16384, 64, 600, 256
    s = make(nv, M, N, K, 1, 8, M)
    g = torch.Generator("cuda").manual_seed(M)
    s["lora_b"] = torch.randn((L, N, R), generator=g, device="cuda", dtype=torch.bfloat16)
    s["lora_a"] = torch.randn((L, R, K), generator=g, device="cuda", dtype=torch.bfloat16)
    s["lora_scale"] = torch.rand((L,), generator=g, device="cuda") * 0.1
    s["adapter_ids"] = (L - 1 - 5 * (torch.arange(M, device="cuda") % 7)).to(torch.int32)
    check(s, run(nv, s))
