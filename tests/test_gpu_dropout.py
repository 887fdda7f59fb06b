"""Dropout against its definition: the mask bit for bit from Philox4x32 in NumPy,
values in float64. Tolerance: scale, product and sum are float32 roundings (2^-24
of the value each), then one rounding to the type."""
import numpy as np
import pytest

F32 = 2.0 ** -24
DTYPES = ("bfloat16", "float16", "float32")


def philox(counter, key, rounds=7):
    """Words (n, 4) of the 128-bit counters (n, 4) under a 64-bit key, all uint32."""
    c, k = [counter[:, i].astype(np.uint64) for i in range(4)], [int(v) for v in key]
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> up) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> up) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def kept(n, p, seed, offset):
    at = (offset + np.arange((n + 3) // 4, dtype=object)) % (1 << 64)
    counter = np.array([[int(v) & 0xFFFFFFFF, int(v) >> 32, 0, 0] for v in at], np.uint64).reshape(-1, 4)
    word = philox(counter, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n].astype(np.float64)
    return word >= np.floor(p * 2.0 ** 32 + 0.5)


def test_generator_known_answers():
    """Published known answers of Philox4x32 in ten rounds."""
    zero, ones = np.zeros((1, 4), np.uint32), np.full((1, 4), 0xFFFFFFFF, np.uint32)
    assert philox(zero, (0, 0), 10).tolist() == [[0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]]
    assert philox(ones, (0xFFFFFFFF, 0xFFFFFFFF), 10).tolist() == [[0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]]


def _rng(seed, offset):
    import torch
    wrap = [v - (1 << 64) if v >= 1 << 63 else v for v in (seed, offset)]
    return torch.tensor(wrap, dtype=torch.int64).cuda()


def _randn(shape, std, seed, dtype):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def check(x, y, p, keep, residual=None):
    import torch
    f = torch.finfo(x.dtype)
    scaled = torch.where(keep, x.double() / (1 - p) if p < 1 else x.double() * 0, torch.zeros((), dtype=torch.float64, device="cuda"))
    ref = scaled if residual is None else scaled + residual.double()
    tol = f.eps / 2 * ref.abs() + (2 * F32 * scaled.abs() + F32 * ref.abs()) * (1 + f.eps) + f.smallest_normal * f.eps / 2
    assert bool(((y.double() - ref).abs() <= tol).all())
    if residual is None:
        assert bool((y[~keep] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,p,seed,offset", [
    ((1,), 0.5, 0, 0), ((3,), 0.25, 7, 5), ((7, 1), 0.1, 1 << 63, 1 << 40), ((1000,), 0.999, 123, (1 << 32) - 100),
    ((33, 257), 0.0, 5, 0), ((33, 257), 1.0, 5, 0), ((301, 2049), 0.25, (1 << 64) - 1, (1 << 64) - 17),
    ((129, 7168), 0.1, 0x0123456789ABCDEF, 99)])
def test_dropout(nv, shape, p, seed, offset, dtype):
    import torch
    dtype = getattr(torch, dtype)
    n = int(np.prod(shape))
    keep = torch.from_numpy(kept(n, p, seed, offset)).cuda().view(shape)
    x, res, rng = _randn(shape, 1.0, n, dtype), _randn(shape, 2.0, n + 1, dtype), _rng(seed, offset)
    y = nv.dropout(x, p, rng)
    assert y.dtype == dtype and y.shape == x.shape
    check(x, y, p, keep)
    check(x, nv.dropout(x, p, rng, residual=res), p, keep, res)
    assert torch.equal(nv.dropout_backward(x, p, rng), y)     # the same linear function
    if p == 0.0:
        assert torch.equal(y, x)


@pytest.mark.gpu
def test_gradient_matches_differences(nv):
    """The function is linear: the difference quotient of sum(y * dy) in an entry
    of x is kept / (1 - p) * dy up to the roundings of y."""
    import torch
    p, rng, h = 0.3, _rng(3, 4), 0.5
    x, dy = _randn((64,), 1.0, 1, torch.float32), _randn((64,), 1.0, 2, torch.float32)
    dx = nv.dropout_backward(dy, p, rng)
    for i in range(0, 64, 5):
        up, down = x.clone(), x.clone()
        up[i] += h
        down[i] -= h
        d = (nv.dropout(up, p, rng).double() - nv.dropout(down, p, rng).double()) @ dy.double()
        width = (up[i] - down[i]).double()
        assert abs(float(d / width - dx[i])) <= 16 * F32 * (abs(float(up[i])) + abs(float(down[i])) + 1) * abs(float(dy[i]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_mask_goes_by_the_element_alone(nv, dtype):
    """Any type and alignment, parts of a tensor with their own offset, in place."""
    import torch
    dtype = getattr(torch, dtype)
    n, p, rng = 4003, 0.4, _rng(11, 1000)
    x = torch.ones(n, dtype=dtype, device="cuda")
    y = nv.dropout(x, p, rng)
    assert torch.equal(y != 0, nv.dropout(torch.ones(n, device="cuda"), p, rng) != 0)
    assert torch.equal(nv.dropout(x[2000:], p, _rng(11, 1500)), y[2000:])
    for shift in (1, 3):
        buf = torch.full((n + 20,), 5.0, dtype=dtype, device="cuda")
        part = buf[shift:shift + n]
        part.copy_(x)
        assert nv.dropout(part, p, rng, y=part) is part and torch.equal(part, y)
        assert bool((buf[:shift] == 5).all()) and bool((buf[shift + n:] == 5).all())
    res = _randn((n,), 1.0, 1, dtype)
    want = nv.dropout(x, p, rng, residual=res)
    nv.dropout(x, p, rng, residual=res, y=res)
    assert torch.equal(res, want)


@pytest.mark.gpu
def test_what_is_dropped_enters_nothing(nv):
    import torch
    n, p, rng = 512, 0.5, _rng(2, 0)
    keep = torch.from_numpy(kept(n, p, 2, 0)).cuda()
    x = torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[1::2] = float("inf")
    y = nv.dropout(x, p, rng, residual=torch.ones_like(x))
    assert bool((y[~keep] == 1).all()) and not bool(y[keep].isfinite().any())
    # an infinite residual stays, kept or not
    y = nv.dropout(torch.ones_like(x), p, rng, residual=torch.full_like(x, float("-inf")))
    assert bool((y == float("-inf")).all())


@pytest.mark.gpu
def test_rate(nv):
    """The share of kept elements: 2^24 draws, within six standard deviations."""
    import torch
    n = 1 << 24
    for p in (0.1, 0.5, 0.9):
        y = nv.dropout(torch.ones(n, device="cuda"), p, _rng(77, 0))
        share = float((y != 0).double().mean())
        assert abs(share - (1 - p)) <= 6 * (p * (1 - p) / n) ** 0.5


@pytest.mark.gpu
def test_a_captured_call_follows_its_state(nv):
    import torch
    x, rng, p = _randn((33, 65), 1.0, 1, torch.bfloat16), _rng(5, 0), 0.3
    step = (x.numel() + 3) // 4
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.dropout(x, p, rng)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.dropout(x, p, rng)
        rng[1] += step
    assert rng.tolist() == [5, 0]
    seen = []
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        seen.append(y.clone())
        assert torch.equal(y, nv.dropout(x, p, _rng(5, i * step)))
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.gpu
def test_offsets_beyond_32_bits(nv):
    import torch
    n, p = (1 << 32) + 1003, 0.5
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = nv.dropout(x, p, _rng(9, 0))
    for at in (0, (1 << 31) - 4, (1 << 32) - 8, n - 1003):
        m = min(1003, n - at)
        assert torch.equal(y[at:at + m] != 0, torch.from_numpy(kept(m, p, 9, at // 4)).cuda())


@pytest.mark.gpu
def test_refusals(nv):
    import torch
    x, rng = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda"), _rng(1, 2)
    bad = [(TypeError, lambda: nv.dropout(x.double(), 0.5, rng)), (TypeError, lambda: nv.dropout(x.cpu(), 0.5, rng)),
           (ValueError, lambda: nv.dropout(x.t(), 0.5, rng)), (ValueError, lambda: nv.dropout(x, 1.5, rng)),
           (ValueError, lambda: nv.dropout(x, -0.1, rng)), (ValueError, lambda: nv.dropout(x, float("nan"), rng)),
           (TypeError, lambda: nv.dropout(x, 0.5, rng.int())), (ValueError, lambda: nv.dropout(x, 0.5, rng[:1])),
           (TypeError, lambda: nv.dropout(x, 0.5, rng.cpu())), (TypeError, lambda: nv.dropout(x, 0.5, rng, residual=x.float())),
           (ValueError, lambda: nv.dropout(x, 0.5, rng, residual=x[:2])), (ValueError, lambda: nv.dropout(x, 0.5, rng, y=x[:2])),
           (TypeError, lambda: nv.dropout_backward(x.long(), 0.5, rng)),
           (ValueError, lambda: nv.dropout_backward(x, 2.0, rng))]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
    assert nv.dropout(x[:0], 0.5, rng).shape == (0, 8)
