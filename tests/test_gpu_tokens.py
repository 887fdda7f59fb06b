"""Tokens sorted by expert and back, their gradients and the router's gradient,
against the definitions: integers and moved rows exactly, sums in float64.

Tolerances, element by element. A result is one rounding (half a step of its type)
of a float32 value; a float32 sum of n terms is off by at most n * 2^-24 of the sum
of magnitudes, each product by 2^-24 of itself; and half the type's smallest number
near zero."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
DTYPES = ("bfloat16", "float16", "float32")


def _half(dtype):
    """Half a step relative to the value, and half the smallest number."""
    import torch
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def _randn(shape, std, seed, dtype):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _ids(T, E, k, seed, routed=None, repeat=False):
    """Distinct experts of each token out of `routed` (repeat: drawn one by one,
    so that a token may have an expert twice, and negative ids too)."""
    g = np.random.RandomState(seed)
    if repeat:
        return g.randint(-2, (routed or E) + 2, (T, k)).astype(np.int32)
    return np.argsort(g.rand(T, routed or E), 1)[:, :k].astype(np.int32)


def _order(ids, E):
    """offsets, slot_row, slots by row: the definition, slot by slot."""
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    row = np.full(flat.shape, -1, np.int32)
    row[slots] = np.arange(len(slots), dtype=np.int32)
    return offsets, row.reshape(ids.shape), np.array(slots, np.int64)


# (T, H, E, k, routed experts, ids drawn with repetition)
SIZES = [(1, 16, 1, 1, 1, False), (1, 7168, 48, 8, 48, False), (3, 1, 4, 2, 4, False), (7, 33, 2, 1, 5, False),
         (8, 7168, 48, 8, 48, False), (33, 257, 5, 9, 11, True), (64, 8, 512, 8, 512, False),
         (130, 2049, 33, 6, 33, False), (511, 48, 3, 8, 16, False), (513, 130, 64, 8, 64, False),
         (1000, 264, 7, 3, 7, True), (4100, 96, 256, 8, 256, False), (20011, 24, 16, 5, 48, False)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,E,k,routed,repeat", SIZES)
def test_sort_and_its_gradient(nv, T, H, E, k, routed, repeat, dtype):
    import torch
    dtype = getattr(torch, dtype)
    ids = _ids(T, E, k, T + H, routed, repeat)
    offsets, slot_row, slots = _order(ids, E)
    x = _randn((T, H), 1.5, T, dtype)
    rows = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    got, off, row = nv.sort_tokens(x, torch.from_numpy(ids).cuda(), E, rows=rows)
    assert got is rows
    assert (off.cpu().numpy() == offsets).all() and (row.cpu().numpy() == slot_row).all()
    n = len(slots)
    token = torch.from_numpy(slots // k).cuda()
    assert torch.equal(rows[:n], x[token])
    assert bool(rows[n:].isnan().all())                       # left as they were
    d_rows = _randn((T * k, H), 0.3, T + 1, dtype)
    d_rows[n:] = float("nan")                                 # no slot's
    dx = nv.sort_tokens_backward(d_rows, row)
    d = d_rows[:n].double()
    zero = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    ref, mag = zero.index_add(0, token, d), zero.index_add(0, token, d.abs())
    half, tiny = _half(dtype)
    assert dx.dtype == dtype
    assert bool(((dx.double() - ref).abs() <= half * ref.abs() + k * F32 * mag * (1 + half) + tiny).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,E,k,routed,repeat", SIZES)
def test_unsort_and_its_gradients(nv, T, H, E, k, routed, repeat, dtype):
    import torch
    dtype = getattr(torch, dtype)
    ids = _ids(T, E, k, T + H + 7, routed, repeat)
    _, slot_row, slots = _order(ids, E)
    n = len(slots)
    rows = _randn((T * k, H), 0.7, T, dtype)
    rows[n:] = float("nan")
    w = _randn((T, k), 1.0, T + 1, torch.float32)
    dy = _randn((T, H), 0.5, T + 2, dtype)
    row = torch.from_numpy(slot_row).cuda()
    slot = torch.from_numpy(slots).cuda()
    token = slot // k
    wr = w.double().view(-1)[slot]
    half, tiny = _half(dtype)

    y = nv.unsort_tokens(rows, row, w)
    terms = rows[:n].double() * wr[:, None]
    zero = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    ref, mag = zero.index_add(0, token, terms), zero.index_add(0, token, terms.abs())
    assert y.dtype == dtype
    assert bool(((y.double() - ref).abs() <= half * ref.abs() + (k + 1) * F32 * mag * (1 + half) + tiny).all())

    d_rows = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    d_weights = torch.full((T, k), float("nan"), device="cuda")
    nv.unsort_tokens_backward(dy, rows, row, w, d_rows=d_rows, d_weights=d_weights)
    ref = dy.double()[token] * wr[:, None]
    assert bool(((d_rows[:n].double() - ref).abs() <= (half + 2 * F32) * ref.abs() + tiny).all())
    assert bool(d_rows[n:].isnan().all())
    prod = dy.double()[token] * rows[:n].double()
    ref, mag = torch.zeros((2, T * k), dtype=torch.float64, device="cuda")
    ref[slot], mag[slot] = prod.sum(1), prod.abs().sum(1)
    err = (d_weights.double().view(-1) - ref).abs()
    assert bool((err <= (H + 1) * F32 * mag + 2.0 ** -149).all())
    assert bool((d_weights.view(-1)[(row < 0).view(-1)] == 0).all())
    # one of them alone: the same bits
    a, none = nv.unsort_tokens_backward(dy, rows, row, w, need_d_weights=False)
    assert none is None and torch.equal(a[:n], d_rows[:n])
    none, b = nv.unsort_tokens_backward(dy, rows, row, w, need_d_rows=False)
    assert none is None and torch.equal(b, d_weights)


def test_slots_without_a_row_and_entries_out_of_range(nv):
    """Entries of slot_row outside [0, R) contribute nothing, whatever their weight;
    tokens without any row give zeros."""
    import torch
    T, H, k, R = 6, 40, 3, 10
    row = torch.tensor([[0, -1, 9], [-1, -1, -1], [10, 3, -7], [1 << 30, -(1 << 31), 4], [5, 6, 7], [8, 2, 1]],
                       dtype=torch.int32).cuda()
    ok = (row >= 0) & (row < R)
    rows, dy = _randn((R, H), 1.0, 1, torch.bfloat16), _randn((T, H), 1.0, 2, torch.bfloat16)
    w = torch.where(ok, _randn((T, k), 1.0, 3, torch.float32), torch.full((), float("nan"), device="cuda"))
    clean = torch.where(ok, row, torch.full((), -1, dtype=torch.int32, device="cuda"))
    y = nv.unsort_tokens(rows, row, w)
    assert bool((y[1] == 0).all()) and bool(y.isfinite().all())
    assert torch.equal(y, nv.unsort_tokens(rows, clean, w.nan_to_num(0.0)))
    dx = nv.sort_tokens_backward(rows, row)
    assert torch.equal(dx, nv.sort_tokens_backward(rows, clean)) and bool((dx[1] == 0).all())
    d_rows = torch.zeros_like(rows)
    _, dw = nv.unsort_tokens_backward(dy, rows, row, w, d_rows=d_rows)
    assert bool((dw[~ok] == 0).all()) and bool(d_rows.isfinite().all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_non_finite_values_stay_where_they_are(nv, dtype):
    import torch
    dtype = getattr(torch, dtype)
    T, H, E, k = 40, 77, 6, 3
    ids = torch.from_numpy(_ids(T, E, k, 5)).cuda()
    x = _randn((T, H), 1.0, 1, dtype)
    x[7], x[8, ::2] = float("inf"), float("nan")
    rows, _, row = nv.sort_tokens(x, ids, E)
    back = nv.sort_tokens_backward(rows, row)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7:9] = False
    assert bool(back[keep].isfinite().all()) and bool((back[7] == float("inf")).all())
    assert bool(back[8, ::2].isnan().all()) and bool(back[8, 1::2].isfinite().all())
    w = torch.ones((T, k), device="cuda")
    w[7, 0] = 0.0                                             # zero times infinity is NaN
    y = nv.unsort_tokens(rows, row, w)
    assert bool(y[keep].isfinite().all()) and bool(y[7].isnan().all())
    d_rows, dw = nv.unsort_tokens_backward(x, rows, row, w)
    assert bool(dw[keep].isfinite().all()) and bool((dw[7] == float("inf")).all()) and bool(dw[8].isnan().all())
    assert bool(d_rows[row[keep].long()].isfinite().all())


def test_results_beyond_the_types_range(nv):
    """A float32 sum beyond float16's range rounds to infinity, and one that comes
    back into it does not."""
    import torch
    rows = torch.tensor([[60000.0], [60000.0], [-60000.0]], dtype=torch.float16).cuda()
    row = torch.tensor([[0, 1, -1], [0, 1, 2]], dtype=torch.int32).cuda()
    dx = nv.sort_tokens_backward(rows, row)
    assert dx[0].item() == float("inf") and dx[1].item() == 60000.0


def test_no_tokens(nv):
    import torch
    x = torch.zeros((0, 48), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    rows, offsets, row = nv.sort_tokens(x, ids, 5)
    assert rows.shape == (0, 48) and row.shape == (0, 2) and bool((offsets == 0).all()) and offsets.shape == (6,)
    w = torch.zeros((0, 2), device="cuda")
    assert nv.unsort_tokens(rows, row, w).shape == (0, 48) and nv.sort_tokens_backward(rows, row).shape == (0, 48)
    d_rows, dw = nv.unsort_tokens_backward(x, rows, row, w)
    assert d_rows.shape == (0, 48) and dw.shape == (0, 2)
    assert nv.route_topk_backward(w, ids, w, 5).shape == (0, 5)
    # tokens, but no rows: all experts are elsewhere
    row = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    y = nv.unsort_tokens(rows, row, torch.ones((3, 2), device="cuda"))
    assert y.shape == (3, 48) and bool((y == 0).all())


def test_nothing_beside_the_outputs_is_written(nv):
    import torch
    T, E, k = 37, 9, 4
    ids = torch.from_numpy(_ids(T, E, k, 3)).cuda()
    for H in (5, 64, 1001):
        bufs = []

        def inside(*shape):
            n = int(np.prod(shape))
            buf = torch.full((n + 2 * 63,), 7.0, dtype=torch.bfloat16, device="cuda")
            bufs.append((buf, n))
            return buf[63:63 + n].view(shape)                 # at an odd element

        x = inside(T, H)
        x.copy_(_randn((T, H), 1.0, H, torch.bfloat16))
        rows, dx, y, d_rows = inside(T * k, H), inside(T, H), inside(T, H), inside(T * k, H)
        _, _, row = nv.sort_tokens(x, ids, E, rows=rows)
        w = torch.ones((T, k), device="cuda")
        nv.sort_tokens_backward(rows, row, dx=dx)
        nv.unsort_tokens(rows, row, w, y=y)
        nv.unsort_tokens_backward(x, rows, row, w, d_rows=d_rows)
        assert torch.equal(dx, y) and torch.equal(d_rows, rows)
        for buf, n in bufs:
            assert bool((buf[:63] == 7).all()) and bool((buf[63 + n:] == 7).all())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 4, 4), (33, 48, 8), (1000, 7, 3), (4097, 256, 8), (70, 512, 512),
                                   (65539, 33, 6)])
def test_router_gradient(nv, T, E, k):
    import torch
    logits = _randn((T, E), 1.0, T + E, torch.float32)
    ids, w = nv.route_topk(logits, k)
    dw = _randn((T, k), 0.5, T, torch.float32)
    got = nv.route_topk_backward(dw, ids, w, E)
    # by automatic differentiation, at the given weights
    z = torch.log(w.double()).requires_grad_(True)
    torch.softmax(z, 1).backward(dw.double())
    ref = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), z.grad)
    # s is off by k + 1 roundings of sum |w dw|; the weights sum to one within k * 2^-24, which
    # normalizing them again (the reference does) moves every term by
    wd, dd = w.double(), dw.double()
    slack = wd * ((3 * k + 6) * F32 * ((wd * dd).abs().sum(1, keepdim=True) + dd.abs()))
    tol = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), slack)
    assert bool(((got.double() - ref).abs() <= tol + 2.0 ** -148).all())


def test_router_gradient_of_repeated_and_foreign_ids(nv):
    """An expert that a token names twice has the sum; ids outside [0, E) name no
    logit and count in the inner sum."""
    import torch
    T, E, k = 50, 6, 5
    ids = torch.from_numpy(_ids(T, E, k, 9, repeat=True)).cuda()
    w, dw = _randn((T, k), 1.0, 1, torch.float32), _randn((T, k), 1.0, 2, torch.float32)
    got = nv.route_topk_backward(dw, ids, w, E)
    wd, dd = w.double(), dw.double()
    v = wd * (dd - (wd * dd).sum(1, keepdim=True))
    ref = torch.stack([torch.where(ids == e, v, torch.zeros((), dtype=torch.float64, device="cuda")).sum(1)
                       for e in range(E)], 1)
    tol = (3 * k + 6) * F32 * (wd.abs() * ((wd * dd).abs().sum(1, keepdim=True) + dd.abs())).sum(1, keepdim=True)
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("T,E", [(700, 16), (1000, 16), (4000, 200)])     # each way to rank the slots
def test_streams_and_graph(nv, T, E):
    """A captured run replays into the same bits on new values, beside eager calls;
    calls in flight on two streams do not meet."""
    import torch
    H, k = 264, 8
    dtype = torch.bfloat16
    x, dy = _randn((T, H), 1.0, 1, dtype), _randn((T, H), 1.0, 2, dtype)
    logits, w = _randn((T, E), 1.0, 3, torch.float32), torch.empty((T, k), device="cuda")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")

    def step():
        nv.route_topk(logits, k, ids=ids, weights=w)
        rows, offsets, row = nv.sort_tokens(x, ids, E)
        y = nv.unsort_tokens(rows, row, w)
        d_rows, dw = nv.unsort_tokens_backward(dy, rows, row, w)
        return rows, offsets, row, y, d_rows, dw, nv.sort_tokens_backward(d_rows, row), nv.route_topk_backward(
            dw, ids, w, E)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (11, 12, 13):
        x.copy_(_randn((T, H), 1.0, seed, dtype)), dy.copy_(_randn((T, H), 1.0, seed + 50, dtype))
        logits.copy_(_randn((T, E), 1.0, seed + 90, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    many = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                many[i].append(nv.sort_tokens(x if i else dy, ids, E))
    torch.cuda.synchronize()
    for i in range(2):
        for rows, offsets, row in many[i]:
            assert torch.equal(row, eager[2]) and torch.equal(rows, (x if i else dy)[torch.argsort(row.view(-1)) // k])


def test_offsets_beyond_32_bits(nv):
    """Rows of more than 8 GiB in all: those of both ends."""
    import torch
    T, H, E, k = 70001, 7168, 4, 8
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)     # every expert twice
    rows, offsets, row = nv.sort_tokens(x, ids, E)
    assert offsets.tolist() == [T * 2 * e for e in range(E + 1)]
    t = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    for j in range(k):
        assert torch.equal(rows[row[t, j].long()], x[t])
    w = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(nv.unsort_tokens(rows, row, w)[t], x[t])
    assert torch.equal(nv.sort_tokens_backward(rows, row)[t], x[t] * 8)
    d_rows, dw = nv.unsort_tokens_backward(x, rows, row, w)
    assert torch.equal(d_rows[row[t, 7].long()], x[t] * 0.125)
    ref = (x[t].double() ** 2).sum(1)
    assert bool(((dw[t].double() - ref[:, None]).abs() <= H * F32 * ref[:, None]).all())


def test_refusals(nv):
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    x, ids, w = torch.zeros((4, 32), **bf), torch.zeros((4, 2), **i32), torch.zeros((4, 2), device="cuda")
    rows, row = torch.zeros((8, 32), **bf), torch.zeros((4, 2), **i32)
    bad = [(TypeError, lambda: nv.sort_tokens(x.double(), ids, 3)),
           (TypeError, lambda: nv.sort_tokens(x.cpu(), ids, 3)),
           (TypeError, lambda: nv.sort_tokens(x, ids.long(), 3)),
           (ValueError, lambda: nv.sort_tokens(x.t(), ids, 3)),
           (ValueError, lambda: nv.sort_tokens(x[:3], ids, 3)),
           (ValueError, lambda: nv.sort_tokens(x, ids.view(-1), 3)),
           (ValueError, lambda: nv.sort_tokens(x, ids, 3, rows=rows[:7])),
           (nv.Nvfp4Error, lambda: nv.sort_tokens(x, ids, 0)),
           (nv.Nvfp4Error, lambda: nv.sort_tokens(x, ids, 513)),
           (nv.Nvfp4Error, lambda: nv.sort_tokens(x.repeat(4096, 1), ids.repeat(4096, 1), 3,
                                                  workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
           (ValueError, lambda: nv.sort_tokens_backward(rows, row[:, :0])),
           (TypeError, lambda: nv.sort_tokens_backward(rows, row.float())),
           (ValueError, lambda: nv.sort_tokens_backward(rows, row, dx=x[:2])),
           (TypeError, lambda: nv.unsort_tokens(rows, row, w.double())),
           (ValueError, lambda: nv.unsort_tokens(rows, row, w[:, :1])),
           (TypeError, lambda: nv.unsort_tokens_backward(x, rows.float(), row, w)),
           (ValueError, lambda: nv.unsort_tokens_backward(x[:2], rows, row, w)),
           (ValueError, lambda: nv.unsort_tokens_backward(x, rows, row, w, need_d_rows=False, need_d_weights=False)),
           (ValueError, lambda: nv.unsort_tokens_backward(x, rows, row, w, d_rows=rows, need_d_rows=False)),
           (TypeError, lambda: nv.route_topk_backward(w.double(), ids, w, 3)),
           (ValueError, lambda: nv.route_topk_backward(w, ids[:2], w, 3)),
           (nv.Nvfp4Error, lambda: nv.route_topk_backward(w, ids, w, 1))]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
