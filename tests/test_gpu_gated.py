"""The gated feed-forward block (nvfp4_gated_forward / _backward) against its
definition in float64.

Tolerances. A bf16 output is one rounding of a float32 result: at most half a
step, 2^-8 relative. The float32 sum of n exact products
carries at most n * 2^-24 * sum |a b|; half the worst case is far above what
random signs give. The gradients' sums take [dgate | dup] rounded to bf16: each
term moves by at most 2^-8 of itself, so the sum by at most 2^-8 * sum |a b|.
Every check is element by element with those sums of magnitudes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8           # half a bf16 step, relative to the value
F32 = 2.0 ** -24


def _rand(shape, std, seed, torch):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def _inputs(T, H, I, seed):
    import torch
    return (_rand((T, H), 1.5, seed, torch), _rand((H, 2 * I), 2.5 / (1.5 * H ** 0.5), seed + 1, torch),
            _rand((T, I), 0.5, seed + 2, torch))


def _sig(g):
    import torch
    return torch.sigmoid(g)


def check_forward(x, w13, act, gate_up=None):
    I = act.shape[1]
    xd, wd = x.double(), w13.double()
    gu = xd @ wd
    mag = xd.abs() @ wd.abs()
    g, u = gu[:, :I], gu[:, I:]
    eps = (x.shape[1] + 2) * F32 * mag              # of the float32 sums
    eg, eu = eps[:, :I], eps[:, I:]
    ref = g * _sig(g) * u
    # |d silu| <= 1.1, |silu(g)| <= |g|; the float32 silu and products: 8 ulps
    tol = HALF * ref.abs() + (1.1 * u.abs() * eg + g.abs() * eu) * (1 + HALF) + 16 * F32 * ref.abs() + 1e-36
    err = (act.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if gate_up is not None:
        err, tol = (gate_up.double() - gu).abs(), HALF * gu.abs() + eps * (1 + HALF) + 1e-37
        assert bool((err <= tol).all()), float((err / tol).max())


def check_backward(d_act, x, w13, gate_up, dx, dw13):
    import torch
    I = d_act.shape[1]
    g, u, d = gate_up[:, :I].double(), gate_up[:, I:].double(), d_act.double()
    s = _sig(g)
    dgu = torch.cat((d * u * s * (1 + g * (1 - s)), d * g * s), 1)
    # float32 error of an element of dgu: 1 + g (1 - s) cancels for g near -1.28
    edgu = HALF * dgu.abs() + 32 * F32 * torch.cat((d * u * s * (1 + g.abs() * (1 - s)), d * g * s), 1).abs() + 1e-37
    for name, got, a, b in (("dx", dx, dgu, w13.double().t()), ("dw13", dw13, x.double().t(), dgu)):
        if got is None:
            continue
        ref, mag = a @ b, a.abs() @ b.abs()
        moved = edgu @ b.abs() if name == "dx" else a.abs() @ edgu
        tol = HALF * ref.abs() + ((a.shape[1] + 2) * F32 * mag + moved) * (1 + HALF) + 1e-37
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))
        rel = float((got.double() - ref).norm() / ref.norm().clamp(min=1e-300))
        assert rel < 2 * HALF, (name, rel)


# one row; tiles of 64, 128 and 256 rows and rows that end inside them; K tails
# (multiples of 16 that are no multiples of 32), widths below a tile, K chunks
SIZES = [(1, 16, 16), (1, 7168, 2048), (2, 48, 32), (3, 32, 16), (17, 272, 144), (64, 512, 128), (65, 528, 272),
         (128, 1024, 256), (129, 256, 400), (200, 2048, 1408), (255, 96, 2064), (257, 1040, 128),
         (1000, 512, 512), (2049, 304, 1040), (4096, 1024, 1024)]


@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward(nv, T, H, I):
    import torch
    x, w13, _ = _inputs(T, H, I, 3 * T + H + I)
    act = torch.full((T, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    gate_up = torch.full((T, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.gated_forward(x, w13, act=act, gate_up=gate_up)
    check_forward(x, w13, act, gate_up)
    assert torch.equal(nv.gated_forward(x, w13), act)       # without the tap: the same bits


@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward(nv, T, H, I):
    import torch
    x, w13, d_act = _inputs(T, H, I, 5 * T + H + I)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    nv.gated_forward(x, w13, gate_up=gate_up)
    dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw13 = torch.full((H, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.gated_backward(d_act, x, w13, gate_up, dx=dx, dw13=dw13)
    check_backward(d_act, x, w13, gate_up, dx, dw13)
    # one gradient alone has the same bits
    a, none = nv.gated_backward(d_act, x, w13, gate_up, need_dw13=False)
    assert none is None and torch.equal(a, dx)
    none, b = nv.gated_backward(d_act, x, w13, gate_up, need_dx=False)
    assert none is None and torch.equal(b, dw13)


def test_empty_batch(nv):
    import torch
    x, w13, d_act = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((0, 64), (64, 96), (0, 48)))
    assert nv.gated_forward(x, w13).shape == (0, 48)
    dw13 = torch.full((64, 96), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx, _ = nv.gated_backward(d_act, x, w13, torch.zeros((0, 96), dtype=torch.bfloat16, device="cuda"), dw13=dw13)
    assert dx.shape == (0, 64) and bool((dw13 == 0).all())


def test_large_gates(nv):
    """silu far from zero on both sides: gates of +-200 neither overflow nor
    give NaN, forward and backward."""
    import torch
    T, H, I = 40, 64, 64
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    w13 = torch.zeros((H, 2 * I), dtype=torch.bfloat16, device="cuda")
    gates = torch.linspace(-200, 200, I).to(torch.bfloat16).cuda()
    w13[0, :I] = gates
    w13[1, I:] = 3.0
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    act = nv.gated_forward(x, w13, gate_up=gate_up)
    check_forward(x, w13, act, gate_up)
    d_act = _rand((T, I), 1.0, 1, torch)
    dx, dw13 = nv.gated_backward(d_act, x, w13, gate_up)
    check_backward(d_act, x, w13, gate_up, dx, dw13)


def test_gates_at_the_end_of_the_range(nv):
    """Gates up to the largest finite bf16: silu is the gate or zero, the
    derivative one or zero (the products stay in range with small up values)."""
    import torch
    T, H, I = 3, 16, 32
    big = float(torch.finfo(torch.bfloat16).max)
    gates = torch.tensor([big, -big, 2.4e38, -2.4e38, 1e38, -1e38, 300.0, -300.0] * 4)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, :2] = 1.0
    w13 = torch.zeros((H, 2 * I), dtype=torch.bfloat16, device="cuda")
    w13[0, :I] = gates.to(torch.bfloat16).cuda()
    w13[1, I:] = 2.0 ** -10
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    act = nv.gated_forward(x, w13, gate_up=gate_up)
    on = (gates > 0).cuda()
    ref = torch.where(on, gate_up[:, :I].double() * 2.0 ** -10, torch.zeros((), dtype=torch.float64, device="cuda"))
    assert bool(((act.double() - ref).abs() <= HALF * ref.abs() + 1e-36).all())
    d_act = torch.ones((T, I), dtype=torch.bfloat16, device="cuda")
    ones = torch.zeros((H, 2 * I), dtype=torch.bfloat16, device="cuda")
    ones[0, :I] = 1.0                               # dx[:, 0] = sum of dgate = 16 gates x 2^-10
    dx, _ = nv.gated_backward(d_act, x, ones, gate_up, need_dw13=False)
    assert bool((dx[:, 0].double() == 16 * 2.0 ** -10).all())


@pytest.mark.parametrize("T,H,I", [(1, 64, 32), (70, 272, 144), (300, 528, 1040)])
def test_nothing_beside_the_outputs_is_written(nv, T, H, I):
    """Outputs and a workspace of exactly the asked size inside larger buffers:
    what lies before and behind them stays."""
    import torch
    x, w13, d_act = _inputs(T, H, I, 31)
    lib = nv._lib
    guard = 4096
    bufs = []

    def inside(shape, dtype=torch.bfloat16):
        n = 1
        for d in shape:
            n *= d
        size = n * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((size + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        bufs.append((buf, size))
        return buf[guard:guard + size].view(dtype).view(shape)

    act, gate_up, dx, dw13 = inside((T, I)), inside((T, 2 * I)), inside((T, H)), inside((H, 2 * I))
    ws = inside((lib.nvfp4_gated_workspace(T, H, I),), torch.uint8)
    wsb = inside((lib.nvfp4_gated_backward_workspace(T, H, I),), torch.uint8)
    nv.gated_forward(x, w13, act=act, gate_up=gate_up, workspace=ws)
    nv.gated_backward(d_act, x, w13, gate_up, dx=dx, dw13=dw13, workspace=wsb)
    check_forward(x, w13, act, gate_up)
    check_backward(d_act, x, w13, gate_up, dx, dw13)
    for buf, size in bufs:
        assert bool((buf[:guard] == 0x5A).all()) and bool((buf[guard + size:] == 0x5A).all())


def test_two_streams_at_once(nv):
    """Calls in flight together on two streams, each with its own workspace."""
    import torch
    cases = [(33, 1024, 512, 41), (200, 2048, 256, 42)]
    data = [_inputs(T, H, I, s) for T, H, I, s in cases]
    alone = [nv.gated_forward(x, w).clone() for x, w, _ in data]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[k].append(nv.gated_forward(data[k][0], data[k][1]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, alone[k]) for o in out[k])


@pytest.mark.parametrize("T,H,I", [(5, 528, 64), (300, 272, 144)])
def test_rows_are_separate(nv, T, H, I):
    """NaN and infinity in one row of x and d_act stay in that row of act and
    dx (they do reach dw13, whose sums run over the rows)."""
    import torch
    x, w13, d_act = _inputs(T, H, I, 77)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    act = nv.gated_forward(x, w13, gate_up=gate_up).clone()
    dx, _ = nv.gated_backward(d_act, x, w13, gate_up, need_dw13=False)
    bad = T - 2
    x2, gu2, d2 = x.clone(), gate_up.clone(), d_act.clone()
    x2[bad, ::2], x2[bad, 1::2] = float("nan"), float("inf")
    gu2[bad], d2[bad] = float("nan"), float("inf")
    act2 = nv.gated_forward(x2, w13)
    dx2, _ = nv.gated_backward(d2, x2, w13, gu2, need_dw13=False)
    keep = torch.arange(T, device="cuda") != bad
    assert torch.equal(act2[keep], act[keep]) and torch.equal(dx2[keep], dx[keep])
    assert bool(act2[bad].isnan().all()) and bool(dx2[bad].isnan().all())


def test_gradients_match_differences(nv):
    """Directional differences of sum(act * d_act), evaluated in float64 by the
    formula, against the kernel's gradients: central differences with step h
    are off by O(h^2); the gradients by their bf16 roundings, which the random
    direction averages (a bound of 1 % leaves a factor of about five)."""
    import torch
    T, H, I = 48, 160, 96
    x, w13, d_act = _inputs(T, H, I, 11)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    nv.gated_forward(x, w13, gate_up=gate_up)
    dx, dw13 = nv.gated_backward(d_act, x, w13, gate_up)

    def loss(xd, wd):
        gu = xd @ wd
        g, u = gu[:, :I], gu[:, I:]
        return float((g * _sig(g) * u * d_act.double()).sum())

    xd, wd, h = x.double(), w13.double(), 1e-5
    for got, which in ((dx, 0), (dw13, 1)):
        v = got.double() / got.double().norm()          # along the gradient: the largest slope
        a = (xd + h * v, wd) if which == 0 else (xd, wd + h * v)
        b = (xd - h * v, wd) if which == 0 else (xd, wd - h * v)
        slope = (loss(*a) - loss(*b)) / (2 * h)
        assert abs(slope - float(got.double().norm())) < 0.01 * slope


def test_streams_graph_and_shared_inputs(nv):
    """A captured call replays into the same bits on new values, beside eager
    calls; a call on a side stream too."""
    import torch
    T, H, I = 33, 512, 256
    x, w13, d_act = _inputs(T, H, I, 21)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    act, dx, dw13 = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((T, I), (T, H), (H, 2 * I)))
    import nvfp4_block_scaled_quant_amd as m
    n = max(m._lib.nvfp4_gated_workspace(T, H, I), m._lib.nvfp4_gated_backward_workspace(T, H, I))
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")

    def both(workspace=None):
        nv.gated_forward(x, w13, act=act, gate_up=gate_up, workspace=workspace)
        nv.gated_backward(d_act, x, w13, gate_up, dx=dx, dw13=dw13, workspace=workspace)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(ws)
    for seed in (22, 23, 24):
        x2, w2, d2 = _inputs(T, H, I, seed)
        x.copy_(x2), w13.copy_(w2), d_act.copy_(d2)
        for t in (act, gate_up, dx, dw13):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (act, gate_up, dx, dw13)]
        both()
        torch.cuda.synchronize()
        for a, b in zip(got, (act, gate_up, dx, dw13)):
            assert torch.equal(a, b)


def test_refusals(nv):
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w13 = torch.zeros((4, 32), **bf), torch.zeros((32, 64), **bf)
    d, gu = torch.zeros((4, 32), **bf), torch.zeros((4, 64), **bf)
    with pytest.raises(TypeError):
        nv.gated_forward(x.float(), w13)
    with pytest.raises(TypeError):
        nv.gated_forward(x.cpu(), w13)
    with pytest.raises(ValueError):
        nv.gated_forward(x.t(), w13)                       # not contiguous
    with pytest.raises(ValueError):
        nv.gated_forward(x, torch.zeros((48, 64), **bf))   # H differs
    with pytest.raises(ValueError):
        nv.gated_forward(torch.zeros((4, 24), **bf), torch.zeros((24, 64), **bf))
    with pytest.raises(ValueError):
        nv.gated_forward(x, torch.zeros((32, 40), **bf))
    with pytest.raises(ValueError):
        nv.gated_forward(x, w13, gate_up=torch.zeros((4, 32), **bf))
    with pytest.raises(nv.Nvfp4Error):
        nv.gated_forward(x, w13, workspace=torch.empty((8,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(nv.Nvfp4Error):                     # not 16-byte aligned
        nv.gated_forward(torch.zeros((4 * 32 + 1,), **bf)[1:].view(4, 32), w13)
    with pytest.raises(ValueError):
        nv.gated_backward(d, x, w13, gu[:, :32].contiguous())
    with pytest.raises(ValueError):
        nv.gated_backward(d, x, w13, gu, need_dx=False, need_dw13=False)
    with pytest.raises(ValueError):
        nv.gated_backward(d, x, w13, gu, dx=torch.zeros((4, 32), **bf), need_dx=False)


@pytest.mark.parametrize("T,H,I", [(140001, 16, 16384), (140001, 16384, 16)])
def test_offsets_beyond_32_bits(nv, T, H, I):
    """Operands and outputs of more than 4 GiB: rows of both ends, and the
    weight gradient's rows and columns of both ends."""
    import torch
    g = torch.Generator("cuda").manual_seed(T + H)

    def normal(shape, std):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std

    x, w13, d_act = normal((T, H), 1.5), normal((H, 2 * I), 2.5 / (1.5 * H ** 0.5)), normal((T, I), 0.5)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    act = nv.gated_forward(x, w13, gate_up=gate_up)
    dx, dw13 = nv.gated_backward(d_act, x, w13, gate_up)
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    check_forward(x[rows], w13, act[rows], gate_up[rows])
    check_backward(d_act[rows], x[rows], w13, gate_up[rows], dx[rows], None)
    h = torch.tensor([0, 7, H - 1], device="cuda")
    c = torch.tensor([0, 5, I - 1], device="cuda")
    both = torch.cat((c, I + c))
    check_backward(d_act[:, c], x[:, h], w13[h][:, both], gate_up[:, both], None, dw13[h][:, both])
