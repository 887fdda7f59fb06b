"""The operators around the experts as programs use them: a training step of a
router and gated experts, and a decode step on 4-bit weights."""
import pytest

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8           # half a bf16 step, relative to the value


def _functions(nv):
    """The operators as a training program wraps them."""
    import torch
    once = torch.autograd.function.once_differentiable

    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k):
            ids, w = nv.route_topk(logits, k)
            ctx.save_for_backward(ids, w)
            ctx.experts = logits.shape[1]
            ctx.mark_non_differentiable(ids)
            return ids, w

        @staticmethod
        @once
        def backward(ctx, _, dw):
            ids, w = ctx.saved_tensors
            return nv.route_topk_backward(dw.contiguous(), ids, w, ctx.experts), None

    class Sort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, ids, experts):
            rows, offsets, row = nv.sort_tokens(x, ids, experts)
            ctx.save_for_backward(row)
            ctx.mark_non_differentiable(offsets, row)
            return rows, offsets, row

        @staticmethod
        @once
        def backward(ctx, d_rows, *_):
            return nv.sort_tokens_backward(d_rows.contiguous(), *ctx.saved_tensors), None, None

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w13):
            gate_up = torch.empty((x.shape[0], w13.shape[1]), dtype=x.dtype, device=x.device)
            act = nv.gated_forward(x, w13, gate_up=gate_up)
            ctx.save_for_backward(x, w13, gate_up)
            return act

        @staticmethod
        @once
        def backward(ctx, d_act):
            return nv.gated_backward(d_act.contiguous(), *ctx.saved_tensors)

    class Unsort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, row, w):
            ctx.save_for_backward(rows, row, w)
            return nv.unsort_tokens(rows, row, w)

        @staticmethod
        @once
        def backward(ctx, dy):
            rows, row, w = ctx.saved_tensors
            d_rows, dw = nv.unsort_tokens_backward(dy.contiguous(), rows, row, w, d_rows=torch.zeros_like(rows))
            return d_rows, None, dw

    class Dropout(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, p, rng):
            ctx.save_for_backward(rng.clone())                # the offset moves on
            ctx.p = p
            return nv.dropout(x, p, rng, residual=residual)

        @staticmethod
        @once
        def backward(ctx, dy):
            dy = dy.contiguous()
            return nv.dropout_backward(dy, ctx.p, *ctx.saved_tensors), dy, None, None

    return Route.apply, Sort.apply, Gated.apply, Unsort.apply, Dropout.apply


def _keep(n, p, seed, offset):
    from test_gpu_dropout import kept
    import torch
    return torch.from_numpy(kept(n, p, seed, offset)).cuda()


@pytest.mark.parametrize("routed", [6, 9])
def test_training_step(nv, routed):
    """y = x + dropout(experts(x)) and the gradients of x, the router's logits and
    the weights against float64 automatic differentiation with the same routing and
    mask. Between the operators values are rounded to bf16 (act, the down
    projection, y, and the same number of gradients on the way back): the norms of
    the differences stay within a step (two halves) for each of the at most eight
    roundings that a gradient passes. routed 9: some slots go to experts elsewhere."""
    import torch
    route, sort, gated, unsort, dropout = _functions(nv)
    T, H, I, E, k, p = 203, 96, 64, 6, 3, 0.2
    g = torch.Generator().manual_seed(4)

    def param(shape, std, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g) * std).to(dtype).cuda().requires_grad_(True)

    x, logits = param((T, H), 1.0), param((T, routed), 1.0, torch.float32)
    w13 = [param((H, 2 * I), H ** -0.5) for _ in range(E)]
    w2 = [param((I, H), I ** -0.5) for _ in range(E)]
    rng = torch.tensor([21, 5], dtype=torch.int64).cuda()
    dy = (torch.randn((T, H), generator=g)).to(torch.bfloat16).cuda()
    leaves = [x, logits] + w13 + w2

    ids, w = route(logits, k)
    rows, offsets, row = sort(x, ids, E)
    ends = offsets.tolist()
    parts = [gated(rows[ends[e]:ends[e + 1]], w13[e]) @ w2[e] for e in range(E)]
    behind = rows.new_zeros((rows.shape[0] - ends[E], H))
    y = dropout(unsort(torch.cat(parts + [behind]), row, w), x, p, rng)
    y.backward(dy)
    got = [y.detach()] + [t.grad for t in leaves]

    xd, ld, *wd = [t.detach().double().requires_grad_(True) for t in leaves]
    wt = torch.softmax(ld.gather(1, ids.long()), 1)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = xd[t] @ wd[e]
        act = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        out = out.index_add(0, t, (act @ wd[E + e]) * wt[t, j][:, None])
    keep = _keep(T * H, p, 21, 5).view(T, H)
    ref = xd + torch.where(keep, out / (1 - p), torch.zeros((), dtype=torch.float64, device="cuda"))
    ref.backward(dy.double())
    want = [ref.detach()] + [t.grad for t in (xd, ld, *wd)]
    for i, (a, b) in enumerate(zip(got, want)):
        assert float((a.double() - b).norm() / b.norm()) <= 8 * 2 * HALF, i


def test_decode_step(nv):
    """Router, sort, gated up projection, down projection and the way back, captured
    once and replayed on new tokens, against float64 over the dequantized weights.
    act and the down projection's rows are rounded to bf16 between the calls, y at
    the end: three half steps of the norm, and their second-order terms."""
    import torch
    from test_gpu_matvec import _randn, _weights
    T, H, I, E, k = 8, 528, 272, 12, 3
    w13, w13_sf, v13, a13 = _weights(nv, E, H, 2 * I, 1, 2)
    w2, w2_sf, v2, a2 = _weights(nv, E, I, H, 2)
    x, logits = _randn((T, H), 1.5, 3, torch.bfloat16), _randn((T, E), 1.0, 4, torch.float32)

    def step():
        ids, w = nv.route_topk(logits, k)
        rows, offsets, row = nv.sort_tokens(x, ids, E)
        act = nv.matvec(rows, w13, w13_sf, a13, offsets=offsets, gated=True)
        down = nv.matvec(act, w2, w2_sf, a2.view(E), offsets=offsets)
        return nv.unsort_tokens(down, row, w), ids

    def exact(ids):
        wt = torch.softmax(logits.double().gather(1, ids.long()), 1)
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j])
                g, u = (x[t].double() @ v13[e]).view(2, I) * a13[e].double()[:, None]
                y[t] += wt[t, j] * ((torch.nn.functional.silu(g) * u) @ v2[e]) * a2.view(E)[e].double()
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ids = step()
    for seed in (5, 6, 7):
        x.copy_(_randn((T, H), 1.5, seed, torch.bfloat16)), logits.copy_(_randn((T, E), 1.0, seed + 9, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        again, _ = step()
        assert torch.equal(y, again)
        ref = exact(ids)
        assert float((y.double() - ref).norm() / ref.norm()) <= 4 * HALF
