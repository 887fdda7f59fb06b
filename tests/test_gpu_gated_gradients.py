"""The gradients of the gated block against differences of the function and
against float64 automatic differentiation, neither of which shares a derivative
formula with the kernel or with test_gpu_gated.py.

Both are taken at the saved gate | up values (bf16), as the kernel's are: the
function is act(G + (x' w' - x w)) for the saved G. Tolerance, per element: half a
bf16 step of the result, of each rounded term dgate / dup of its sum (2^-8 each),
and the float32 sum's n 2^-24 of the sum of magnitudes."""
import pytest

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
F32 = 2.0 ** -24


def _inputs(nv, T, H, I, seed):
    import torch
    g = torch.Generator().manual_seed(seed)

    def normal(shape, std):
        return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()

    x, w13, d_act = normal((T, H), 1.5), normal((H, 2 * I), 2.5 / (1.5 * H ** 0.5)), normal((T, I), 0.5)
    gate_up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    nv.gated_forward(x, w13, gate_up=gate_up)
    return x, w13, d_act, gate_up


def _exact(x, w13, d_act, gate_up):
    """dx, dw13 and their tolerances, by automatic differentiation in float64."""
    import torch
    I = d_act.shape[1]
    gu = gate_up.double().requires_grad_(True)
    act = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    dgu, = torch.autograd.grad(act, gu, d_act.double())
    x, w = x.double(), w13.double()
    # the float32 evaluation of dgate cancels where 1 + g (1 - s) is near zero
    g = gu.detach()[:, :I]
    wide = d_act.double() * gu.detach()[:, I:] * torch.sigmoid(g) * (1 + g.abs())
    e = HALF * dgu.abs() + 32 * F32 * torch.cat((wide, dgu[:, I:]), 1).abs()
    dx, dw = dgu @ w.t(), x.t() @ dgu
    tx = HALF * dx.abs() + (e @ w.abs().t() + (2 * I + 2) * F32 * (dgu.abs() @ w.abs().t())) * (1 + HALF)
    tw = HALF * dw.abs() + (x.abs().t() @ e + (x.shape[0] + 2) * F32 * (x.abs().t() @ dgu.abs())) * (1 + HALF)
    return dx, dw, tx + 1e-37, tw + 1e-37


@pytest.mark.parametrize("T,H,I", [(1, 64, 32), (48, 160, 96), (129, 272, 400), (300, 528, 144), (1000, 512, 512)])
def test_gradients_match_automatic_differentiation(nv, T, H, I):
    x, w13, d_act, gate_up = _inputs(nv, T, H, I, 13 * T + I)
    dx, dw13 = nv.gated_backward(d_act, x, w13, gate_up)
    rx, rw, tx, tw = _exact(x, w13, d_act, gate_up)
    assert bool(((dx.double() - rx).abs() <= tx).all())
    assert bool(((dw13.double() - rw).abs() <= tw).all())


def test_gradients_match_differences_entry_by_entry(nv):
    """Central differences in single entries of x and of each half of w13, drawn
    without looking at the gradients. Step 1e-5 in float64: the truncation is
    below 1e-9 and the cancellation about 1e-7 (the function's terms sum to about
    1e3), so 1e-5 covers both."""
    import torch
    T, H, I = 48, 160, 96
    x, w13, d_act, gate_up = _inputs(nv, T, H, I, 11)
    dx, dw13 = nv.gated_backward(d_act, x, w13, gate_up)
    _, _, tx, tw = _exact(x, w13, d_act, gate_up)
    xd, wd, d, at = x.double(), w13.double(), d_act.double(), gate_up.double()
    gu0 = xd @ wd

    def loss(xe, we):
        gu = at + (xe @ we - gu0)
        g = gu[:, :I]
        return float((g / (1 + torch.exp(-g)) * gu[:, I:] * d).sum())

    gen = torch.Generator().manual_seed(5)
    h = 1e-5
    for got, tol, of_x, cols in ((dx, tx, True, (0, H)), (dw13, tw, False, (0, I)), (dw13, tw, False, (I, 2 * I))):
        rows = torch.randint(0, got.shape[0], (64,), generator=gen)
        picks = torch.randint(cols[0], cols[1], (64,), generator=gen)
        for r, c in zip(rows.tolist(), picks.tolist()):
            ends = []
            for sign in (1, -1):
                e = (xd if of_x else wd).clone()
                e[r, c] += sign * h
                ends.append(loss(e, wd) if of_x else loss(xd, e))
            slope = (ends[0] - ends[1]) / (2 * h)
            assert abs(slope - float(got[r, c])) <= float(tol[r, c]) + 1e-5, (r, c, slope, float(got[r, c]))
