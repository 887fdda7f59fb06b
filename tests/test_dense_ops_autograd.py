"""The dense operators write their results without a graph: while gradients are
recorded, an input that requires one is refused rather than dropped from the
graph. (The refusal needs no GPU: it comes before any other check.)"""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import nvfp4_block_scaled_quant_amd as nv
    return nv


def _calls(nv, device):
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    M, N, K, L, R = 4, 32, 64, 2, 8
    u8, f32 = torch.uint8, torch.float32
    lora = dict(aq=z(M, K // 2, dtype=u8), asf=z(M, K // 16, dtype=u8), a_gs=z(1, dtype=f32),
                bq=z(N // 16, 2, 16, 32, dtype=u8), bsf=z(N // 16, 1, 16, 32, dtype=u8), b_alpha=z(1, dtype=f32),
                x=z(M, K), lora_a=z(L, R, K), lora_b=z(L, N, R), lora_scale=z(L, dtype=f32),
                adapter_ids=z(M, dtype=torch.int32))
    fwd = dict(x=z(4, 32), w13=z(32, 64))
    bwd = dict(d_act=z(4, 32), x=z(4, 32), w13=z(32, 64), gate_up=z(4, 64))
    return ((nv.gemm_lora, lora, ("a_gs", "b_alpha", "x", "lora_a", "lora_b", "lora_scale")),
            (nv.gated_forward, fwd, ("x", "w13")), (nv.gated_backward, bwd, ("d_act", "x", "w13", "gate_up")))


def test_inputs_that_require_a_gradient_are_refused(lib):
    for op, args, names in _calls(lib, "cpu"):
        for name in names:
            args[name].requires_grad_(True)
            with pytest.raises(RuntimeError, match="requires a gradient"):
                op(**args)
            with torch.no_grad(), pytest.raises(TypeError):       # not refused for this: CPU tensors
                op(**args)
            args[name].requires_grad_(False)
        with pytest.raises(TypeError):
            op(**args)


@pytest.mark.gpu
def test_without_recording_they_run(nv):
    for op, args, names in _calls(nv, "cuda"):
        first = op(**args)
        first = first if isinstance(first, tuple) else (first,)
        for name in names:
            args[name].requires_grad_(True)
        with pytest.raises(RuntimeError, match="requires a gradient"):
            op(**args)
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                again = op(**args)
            again = again if isinstance(again, tuple) else (again,)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.gpu
def test_in_an_autograd_function(nv):
    """How a training program has the gradients: the two calls inside a function of
    its own, where nothing is recorded."""
    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w13):
            gate_up = torch.empty((x.shape[0], w13.shape[1]), dtype=x.dtype, device=x.device)
            act = nv.gated_forward(x, w13, gate_up=gate_up)
            ctx.save_for_backward(x, w13, gate_up)
            return act

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_act):
            return nv.gated_backward(d_act.contiguous(), *ctx.saved_tensors)

    g = torch.Generator().manual_seed(3)
    x = torch.randn((33, 64), generator=g).to(torch.bfloat16).cuda().requires_grad_(True)
    w13 = (torch.randn((64, 96), generator=g) * 0.2).to(torch.bfloat16).cuda().requires_grad_(True)
    d = torch.randn((33, 48), generator=g).to(torch.bfloat16).cuda()
    Gated.apply(x, w13).backward(d)
    with torch.no_grad():
        gate_up = torch.empty((33, 96), dtype=torch.bfloat16, device="cuda")
        nv.gated_forward(x, w13, gate_up=gate_up)
        dx, dw13 = nv.gated_backward(d, x, w13, gate_up)
    assert torch.equal(x.grad, dx) and torch.equal(w13.grad, dw13)
