"""Argument checks on the host of the operators around the experts, before any
device is touched, and the refusal of inputs whose gradient would be lost (runs
without a GPU)."""
import ctypes

import pytest
import torch

A16 = 1 << 20          # a fake, aligned, never-dereferenced address
BIG = 1 << 44


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quant_amd as nv
    return nv


@pytest.fixture(scope="module")
def lib(nv):
    return nv._lib


def p(v):
    return ctypes.c_void_p(v)


def test_sort_tokens_argument_errors(lib):
    ws = lib.nvfp4_sort_tokens_workspace

    def call(T=4, H=33, E=5, k=2, dtype=0, x=A16, ids=A16, rows=A16, off=A16, row=A16, wsp=A16, nbytes=BIG):
        return lib.nvfp4_sort_tokens(p(x), dtype, p(ids), T, H, E, k, p(rows), p(off), p(row), p(wsp), nbytes, None)

    assert call(T=-1) == 1 and call(H=0) == 1 and call(E=0) == 1 and call(k=0) == 1 and call(dtype=3) == 1
    assert call(dtype=-1) == 1
    assert call(E=513) == 2 and call(k=513) == 2 and call(T=(1 << 24) + 1) == 2 and call(H=(1 << 20) + 1) == 2
    assert call(T=1 << 23, k=129) == 2
    for name in ("x", "ids", "rows", "off", "row"):
        assert call(**{name: 0}) == 1 and call(**{name: A16 + 1}) == 1, name
    assert call(T=0, x=0, ids=0, rows=0, row=0, off=0) == 1
    assert call(x=A16 + 2, dtype=2) == 1 and call(rows=A16 + 2, dtype=2) == 1
    # small batches need no workspace, larger ones and invalid sizes see to it
    assert ws(0, 5, 2) == 0 and ws(4, 5, 2) == 0 and ws(4, 513, 2) == 0 and ws(-1, 5, 2) == 0
    for T, E, k in ((4096, 48, 8), (1 << 16, 256, 8)):
        need = ws(T, E, k)
        assert need > 0 and need % 256 == 0
        big = dict(T=T, E=E, k=k)
        assert call(nbytes=need - 1, **big) == 3 and call(wsp=0, **big) == 3 and call(wsp=A16 + 64, **big) == 3
        assert call(x=A16 + 2, rows=A16 + 6, nbytes=need - 1, **big) == 3           # any element's alignment


def test_gather_argument_errors(lib):
    def back(T=4, H=33, k=2, R=8, dtype=1, d=A16, row=A16, dx=A16):
        return lib.nvfp4_sort_tokens_backward(p(d), dtype, p(row), T, H, k, R, p(dx), None)

    def unsort(T=4, H=33, k=2, R=8, dtype=1, d=A16, row=A16, w=A16, dx=A16):
        return lib.nvfp4_unsort_tokens(p(d), dtype, p(row), p(w), T, H, k, R, p(dx), None)

    for f in (back, unsort):
        assert f(T=0, d=0, row=0, dx=0) == 0
        assert f(T=-1) == 1 and f(H=0) == 1 and f(k=0) == 1 and f(R=-1) == 1 and f(dtype=5) == 1
        assert f(k=513) == 2 and f(R=(1 << 30) + 1) == 2 and f(H=(1 << 20) + 1) == 2
        for name in ("d", "row", "dx"):
            assert f(**{name: 0}) == 1 and f(**{name: A16 + 1}) == 1, name
        assert f(dtype=2, d=A16 + 2) == 1 and f(dtype=2, dx=A16 + 2) == 1
    assert unsort(w=0) == 1 and unsort(w=A16 + 2) == 1


def test_unsort_backward_argument_errors(lib):
    def f(T=4, H=33, k=2, R=8, dtype=0, dy=A16, rows=A16, row=A16, w=A16, dr=A16, dw=A16):
        return lib.nvfp4_unsort_tokens_backward(p(dy), p(rows), dtype, p(row), p(w), T, H, k, R, p(dr), p(dw), None)

    assert f(T=0, dy=0, dr=0, dw=0) == 0 and f(R=0, dw=0) == 0
    assert f(dr=0, dw=0) == 1 and f(T=-1) == 1 and f(dtype=9) == 1 and f(k=513) == 2
    assert f(dy=0) == 1 and f(row=0) == 1 and f(w=0) == 1 and f(rows=0) == 1
    for name in ("dy", "rows", "row", "w", "dr", "dw"):
        assert f(**{name: A16 + 1}) == 1, name


def test_router_gradient_argument_errors(lib):
    def f(T=4, E=5, k=2, dw=A16, ids=A16, w=A16, dl=A16):
        return lib.nvfp4_route_topk_backward(p(dw), p(ids), p(w), T, E, k, p(dl), None)

    assert f(T=0, dw=0, ids=0, w=0, dl=0) == 0
    assert f(T=-1) == 1 and f(E=0) == 1 and f(k=0) == 1
    assert f(k=6) == 2 and f(E=513) == 2 and f(T=1 << 23, E=256) == 2
    for name in ("dw", "ids", "w", "dl"):
        assert f(**{name: 0}) == 1 and f(**{name: A16 + 2}) == 1, name


def test_matvec_argument_errors(lib):
    def f(M=4, N=32, K=64, E=1, flags=0, dtype=0, x=A16, bq=A16, bsf=A16, alpha=A16, off=0, out=A16):
        return lib.nvfp4_matvec(p(x), dtype, p(bq), p(bsf), p(alpha), p(off), M, N, K, E, flags, p(out), None)

    assert f(M=0, x=0, bq=0, out=0) == 0
    assert f(M=-1) == 1 and f(N=0) == 1 and f(K=-16) == 1 and f(E=0) == 1 and f(dtype=2) == 1 and f(flags=4) == 1
    assert f(flags=2) == 1                                    # two alphas without a gate
    assert f(K=24) == 2 and f(N=24) == 2 and f(N=48, flags=1) == 2 and f(E=2) == 2 and f(E=513, off=A16) == 2
    assert f(N=1 << 20, K=1 << 13) == 2 and f(M=(1 << 24) + 1) == 2 and f(K=(1 << 20) + 16, N=16) == 2
    assert f(M=1 << 24, N=1 << 16, K=16) == 2                 # too many work-groups
    for name in ("x", "bq", "bsf", "alpha", "out"):
        assert f(**{name: 0}) == 1, name
    for name, off in (("x", 8), ("bq", 8), ("bsf", 4), ("alpha", 2), ("off", 2), ("out", 1)):
        assert f(**{name: A16 + off}) == 1, name


def test_dropout_argument_errors(lib):
    def f(n=8, prob=0.5, dtype=0, x=A16, res=0, rng=A16, y=A16):
        return lib.nvfp4_dropout(p(x), p(res), dtype, n, prob, p(rng), p(y), None)

    def b(n=8, prob=0.5, dtype=0, x=A16, rng=A16, y=A16):
        return lib.nvfp4_dropout_backward(p(x), dtype, n, prob, p(rng), p(y), None)

    for g in (f, b):
        assert g(n=0, x=0, rng=0, y=0) == 0
        assert g(n=-1) == 1 and g(prob=-0.1) == 1 and g(prob=1.1) == 1 and g(prob=float("nan")) == 1
        assert g(dtype=3) == 1 and g(n=(1 << 48) + 1) == 2
        assert g(x=0) == 1 and g(rng=0) == 1 and g(y=0) == 1 and g(rng=A16 + 4) == 1 and g(x=A16 + 1) == 1
    assert f(res=A16 + 1) == 1 and f(res=A16 + 2, dtype=2) == 1


def _calls(nv, device):
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    x, rows, row, w = z(4, 32), z(8, 32), z(4, 2, dtype=i32), z(4, 2, dtype=f32)
    rng = z(2, dtype=torch.int64)
    return ((nv.sort_tokens, dict(x=x, topk_ids=row, num_experts=3), ("x",)),
            (nv.sort_tokens_backward, dict(d_rows=rows, slot_row=row), ("d_rows",)),
            (nv.unsort_tokens, dict(rows=rows, slot_row=row, topk_weights=w), ("rows", "topk_weights")),
            (nv.unsort_tokens_backward, dict(dy=x, rows=rows, slot_row=row, topk_weights=w),
             ("dy", "rows", "topk_weights")),
            (nv.route_topk_backward, dict(d_weights=w, topk_ids=row, topk_weights=w.clone(), num_experts=3),
             ("d_weights", "topk_weights")),
            (nv.matvec, dict(x=x, bq=z(2, 2, 16, 32, dtype=u8), bsf=z(2, 1, 16, 32, dtype=u8), b_alpha=z(1, dtype=f32)),
             ("x", "b_alpha")),
            (nv.dropout, dict(x=x, p=0.5, rng=rng, residual=x.clone()), ("x", "residual")),
            (nv.dropout_backward, dict(dy=x, p=0.5, rng=rng), ("dy",)))


def test_inputs_that_require_a_gradient_are_refused(nv):
    for op, args, names in _calls(nv, "cpu"):
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
def test_without_recording_they_run():
    import nvfp4_block_scaled_quant_amd as nv
    for op, args, names in _calls(nv, "cuda"):
        for name in names:
            args[name].requires_grad_(True)
        with pytest.raises(RuntimeError, match="requires a gradient"):
            op(**args)
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                op(**args)
