"""Cases and plain forms of the projection and feed-forward operators that
stand beside the expert layer:

    gemm_lora       one shared NVFP4 projection with the low-rank adapters of
                    many requests added to its rows (serving)
    gated_forward   act = silu(x @ W_gate) * (x @ W_up), bf16 weights (a dense
                    or shared expert; serving, and the forward of training)
    gated_backward  the gradients of x and of [W_gate | W_up]

`run` computes the plain form (elementary torch operations in float32, one
rounding at the end), or, where `own` is true, calls the framework.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ------------------------------------------------------------------- cases

def _lora(name, M, N, K, L, R, rows, mixed_ranks=False):
    """rows: "each" = every row has the adapter of its own request, drawn at
    random (decode batches); "runs" = requests are runs of rows (prefill).
    About one request in eight has no adapter. mixed_ranks: adapters of ranks
    up to R, stored with R rows."""
    return dict(name=name, op="gemm_lora", M=M, N=N, K=K, L=L, R=R, rows=rows,
                mixed_ranks=mixed_ranks)


def _gated(name, T, H, I, keep=False):
    """keep: also return the rounded gate | up values for the backward pass."""
    return dict(name=name, op="gated_forward", T=T, H=H, I=I, keep=keep)


def _grad(name, T, H, I):
    return dict(name=name, op="gated_backward", T=T, H=H, I=I)


def listed():
    return [
        # one sequence that generates one token through an adapted projection
        _lora("lora_token", 1, 6144, 7168, 8, 16, "each"),
        # a decode batch of 13 sequences, adapters of several ranks, short K
        _lora("lora_decode", 13, 7168, 2048, 16, 64, "each", mixed_ranks=True),
        # a fuller decode batch with many adapters
        _lora("lora_batch", 61, 6144, 7168, 32, 32, "each"),
        # a few prompts' chunks beside each other (the dense GEMM's shape)
        _lora("lora_chunks", 256, 6144, 7168, 6, 16, "runs"),
        # a prefill batch, an odd number of rows
        _lora("lora_prefill", 4093, 6144, 7168, 8, 64, "runs"),
        # the shared expert of one generated token
        _gated("gated_token", 1, 7168, 2048),
        # the shared expert of a decode batch
        _gated("gated_decode", 23, 7168, 2048),
        # a prompt chunk, ragged
        _gated("gated_chunk", 301, 7168, 2048),
        # the forward pass of a training step, gate | up kept
        _gated("gated_train", 4096, 7168, 2048, keep=True),
        # gradients for a short odd batch in a small layer
        _grad("grad_small", 129, 2048, 1408),
        # an odd number of rows and widths that end inside tiles
        _grad("grad_ragged", 1001, 4112, 1360),
        # a training step's backward pass
        _grad("grad_train", 4096, 7168, 2048),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gemm_lora", "gemm_lora", "gated_forward", "gated_backward"))
    if op == "gemm_lora":
        M = _logint(rng, 1, 4096)
        return _lora("", M, 16 * _logint(rng, 32, 448), 16 * _logint(rng, 64, 448), _logint(rng, 1, 48),
                     8 * _logint(rng, 1, 16), "each" if M <= 64 else rng.choice(("each", "runs")),
                     rng.random() < 0.5)
    T = _logint(rng, 1, 4096)
    H, I = 16 * _logint(rng, 64, 448), 16 * _logint(rng, 32, 128)
    if op == "gated_forward":
        return _gated("", T, H, I, rng.random() < 0.5)
    return _grad("", T, H, I)


def work(case):
    if case["op"] == "gemm_lora":
        M, N, K, R = case["M"], case["N"], case["K"], case["R"]
        r = 0.625 * R if case["mixed_ranks"] else R           # the mean rank
        adapters = min(M, case["L"])
        quant = (M + N) * K * (1 / 2 + 1 / 16)
        return {"bytes": quant + 2 * M * K + 2 * adapters * r * (K + N) + 2 * M * N,
                "flops": 2 * M * N * K + 2 * M * r * (K + N)}
    T, H, I = case["T"], case["H"], case["I"]
    if case["op"] == "gated_forward":
        return {"bytes": 2 * (T * H + 2 * H * I + T * I + (2 * T * I if case["keep"] else 0)),
                "flops": 4 * T * H * I}
    return {"bytes": 2 * (T * I + T * H + 2 * H * I + 2 * T * I + T * H + 2 * H * I),
            "flops": 8 * T * H * I}


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _quantize(x):
    """NVFP4 of (rows, K) values, blocks of 16 along K: codes (rows, K) 0..15,
    E4M3 scale bytes (rows, K / 16), global scale (1,)."""
    x = x.float()
    gs = x.abs().max() / 2688.0
    blocks = x.view(x.shape[0], -1, 16)
    sf = (blocks.abs().amax(2) / (6.0 * gs)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (sf.float() * gs).clamp(min=1e-30)
    borders = torch.tensor(E2M1_BORDERS, device=x.device)
    code = torch.bucketize((blocks.abs() / den[:, :, None]).contiguous(), borders)
    code = code.to(torch.uint8) | ((blocks < 0).to(torch.uint8) << 3)
    return code.view(x.shape), sf.view(torch.uint8), gs.view(1)


def _pad(t, n):
    return torch.nn.functional.pad(t, (0, n - t.shape[1]))


def _pack_weights(code, sf):
    """Codes (N, K) and scales (N, K / 16) of the weight columns into the
    packed layout: 16-row blocks, 64-element half steps, scales by groups of
    four 128-element steps."""
    N, K = code.shape
    steps = -(-K // 128)
    quads = -(-steps // 4)
    code = _pad(code, 128 * steps)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    q = q.view(N // 16, 16, 2 * steps, 32).permute(0, 2, 1, 3).contiguous()
    sf = _pad(sf, 32 * quads).view(N // 16, 16, quads, 4, 4, 2)      # row, quad, step, pair, byte
    sf = sf.permute(0, 2, 1, 4, 3, 5).reshape(N // 16, quads, 16, 32).contiguous()
    return q, sf


def _row_ids(gen, rows, M, L):
    """Adapter of each row, -1 for none."""
    def ids(n):
        i = torch.randint(0, L, (n,), generator=gen, device="cuda", dtype=torch.int32)
        bare = torch.rand((n,), generator=gen, device="cuda") < 0.125
        return torch.where(bare & (n > 1), torch.full_like(i, -1), i)
    if rows == "each":
        return ids(M)
    n = min(M, L + 2)                                                # requests
    starts = torch.rand((M,), generator=gen, device="cuda").argsort()[:n]
    run = torch.zeros((M,), dtype=torch.int64, device="cuda")
    run[starts] = 1
    run[0] = 1
    return ids(n + 1)[run.cumsum(0) - 1].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    if case["op"] == "gemm_lora":
        M, N, K, L, R = (case[k] for k in ("M", "N", "K", "L", "R"))
        x = _normal(gen, (M, K), 1.5)
        code, asf, gs = _quantize(x)
        s["x"], s["asf"], s["a_gs"] = x, asf.contiguous(), gs
        s["aq"] = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
        wcode, wsf, s["b_alpha"] = _quantize(_normal(gen, (N, K), 0.02))
        s["bq"], s["bsf"] = _pack_weights(wcode, wsf)
        s["lora_a"] = _normal(gen, (L, R, K), 1.0 / math.sqrt(K))
        s["lora_b"] = _normal(gen, (L, N, R), 0.02)
        s["lora_scale"] = torch.rand((L,), generator=gen, device="cuda") * 1.5 + 0.5
        s["lora_rank"] = None
        if case["mixed_ranks"]:
            s["lora_rank"] = torch.randint(R // 4, R + 1, (L,), generator=gen, device="cuda",
                                           dtype=torch.int32)
        s["adapter_ids"] = _row_ids(gen, case["rows"], M, L)
        return s
    T, H, I = case["T"], case["H"], case["I"]
    s["x"] = _normal(gen, (T, H), 1.5)
    s["w13"] = _normal(gen, (H, 2 * I), 0.02)
    if case["op"] == "gated_backward":
        s["d_act"] = _normal(gen, (T, I), 0.01)
        s["gate_up"] = _normal(gen, (T, 2 * I), 0.03 * math.sqrt(H))  # as x @ w13 spreads
    return s


# -------------------------------------------------------------------- run

def _plain_gemm_lora(s):
    M, N, K, L, R = (s[k] for k in ("M", "N", "K", "L", "R"))
    dev = s["x"].device
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=dev)

    def dequantize(q, sf, rows):
        v = torch.stack((values[(q & 15).long()], values[(q >> 4).long()]), -1).view(rows, -1)
        return v * sf.view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)

    a = dequantize(s["aq"], s["asf"], M)
    steps, quads = s["bq"].shape[1] // 2, s["bsf"].shape[1]
    bq = s["bq"].permute(0, 2, 1, 3).reshape(N, 64 * steps)
    bsf = s["bsf"].view(N // 16, quads, 16, 4, 4, 2).permute(0, 2, 1, 4, 3, 5).reshape(N, 32 * quads)
    b = dequantize(bq, bsf[:, :8 * steps].contiguous(), N)[:, :K]
    base = (a @ b.t()) * (s["a_gs"] * s["b_alpha"])
    v = (s["x"].float() @ s["lora_a"].float().view(L * R, K).t()).view(M, L, R)
    v = v * s["lora_scale"][None, :, None]
    used = s["adapter_ids"][:, None] == torch.arange(L, device=dev)[None, :]
    used = used[:, :, None].expand(M, L, R)
    if s["lora_rank"] is not None:
        used = used & (torch.arange(R, device=dev)[None, :] < s["lora_rank"][:, None])[None]
    v = torch.where(used, v, torch.zeros((), device=dev)).reshape(M, L * R)
    delta = v @ s["lora_b"].float().permute(0, 2, 1).reshape(L * R, N)
    return (base + delta).to(torch.bfloat16)


def _plain_gated_forward(s):
    I = s["I"]
    gu = s["x"].float() @ s["w13"].float()
    g, u = gu[:, :I], gu[:, I:]
    act = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
    return (act, gu.to(torch.bfloat16)) if s["keep"] else act


def _plain_gated_backward(s):
    I = s["I"]
    gu, d = s["gate_up"].float(), s["d_act"].float()
    g, u = gu[:, :I], gu[:, I:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    dgu = torch.cat((d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig), 1)
    dx = dgu @ s["w13"].float().t()
    dw13 = s["x"].float().t() @ dgu
    return dx.to(torch.bfloat16), dw13.to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import nvfp4_block_scaled_quant_amd as nv
        if s["op"] == "gemm_lora":
            return nv.gemm_lora(s["aq"], s["asf"], s["a_gs"], s["bq"], s["bsf"], s["b_alpha"], s["x"],
                                s["lora_a"], s["lora_b"], s["lora_scale"], s["adapter_ids"],
                                lora_rank=s["lora_rank"])
        if s["op"] == "gated_forward":
            if s["keep"]:
                gate_up = torch.empty((s["T"], 2 * s["I"]), dtype=torch.bfloat16, device=s["x"].device)
                return nv.gated_forward(s["x"], s["w13"], gate_up=gate_up), gate_up
            return nv.gated_forward(s["x"], s["w13"])
        return nv.gated_backward(s["d_act"], s["x"], s["w13"], s["gate_up"])
    if s["op"] == "gemm_lora":
        return _plain_gemm_lora(s)
    if s["op"] == "gated_forward":
        return _plain_gated_forward(s)
    return _plain_gated_backward(s)


# ------------------------------------------------------------------ exact

def _e4m3_f64(byte):
    e, m = (byte >> 3).double(), (byte & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * torch.exp2(torch.full_like(e, -6.0)))


def _e2m1_f64(code):
    sign = 1.0 - 2.0 * (code >> 3).double()
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    return sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)


def _silu_f64(g):
    return g * torch.sigmoid(g)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm_lora":
        M, N, K = case["M"], case["N"], case["K"]
        k = torch.arange(K, device="cuda")
        byte = s["aq"][:, k // 2].to(torch.int32)
        a = _e2m1_f64((byte >> (4 * (k % 2))) & 15) * _e4m3_f64(s["asf"].to(torch.int32))[:, k // 16]
        out = torch.empty((M, N), dtype=torch.float64, device="cuda")
        st, g = k // 128, k // 16
        for n0 in range(0, N, 512):                     # columns, by the layout's address formulas
            n = torch.arange(n0, min(N, n0 + 512), device="cuda")[:, None]
            ldq, ldsf = 32 * s["bq"].shape[1], 32 * s["bsf"].shape[1]
            at = n // 16 * 16 * ldq + k // 64 * 512 + n % 16 * 32 + k // 2 % 32
            byte = s["bq"].view(-1)[at].to(torch.int32)
            at = n // 16 * 16 * ldsf + st // 4 * 512 + n % 16 * 32 + g % 8 // 2 * 8 + st % 4 * 2 + g % 2
            b = _e2m1_f64((byte >> (4 * (k % 2))) & 15) * _e4m3_f64(s["bsf"].view(-1)[at].to(torch.int32))
            out[:, n0:n0 + b.shape[0]] = a @ b.t()
        out *= s["a_gs"].double() * s["b_alpha"].double()
        for i in range(case["L"]):
            rows = (s["adapter_ids"] == i).nonzero()[:, 0]
            r = case["R"] if s["lora_rank"] is None else int(s["lora_rank"][i])
            v = s["x"][rows].double() @ s["lora_a"][i, :r].double().t()
            out[rows] += s["lora_scale"][i].double() * (v @ s["lora_b"][i, :, :r].double().t())
        return out
    I = case["I"]
    x, w = s["x"].double(), s["w13"].double()
    if case["op"] == "gated_forward":
        gate, up = x @ w[:, :I].contiguous(), x @ w[:, I:].contiguous()
        act = _silu_f64(gate) * up
        return (act, torch.cat((gate, up), 1)) if case["keep"] else act
    g = s["gate_up"][:, :I].double().requires_grad_(True)
    u = s["gate_up"][:, I:].double().requires_grad_(True)
    (_silu_f64(g) * u).backward(s["d_act"].double())
    dx = g.grad @ w[:, :I].t() + u.grad @ w[:, I:].t()
    return dx, torch.cat((x.t() @ g.grad, x.t() @ u.grad), 1)
