"""Cases and plain forms of the operators around the experts:

    sort_tokens      tokens sorted by expert, and its gradient
    unsort_tokens    expert rows back to their tokens, weights applied, and its
                     gradients
    route_topk_backward
                     the router's gradient
    matvec           a few rows times 4-bit weights with group scales: one
                     matrix, or each row with its expert's, gated or not
    dropout          from a counter-based generator, and its gradient

`run` computes the plain form (elementary torch operations in float32, one
rounding at the end), or, where `own` is true, calls the framework.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def _tokens(name, op, T, H, E, k, dtype, routed=None):
    """E experts of this GPU out of `routed` that the router chooses from (the
    slots of the others are skipped)."""
    return dict(name=name, op=op, T=T, H=H, E=E, k=k, dtype=dtype, routed=routed or E)


def _router(name, T, E, k):
    return dict(name=name, op="route_topk_backward", T=T, E=E, k=k)


def _matvec(name, M, N, K, dtype):
    return dict(name=name, op="matvec", M=M, N=N, K=K, dtype=dtype)


def _experts(name, T, k, E, N, K, dtype, gated):
    """The sorted rows of T tokens, each times its expert's matrix. gated: N
    is gate and up together."""
    return dict(name=name, op="matvec_experts", T=T, k=k, E=E, N=N, K=K, dtype=dtype, gated=gated)


def _dropout(name, T, H, p, dtype, residual=False, backward=False):
    return dict(name=name, op="dropout", T=T, H=H, p=p, dtype=dtype, residual=residual, backward=backward)


def listed():
    return [
        # a decode batch of 8 sequences on its way to 48 experts
        _tokens("sort_decode", "sort", 8, 7168, 48, 8, "bf16"),
        # a ragged prefill batch where the GPU holds a third of the experts
        _tokens("sort_share", "sort", 4093, 7168, 16, 8, "f16", routed=48),
        # the gradient of a training step's tokens
        _tokens("sort_grad_train", "sort_backward", 4096, 7168, 48, 8, "bf16"),
        # a short odd batch of a small layer in float32, the way back
        _tokens("unsort_small", "unsort", 301, 2049, 33, 6, "f32"),
        # a training step's way back, both gradients
        _tokens("unsort_grad_train", "unsort_backward", 4096, 7168, 48, 8, "bf16"),
        # the router's gradient of that step
        _router("router_grad", 4096, 48, 8),
        # the same over a long batch and many experts
        _router("router_grad_long", 65539, 256, 8),
        # one token through one projection
        _matvec("matvec_token", 1, 6144, 7168, "bf16"),
        # a decode batch of 13 sequences, short K
        _matvec("matvec_batch", 13, 7168, 2048, "f16"),
        # the gated up-projection of 8 tokens' experts
        _experts("matvec_experts", 8, 8, 48, 4096, 7168, "bf16", True),
        # dropout of a training step's expert outputs, added to the residual
        _dropout("dropout_train", 4096, 7168, 0.1, "bf16", residual=True),
        # gradient of a short odd batch
        _dropout("dropout_grad_odd", 301, 2049, 0.25, "f32", backward=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sort", "sort_backward", "unsort", "unsort_backward", "route_topk_backward", "matvec",
                     "matvec_experts", "dropout"))
    if op == "route_topk_backward":
        E = _logint(rng, 2, 256)
        return _router("", _logint(rng, 1, 65539), E, rng.randint(1, min(E, 8)))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "dropout":
        H = _logint(rng, 33, 7168)
        most = 4096 * 7168 * 2 // (BYTES[dtype] * H)
        return _dropout("", _logint(rng, 1, min(4096, most)), H, round(rng.uniform(0.02, 0.6), 3), dtype,
                        *rng.choice(((False, False), (True, False), (False, True))))
    if op == "matvec":
        return _matvec("", rng.randint(1, 16), 16 * _logint(rng, 32, 448), 16 * _logint(rng, 32, 448),
                       rng.choice(("bf16", "f16")))
    if op == "matvec_experts":
        E = _logint(rng, 2, 48)
        return _experts("", rng.randint(1, 8), rng.randint(1, min(E, 8)), E, 32 * _logint(rng, 16, 128),
                        16 * _logint(rng, 32, 448), rng.choice(("bf16", "f16")), rng.random() < 0.5)
    E, k = _logint(rng, 2, 256), rng.randint(1, 8)
    k = min(k, E)
    H = _logint(rng, 33, 4097) if rng.random() < 0.2 else 16 * _logint(rng, 16, 448)
    most = 4096 * 8 * 7168 * 2 // (BYTES[dtype] * H * k)
    return _tokens("", op, _logint(rng, 1, min(4096, most)), H, E, k, dtype,
                   E if rng.random() < 0.6 else min(512, E * rng.randint(2, 4)))


def work(case):
    op = case["op"]
    if op == "route_topk_backward":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 12 * T * k + 4 * T * E, "flops": 4 * T * k}
    if op == "matvec":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K * 9 / 16 + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "matvec_experts":
        S, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
        used = E * (1 - (1 - case["k"] / E) ** case["T"])     # experts with a row, in the mean
        return {"bytes": used * N * K * 9 / 16 + 2 * S * K + S * N * (1 if case["gated"] else 2),
                "flops": 2 * S * N * K}
    b = BYTES[case["dtype"]]
    if op == "dropout":
        n = case["T"] * case["H"]
        return {"bytes": n * b * (3 if case["residual"] else 2), "flops": 2 * n}
    T, H, k = case["T"], case["H"], case["k"]
    S = T * k * min(1.0, case["E"] / case["routed"])          # valid slots, in the mean
    if op == "sort":
        return {"bytes": (T + S) * H * b + 8 * T * k, "flops": 0}
    if op == "sort_backward":
        return {"bytes": (T + S) * H * b + 4 * T * k, "flops": S * H}
    if op == "unsort":
        return {"bytes": (T + S) * H * b + 8 * T * k, "flops": 2 * S * H}
    return {"bytes": (T + 2 * S) * H * b + 12 * T * k, "flops": 3 * S * H}


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _routing(gen, T, E, k):
    """Distinct experts of each token, most likely first, and their weights."""
    logits = torch.randn((T, E), generator=gen, device="cuda")
    logits += torch.randn((E,), generator=gen, device="cuda") * 0.5          # some experts are chosen more often
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _order(ids, E):
    """offsets (E + 1) and slot_row (T, k) of the stable order by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    bounds = torch.arange(E + 1, device=ids.device)
    offsets = (key[None, :] < bounds[:, None]).sum(1) if key.numel() < 4096 else \
        torch.searchsorted(key[order], bounds)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    row = torch.where(key < E, row, -1)
    return offsets.to(torch.int32), row.to(torch.int32).view(ids.shape), order


def _quantize(x):
    """NVFP4 of (rows, K) values, blocks of 16 along K: codes (rows, K) 0..15,
    E4M3 scale bytes (rows, K / 16), global scale (1,)."""
    x = x.float()
    gs = x.abs().max() / 2688.0
    blocks = x.view(x.shape[0], -1, 16)
    sf = (blocks.abs().amax(2) / (6.0 * gs)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (sf.float() * gs).clamp(min=1e-30)
    borders = torch.tensor(E2M1_BORDERS, device=x.device)
    code = torch.bucketize((blocks.abs() / den[:, :, None]).contiguous(), borders, out_int32=True)
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    s = dict(case)
    op = case["op"]
    if op == "route_topk_backward":
        T, E, k = case["T"], case["E"], case["k"]
        s["ids"], s["weights"] = _routing(gen, T, E, k)
        s["d_weights"] = _normal(gen, (T, k), 0.05, torch.float32)
        return s
    if op in ("matvec", "matvec_experts"):
        N, K, dtype = case["N"], case["K"], TYPES[case["dtype"]]
        E = case.get("E", 1)
        parts = []
        for _ in range(E):
            code, sf, alpha = _quantize(_normal(gen, (N, K), 0.02))
            parts.append(_pack_weights(code, sf) + (alpha,))
        if op == "matvec":
            s["x"] = _normal(gen, (case["M"], K), 1.5, dtype)
            s["bq"], s["bsf"], s["alpha"] = parts[0]
            return s
        s["bq"], s["bsf"], s["alpha"] = (torch.stack([p[i] for p in parts]) for i in range(3))
        s["alpha"] = s["alpha"].view(E)
        ids, _ = _routing(gen, case["T"], E, case["k"])
        s["offsets"], _, order = _order(ids, E)
        s["x"] = _normal(gen, (case["T"], K), 1.5, dtype)[order // case["k"]].contiguous()
        return s
    dtype = TYPES[case["dtype"]]
    T, H = case["T"], case["H"]
    if op == "dropout":
        s["x"] = _normal(gen, (T, H), 1.0, dtype)
        s["res"] = _normal(gen, (T, H), 2.0, dtype) if case["residual"] else None
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")      # seed, offset
        return s
    E, k = case["E"], case["k"]
    s["ids"], s["weights"] = _routing(gen, T, case["routed"], k)
    if op == "sort":
        s["x"] = _normal(gen, (T, H), 1.5, dtype)
        s["rows"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")      # the rows of skipped slots stay zero
        return s
    s["offsets"], s["slot_row"], _ = _order(s["ids"], E)
    if op == "sort_backward":
        s["d_rows"] = _normal(gen, (T * k, H), 0.01, dtype)
        return s
    s["rows"] = _normal(gen, (T * k, H), 0.7, dtype)
    if op == "unsort_backward":
        s["dy"] = _normal(gen, (T, H), 0.01, dtype)
        s["d_rows"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")
    return s


# -------------------------------------------------------------------- run

def _plain_sort(s):
    offsets, slot_row, order = _order(s["ids"], s["E"])
    valid = torch.arange(order.numel(), device=order.device) < offsets[-1]
    rows = torch.where(valid[:, None], s["x"][order // s["k"]], torch.zeros((), dtype=s["x"].dtype, device="cuda"))
    return rows, offsets, slot_row


def _gathered(rows, slot_row):
    """The rows of each token's slots in float32, zeros where there is none."""
    none = (slot_row < 0)[:, :, None]
    return torch.where(none, torch.zeros((), device="cuda"), rows[slot_row.clamp(min=0).long()].float())


def _plain_unsort_backward(s):
    dy = s["dy"].float()
    has = s["slot_row"] >= 0
    d_weights = (_gathered(s["rows"], s["slot_row"]) * dy[:, None, :]).sum(2)
    d_weights = torch.where(has, d_weights, torch.zeros((), device="cuda"))
    n = s["rows"].shape[0]
    at = torch.where(has, s["slot_row"].long(), n).reshape(-1)               # skipped slots go to a row of their own
    d_rows = torch.zeros((n + 1, s["H"]), dtype=s["dy"].dtype, device="cuda")
    d_rows[at] = (s["weights"][:, :, None] * dy[:, None, :]).to(s["dy"].dtype).view(at.numel(), -1)
    return d_rows[:n], d_weights


def _plain_route_topk_backward(s):
    w, dw = s["weights"], s["d_weights"]
    d = w * (dw - (w * dw).sum(1, keepdim=True))
    return torch.zeros((s["T"], s["E"]), device="cuda").scatter_add_(1, s["ids"].long(), d)


def _dequantize(bq, bsf, K):
    """Packed weights (E, N / 16, ...) -> (E, N, K) float32 without alpha."""
    E, blocks, halves = bq.shape[:3]
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    q = bq.permute(0, 1, 3, 2, 4).reshape(E, 16 * blocks, 32 * halves)[:, :, :K // 2].int()
    w = torch.stack((values[q & 15], values[q >> 4]), -1).view(E, 16 * blocks, K // 16, 16)
    sf = bsf.view(E, blocks, -1, 16, 4, 4, 2).permute(0, 1, 3, 2, 5, 4, 6).reshape(E, 16 * blocks, -1)
    sf = sf[:, :, :K // 16].contiguous().view(torch.float8_e4m3fn).float()
    return (w * sf[:, :, :, None]).view(E, 16 * blocks, K)


def _plain_matvec_experts(s):
    w = _dequantize(s["bq"], s["bsf"], s["K"])
    e = torch.searchsorted(s["offsets"][1:], torch.arange(s["x"].shape[0], device="cuda", dtype=torch.int32),
                           right=True)
    out = torch.bmm(w[e], s["x"].float()[:, :, None])[:, :, 0] * s["alpha"][e][:, None]
    if s["gated"]:
        g, u = out.chunk(2, 1)
        out = g / (1.0 + torch.exp(-g)) * u
    return out.to(s["x"].dtype)


def _plain_words(rng, n):
    """n 32-bit words (as int64) of the counter-based generator: Philox4x32 in
    seven rounds, four words for each counter from rng[1] on, key rng[0]."""
    low = 0xFFFFFFFF
    counter = rng[1] + torch.arange(-(-n // 4), device="cuda")
    c = [counter & low, (counter >> 32) & low, torch.zeros_like(counter), torch.zeros_like(counter)]
    key = [rng[0] & low, (rng[0] >> 32) & low]
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57          # 64-bit products, the high half masked out of the sign
        c = [((b >> 32) & low) ^ c[1] ^ key[0], b & low, ((a >> 32) & low) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    return torch.stack(c, 1).reshape(-1)[:n]


def _plain_dropout(s):
    x = s["x"]
    keep = (_plain_words(s["rng"], x.numel()) >= round(s["p"] * 2.0 ** 32)).view(x.shape)
    y = torch.where(keep, x.float() * (1.0 / (1.0 - s["p"])), torch.zeros((), device="cuda"))
    return (y if s["res"] is None else s["res"].float() + y).to(x.dtype)


def _own(s):
    import nvfp4_block_scaled_quant_amd as nv
    op = s["op"]
    if op == "sort":
        return nv.sort_tokens(s["x"], s["ids"], s["E"], rows=s["rows"])
    if op == "sort_backward":
        return nv.sort_tokens_backward(s["d_rows"], s["slot_row"])
    if op == "unsort":
        return nv.unsort_tokens(s["rows"], s["slot_row"], s["weights"])
    if op == "unsort_backward":
        return nv.unsort_tokens_backward(s["dy"], s["rows"], s["slot_row"], s["weights"], d_rows=s["d_rows"])
    if op == "route_topk_backward":
        return nv.route_topk_backward(s["d_weights"], s["ids"], s["weights"], s["E"])
    if op == "matvec":
        return nv.matvec(s["x"], s["bq"], s["bsf"], s["alpha"])
    if op == "matvec_experts":
        return nv.matvec(s["x"], s["bq"], s["bsf"], s["alpha"], offsets=s["offsets"], gated=s["gated"])
    if s["backward"]:
        return nv.dropout_backward(s["x"], s["p"], s["rng"])
    return nv.dropout(s["x"], s["p"], s["rng"], residual=s["res"])


def run(state):
    s = state
    if own:
        return _own(s)
    op = s["op"]
    if op == "sort":
        return _plain_sort(s)
    if op == "sort_backward":
        return _gathered(s["d_rows"], s["slot_row"]).sum(1).to(s["d_rows"].dtype)
    if op == "unsort":
        return (_gathered(s["rows"], s["slot_row"]) * s["weights"][:, :, None]).sum(1).to(s["rows"].dtype)
    if op == "unsort_backward":
        return _plain_unsort_backward(s)
    if op == "route_topk_backward":
        return _plain_route_topk_backward(s)
    if op == "matvec":
        w = _dequantize(s["bq"][None], s["bsf"][None], s["K"])[0]
        return ((s["x"].float() @ w.t()) * s["alpha"]).to(s["x"].dtype)
    if op == "matvec_experts":
        return _plain_matvec_experts(s)
    return _plain_dropout(s)


# ------------------------------------------------------------------ exact

def _e4m3_f64(byte):
    e, m = (byte >> 3).double(), (byte & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * torch.exp2(torch.full_like(e, -6.0)))


def _e2m1_f64(code):
    sign = 1.0 - 2.0 * (code >> 3).double()
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    return sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)


def _exact_product(x, bq, bsf, alpha):
    """x (m, K) times one packed matrix, by the layout's address formulas."""
    K, N = x.shape[1], 16 * bq.shape[0]
    k = torch.arange(K, device="cuda")
    st, g = k // 128, k // 16
    ldq, ldsf = 32 * bq.shape[1], 32 * bsf.shape[1]
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device="cuda")
    for n0 in range(0, N, 1024):
        n = torch.arange(n0, min(N, n0 + 1024), device="cuda")[:, None]
        byte = bq.view(-1)[n // 16 * 16 * ldq + k // 64 * 512 + n % 16 * 32 + k // 2 % 32].to(torch.int32)
        at = n // 16 * 16 * ldsf + st // 4 * 512 + n % 16 * 32 + g % 8 // 2 * 8 + st % 4 * 2 + g % 2
        b = _e2m1_f64((byte >> (4 * (k % 2))) & 15) * _e4m3_f64(bsf.view(-1)[at].to(torch.int32))
        out[:, n0:n0 + b.shape[0]] = x.double() @ b.t()
    return out * alpha.double()


def _exact_keep(rng, n, p):
    """The kept elements, on the host."""
    seed, offset = (int(v) for v in rng.tolist())
    counter = np.uint64(offset) + np.arange(-(-n // 4), dtype=np.uint64)
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    x0, x1 = counter & low, counter >> up
    x2 = x3 = np.zeros_like(x0)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(7):
        p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (p1 >> up) ^ x1 ^ np.uint64(k0), p1 & low, (p0 >> up) ^ x3 ^ np.uint64(k1), p0 & low
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    word = np.empty((x0.size, 4), dtype=np.uint64)
    for i, v in enumerate((x0, x1, x2, x3)):
        word[:, i] = v
    return torch.from_numpy(word.reshape(-1)[:n] >= np.uint64(round(p * 2.0 ** 32))).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route_topk_backward":
        w, dw = s["weights"].double(), s["d_weights"].double()
        out = torch.zeros((case["T"], case["E"]), dtype=torch.float64, device="cuda")
        t = torch.arange(case["T"], device="cuda")
        for j in range(case["k"]):
            rest = sum(w[:, i] * (dw[:, j] - dw[:, i]) for i in range(case["k"]))    # the weights' sum is one
            rest = rest + dw[:, j] * (1 - w.sum(1))
            out[t, s["ids"][:, j].long()] += w[:, j] * rest
        return out
    if op == "matvec":
        return _exact_product(s["x"], s["bq"], s["bsf"], s["alpha"][0])
    if op == "matvec_experts":
        out = torch.zeros((s["x"].shape[0], case["N"]), dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            if b > a:
                out[a:b] = _exact_product(s["x"][a:b], s["bq"][e], s["bsf"][e], s["alpha"][e])
        if case["gated"]:
            n = case["N"] // 2
            out = out[:, :n] * torch.sigmoid(out[:, :n]) * out[:, n:]
        return out
    if op == "dropout":
        x = s["x"].double()
        y = x * _exact_keep(s["rng"], x.numel(), case["p"]).view(x.shape) / (1 - case["p"])
        return y if s["res"] is None else y + s["res"].double()
    T, H, k = case["T"], case["H"], case["k"]
    ids = s["ids"].reshape(-1).cpu().numpy()
    slots = np.nonzero(ids < case["E"])[0]
    slots = slots[np.lexsort((slots, ids[slots]))]                               # the slot of each row
    slot = torch.from_numpy(slots).cuda()
    token, n = slot // k, slot.numel()
    if op == "sort":
        rows = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        rows[:n] = s["x"].double()[token]
        return rows, None, None
    w = s["weights"].double().reshape(-1)[slot]
    if op in ("sort_backward", "unsort"):
        rows = s["d_rows" if op == "sort_backward" else "rows"][:n].double()
        if op == "unsort":
            rows *= w[:, None]
        return torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, token, rows)
    dy = s["dy"].double()[token]
    d_weights = torch.zeros((T * k,), dtype=torch.float64, device="cuda")
    d_weights[slot] = torch.linalg.vecdot(dy, s["rows"][:n].double())
    d_rows = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    d_rows[:n] = dy * w[:, None]
    return d_rows, d_weights.view(T, k)
