"""What is measured of the mixture-of-experts operators: cases, inputs, the plain
form of each operator in elementary torch operations and the framework's calls.

Operators (the formulas are those of include/sqint8.h):
  norm     residual' = bf16(h + residual), RMSNorm of residual' with the folded
           weight gamma, 8-bit codes with scales ("i8": per token, "i8_group": per
           128 columns, "fp8": E4M3 per 128 columns)
  grouped  the experts' products: row t of the expert-sorted order reads token
           rows[t] and the weights of the expert that owns t ("i8": per-token x
           per-channel scales, "fp8": 1x128 x [128, 128] block scales)
  silu     silu(gate) * up of a [T, 2 I] matrix, times 1/s, as 8-bit codes
  experts  gate-up product -> silu -> down product, as a layer calls them

INT8 codes are whole numbers (the norm's arithmetic is exact to the bit); E4M3
codes are returned as the float8 values they are.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one decode step of 8 sequences, the hidden size of the repository's decode workload
        {"name": "norm_i8_decode", "op": "norm", "fmt": "i8", "M": 8, "K": 5120},
        # the repository's prefill workload
        {"name": "norm_i8_prefill", "op": "norm", "fmt": "i8", "M": 8192, "K": 5120},
        # a ragged chunk of a prefill that feeds FP8 block products
        {"name": "norm_fp8_chunk", "op": "norm", "fmt": "fp8", "M": 1777, "K": 2048},
        # a single token that reaches 2 of 8 experts: the smallest call
        {"name": "grouped_i8_one_token", "op": "grouped", "fmt": "i8", "M": 1, "top": 2, "E": 8,
         "K": 2048, "N": 2048, "gather": True},
        # decode of 16 sequences over 64 small experts: weights decide
        {"name": "grouped_i8_decode", "op": "grouped", "fmt": "i8", "M": 16, "top": 8, "E": 64,
         "K": 2048, "N": 1536, "gather": True},
        # a prefill of 4096 tokens over 64 experts, about 512 rows each
        {"name": "grouped_i8_prefill", "op": "grouped", "fmt": "i8", "M": 4096, "top": 8, "E": 64,
         "K": 2048, "N": 2048, "gather": True},
        # decode with FP8 blocks, rows already in the experts' order (the down product)
        {"name": "grouped_fp8_decode", "op": "grouped", "fmt": "fp8", "M": 37, "top": 6, "E": 64,
         "K": 1408, "N": 2048, "gather": False},
        # a long prefill with FP8 blocks over few, wide experts
        {"name": "grouped_fp8_prefill", "op": "grouped", "fmt": "fp8", "M": 4099, "top": 2, "E": 8,
         "K": 5120, "N": 2048, "gather": True},
        # the activation between the two products: decode, and a prefill
        {"name": "silu_fp8_decode", "op": "silu", "fmt": "fp8", "M": 128, "K": 768},
        {"name": "silu_fp8_prefill", "op": "silu", "fmt": "fp8", "M": 32768, "K": 1024},
        # the whole run of a layer's experts: mixed decode and chunked prefill
        {"name": "experts_i8_mixed", "op": "experts", "fmt": "i8", "M": 256, "top": 8, "E": 64,
         "K": 2048, "I": 768},
        {"name": "experts_fp8_chunk", "op": "experts", "fmt": "fp8", "M": 1025, "top": 4, "E": 32,
         "K": 2048, "I": 1024},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["norm", "grouped", "grouped", "silu", "experts"])
    if op == "norm":
        return {"op": op, "fmt": rng.choice(["i8", "i8_group", "fp8"]), "M": size(1, 8192),
                "K": size(256, 5120, 128)}
    if op == "silu":
        return {"op": op, "fmt": "fp8", "M": size(1, 32768), "K": size(128, 1024, 128)}
    fmt = rng.choice(["i8", "fp8"])
    E = size(4, 64)
    top = rng.randint(1, min(8, E))
    M = size(1, max(1, 32768 // top))
    # the weights and the products stay below those of the largest listed case
    if op == "grouped":
        step = 16 if fmt == "i8" else 128
        return {"op": op, "fmt": fmt, "M": M, "top": top, "E": E, "K": size(256, 2048, 128),
                "N": size(256, 2048, step), "gather": rng.random() < 0.5}
    return {"op": op, "fmt": fmt, "M": max(1, M // 4), "top": top, "E": E, "K": size(256, 2048, 128),
            "I": size(128, 1024, 128)}


def _rand_codes(shape, fmt, gen):
    """8-bit codes of normally distributed values scaled to their largest: INT8 or E4M3 bits."""
    v = torch.randn(shape, generator=gen, device=DEV)
    if fmt == "i8":
        return v.mul_(127 / 4.5).round_().clamp_(-127, 127).to(torch.int8)
    return v.mul_(448 / 4.5).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, around, gen):
    return (torch.rand(shape, generator=gen, device=DEV) + 0.5) * around


def _weights(E, N, K, fmt, gen):
    q = _rand_codes((E, N, K), fmt, gen)
    top = 127 if fmt == "i8" else 448
    shape = (E, N) if fmt == "i8" else (E, N // 128, K // 128)
    return q, _scales(shape, 4.5 / top / math.sqrt(K), gen)


def _tokens(M, K, fmt, gen):
    q = _rand_codes((M, K), fmt, gen)
    top = 127 if fmt == "i8" else 448
    return q, _scales((M,) if fmt == "i8" else (M, K // 128), 4.5 / top, gen)


def _route(case, gen):
    """A router's answer: `top` different experts for each token, some experts liked more than
    others, and the rows sorted by expert."""
    M, E, top = case["M"], case["E"], case["top"]
    liked = torch.randn(E, generator=gen, device=DEV) * 0.5
    u = torch.rand((M, E), generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
    ids = (liked - torch.log(-torch.log(u))).topk(top, dim=1).indices.flatten()
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return (order // top).to(torch.int32), offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op, fmt, M, K = case["op"], case["fmt"], case["M"], case["K"]
    if op == "norm":
        h = torch.randn((M, K), generator=gen, device=DEV)
        h[:, torch.randint(0, K, (max(1, K // 100),), generator=gen, device=DEV)] *= 30  # outlier columns
        s["h"] = h.bfloat16()
        s["residual"] = (torch.randn((M, K), generator=gen, device=DEV) * 4).bfloat16()
        s["gamma"] = torch.rand(K, generator=gen, device=DEV) + 0.25  # (1 + w) / s
    elif op == "silu":
        s["gate_up"] = (torch.randn((M, 2 * K), generator=gen, device=DEV) * 2).bfloat16()
        s["inv_s"] = torch.rand(K, generator=gen, device=DEV) + 0.25
    else:
        s["rows"], s["offsets"], s["most"] = _route(case, gen)
        E = case["E"]
        if op == "grouped":
            T = M * case["top"]
            if not case["gather"]:
                s["rows"] = None
            s["q_a"], s["s_a"] = _tokens(M if case["gather"] else T, K, fmt, gen)
            s["q_w"], s["s_w"] = _weights(E, case["N"], K, fmt, gen)
        else:
            s["q_a"], s["s_a"] = _tokens(M, K, fmt, gen)
            s["q_up"], s["s_up"] = _weights(E, 2 * case["I"], K, fmt, gen)
            s["q_down"], s["s_down"] = _weights(E, K, case["I"], fmt, gen)
            s["inv_s"] = torch.rand(case["I"], generator=gen, device=DEV) + 0.25
    return s


# ------------------------------------------------------------------ plain forms


def _f8(q):
    return q.view(torch.float8_e4m3fn)


def _plain_quant(v, fmt):
    """Codes and scales of fp32 values [M, K]."""
    M, K = v.shape
    g = v.view(M, 1, K) if fmt == "i8" else v.view(M, K // 128, 128)
    top = 448.0 if fmt == "fp8" else 127.0
    amax = g.abs().amax(dim=2, keepdim=True)
    mult = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    if fmt == "fp8":
        q = (g * mult).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        q = (g * mult).round().clamp(-127, 127).to(torch.int8)
    scale = (amax / top).view(M, -1)
    return q.view(M, K), scale.view(M) if fmt == "i8" else scale


def _plain_norm(s):
    res = (s["h"].float() + s["residual"].float()).bfloat16()
    r32 = res.float()
    # long sums of squares: 64 bits, rounded once
    ms = r32.double().square().sum(dim=1).float() / s["K"]
    r = 1.0 / torch.sqrt(ms + EPS)
    q, scale = _plain_quant((r32 * r[:, None]) * s["gamma"], s["fmt"])
    return res, q, scale, r


def _plain_grouped(q_a, s_a, rows, q_w, s_w, offsets, most, fmt):
    """Every expert's rows padded to the longest, one batched fp32 product."""
    E, N, K = q_w.shape
    T = q_a.shape[0] if rows is None else rows.shape[0]
    lo = offsets[:-1].long()
    at = (lo[:, None] + torch.arange(most, device=DEV)).clamp_(max=T - 1)
    token = at if rows is None else rows.long()[at]
    if fmt == "i8":
        x, w = q_a.float(), q_w.float()
    else:
        x = (_f8(q_a).float().view(-1, K // 128, 128) * s_a[:, :, None]).view(-1, K)
        w = (_f8(q_w).float().view(E, N // 128, 128, K // 128, 128)
             * s_w[:, :, None, :, None]).view(E, N, K)
    y = torch.bmm(x[token], w.transpose(1, 2))
    if fmt == "i8":
        y = (y * s_a[token][:, :, None]) * s_w[:, None, :]
    t = torch.arange(T, device=DEV)
    e = torch.searchsorted(offsets[1:].long(), t, right=True)
    return y[e, t - lo[e]].bfloat16()


def _plain_silu(gate_up, inv_s, fmt):
    K = gate_up.shape[1] // 2
    g, u = gate_up[:, :K].float(), gate_up[:, K:].float()
    return _plain_quant((g / (1.0 + torch.exp(-g)) * u) * inv_s, fmt)


def _plain(s):
    op, fmt = s["op"], s["fmt"]
    if op == "norm":
        return _plain_norm(s)
    if op == "silu":
        return _plain_silu(s["gate_up"], s["inv_s"], fmt)
    if op == "grouped":
        return _plain_grouped(s["q_a"], s["s_a"], s["rows"], s["q_w"], s["s_w"], s["offsets"],
                              s["most"], fmt)
    up = _plain_grouped(s["q_a"], s["s_a"], s["rows"], s["q_up"], s["s_up"], s["offsets"],
                        s["most"], fmt)
    q, sc = _plain_silu(up, s["inv_s"], fmt)
    return _plain_grouped(q.view(torch.uint8) if fmt == "fp8" else q, sc, None, s["q_down"],
                          s["s_down"], s["offsets"], s["most"], fmt)


# --------------------------------------------------------- the framework's calls


def _calls(s):
    import w8a8_int8_quantized_sq_b200 as sq

    op, fmt = s["op"], s["fmt"]
    if op == "norm":
        if fmt == "fp8":
            res, q, scale, r = sq.add_rmsnorm_quant_fp8(s["h"], s["residual"], s["gamma"], EPS)
            return res, _f8(q), scale, r
        return sq.add_rmsnorm_quant(s["h"], s["residual"], s["gamma"], EPS,
                                    group=128 if fmt == "i8_group" else 0)
    if op == "silu":
        q, scale = sq.silu_mul_quant_fp8(s["gate_up"], s["inv_s"])
        return _f8(q), scale
    mm = sq.w8a8_grouped_mm if fmt == "i8" else sq.fp8_block_grouped_mm
    if op == "grouped":
        return mm(s["q_a"], s["s_a"], s["q_w"], s["s_w"], s["offsets"], rows=s["rows"])
    up = mm(s["q_a"], s["s_a"], s["q_up"], s["s_up"], s["offsets"], rows=s["rows"])
    act = sq.silu_mul_quant if fmt == "i8" else sq.silu_mul_quant_fp8
    q, scale = act(up, s["inv_s"])
    return mm(q, scale, s["q_down"], s["s_down"], s["offsets"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------------- work


def _product_work(T, M, N, K, E, active, fmt, gather):
    tokens = (M if gather else T) * (K + (4 if fmt == "i8" else K // 128 * 4))
    weights = active * N * (K + 4) if fmt == "i8" else active * (N * K + N // 128 * (K // 128) * 4)
    index = (4 * T if gather else 0) + 4 * (E + 1)
    return {"bytes": tokens + weights + index + 2 * T * N, "flops": 2 * T * N * K}


def work(case):
    op, fmt, M, K = case["op"], case["fmt"], case["M"], case["K"]
    if op == "norm":
        scales = 4 * M if fmt == "i8" else 4 * M * (K // 128)
        return {"bytes": M * K * 7 + 4 * K + scales + 4 * M, "flops": 10 * M * K}
    if op == "silu":
        return {"bytes": M * K * 5 + 4 * K + 4 * M * (K // 128), "flops": 10 * M * K}
    E, top = case["E"], case["top"]
    T = M * top
    active = E * (1 - (1 - top / E) ** M)  # experts that a step reaches, where all are liked alike
    if op == "grouped":
        return _product_work(T, M, case["N"], K, E, active, fmt, case["gather"])
    width = case["I"]
    a = _product_work(T, M, 2 * width, K, E, active, fmt, True)
    b = _product_work(T, T, K, width, E, active, fmt, False)
    scales = 4 * T if fmt == "i8" else 4 * T * (width // 128)
    return {"bytes": a["bytes"] + b["bytes"] + T * width * 5 + 4 * width + scales,
            "flops": a["flops"] + b["flops"] + 10 * T * width}


# ------------------------------------------------------------------ 64-bit values


def _exact_codes(v, top, per):
    """scale and v / scale of blocks of `per` columns, in 64 bits."""
    M, K = v.shape
    blocks = v.reshape(M, K // per, per)
    scale = blocks.abs().amax(2) / top
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (blocks / safe[:, :, None]).reshape(M, K), scale


def _exact_fp8(v):
    code, scale = _exact_codes(v, 448.0, 128)
    return code.to(torch.float8_e4m3fn), scale


def _exact_product(q_a, s_a, rows, q_w, s_w, offsets, fmt):
    bounds = offsets.tolist()
    E, N, K = q_w.shape
    T = q_a.shape[0] if rows is None else rows.shape[0]
    y = torch.zeros((T, N), dtype=torch.float64, device=DEV)
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        pick = torch.arange(lo, hi, device=DEV) if rows is None else rows[lo:hi].long()
        if fmt == "i8":
            x = q_a[pick].double() * s_a[pick].double()[:, None]
            w = q_w[e].double() * s_w[e].double()[:, None]
        else:
            x = _f8(q_a[pick]).double() * s_a[pick].double().repeat_interleave(128, 1)
            w = (_f8(q_w[e]).double()
                 * s_w[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1))
        y[lo:hi] = x @ w.T
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "norm":
        res = s["h"].double() + s["residual"].double()
        kept = res.bfloat16().double()  # what is normalised is the stored residual
        r = (kept.pow(2).mean(1) + EPS).rsqrt()
        v = kept * r[:, None] * s["gamma"].double()
        if fmt == "fp8":
            q, scale = _exact_fp8(v)
            return res, q, scale, r
        scale = _exact_codes(v, 127.0, case["K"] if fmt == "i8" else 128)[1]
        return res, None, scale[:, 0] if fmt == "i8" else scale, r
    if op == "silu":
        g, u = s["gate_up"].double().chunk(2, dim=1)
        return _exact_fp8(g * torch.sigmoid(g) * u * s["inv_s"].double())
    if op == "grouped":
        return _exact_product(s["q_a"], s["s_a"], s["rows"], s["q_w"], s["s_w"], s["offsets"], fmt)
    up = _exact_product(s["q_a"], s["s_a"], s["rows"], s["q_up"], s["s_up"], s["offsets"], fmt)
    g, u = up.bfloat16().double().chunk(2, dim=1)  # the gate-up product is stored in bf16
    v = g * torch.sigmoid(g) * u * s["inv_s"].double()
    if fmt == "fp8":
        q, scale = _exact_fp8(v)
        q = q.view(torch.uint8)
    else:
        code, scale = _exact_codes(v, 127.0, case["I"])
        q, scale = code.round(), scale[:, 0]
    return _exact_product(q, scale, None, s["q_down"], s["s_down"], s["offsets"], fmt)
