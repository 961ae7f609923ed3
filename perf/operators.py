"""Operators of a mixture-of-experts block when it serves: their plain forms and the calls of this package.

Three operators, as a server uses them around and inside the layer:

- ``norm``: the block's entry. The residual is added to the branch's output, the sum is normalised by its root
  mean square and scaled; the 8-bit form adds E4M3 codes with one scale a row (``moe_add_rmsnorm``).
- ``quant``: expert weights to 4 bits with group scales, and back to bf16 values (``moe_quantize_w4``,
  ``moe_dequantize_w4``).
- ``experts``: the whole layer on 4-bit expert weights, from the router to the combined output
  (``moe_layer_forward_w4``).

The 4-bit format. A row of ``cols`` weights is cut into groups of 32, 64 or 128 columns (the last may be shorter). A
group's scale is max|v| / 7 rounded to 5 significant bits (so that code x scale is a bf16 number; 1 where that is
below 2^-126); a code is v / scale rounded to the nearest whole number and held as code + 8 in 4 bits. A row is a
sequence of 32-bit words of 8 columns: columns 0, 2, 4, 6 in bits 0, 4, 8, 12 and columns 1, 3, 5, 7 in bits 16, 20,
24, 28. Scales are bf16, [matrix, group, row].
"""
import math

import torch

own = False

E4M3_MAX = 448.0
ORDER = (0, 4, 1, 5, 2, 6, 3, 7)  # the nibble that holds each of a word's 8 columns
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    mixtral = {"op": "experts", "d": 4096, "f": 14336, "m": 8, "k": 2, "shared": 0, "f_shared": 0, "group": 128,
               "act": "swiglu", "renorm": True}
    dsv2 = {"op": "experts", "d": 2048, "f": 1408, "m": 64, "k": 6, "shared": 2, "f_shared": 1408, "group": 64,
            "act": "swiglu", "renorm": False}
    return [
        # the entry of the block in a decode step of 16 sequences, codes for 8-bit experts
        {"name": "norm_decode", "op": "norm", "rows": 16, "d": 4096, "dtype": "bf16", "residual": True, "codes": True},
        # the same in a prefill of 4096 tokens
        {"name": "norm_prefill", "op": "norm", "rows": 4096, "d": 4096, "dtype": "bf16", "residual": True,
         "codes": True},
        # an fp32 model's norm of an odd width and count, without residual or codes
        {"name": "norm_fp32_odd", "op": "norm", "rows": 8191, "d": 2056, "dtype": "f32", "residual": False,
         "codes": False},
        # the down projections of a large layer quantised while a checkpoint is loaded
        {"name": "quant_down", "op": "quant", "n": 8, "rows": 4096, "cols": 14336, "group": 128},
        # small odd matrices with fine groups and a short last group
        {"name": "quant_odd", "op": "quant", "n": 3, "rows": 264, "cols": 1376, "group": 64},
        # one sequence decoding: two of eight experts are read
        dict(mixtral, name="experts_token", T=1),
        # the decode step of 16 sequences
        dict(mixtral, name="experts_decode", T=16),
        # many small experts and shared ones, 16 sequences
        dict(dsv2, name="experts_decode_fine", T=16),
        # odd sizes: ReLU experts, groups of 32, a width that no tile divides, a batch between decode and prefill
        {"name": "experts_odd", "op": "experts", "T": 173, "d": 2080, "f": 5408, "m": 12, "k": 3, "shared": 0,
         "f_shared": 0, "group": 32, "act": "relu", "renorm": False},
        # a chunk of a prompt
        dict(mixtral, name="experts_chunk", T=506),
        # prefill with many small experts and shared ones
        dict(dsv2, name="experts_prefill_fine", T=2048),
        # prefill with large experts
        dict(mixtral, name="experts_prefill", T=4096),
    ]


def _spread(rng, lo, hi, step=1):
    """A size from lo to hi, even over the logarithm, a multiple of step."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step))


def draw(rng):
    op = rng.choice(["norm", "quant", "experts", "experts", "experts"])
    if op == "norm":
        codes = rng.random() < 0.5
        dtype = "bf16" if codes else rng.choice(["bf16", "f32"])
        d = _spread(rng, 256, 8192, 16 if codes else 8)
        return {"op": op, "rows": _spread(rng, 1, min(16384, (1 << 25) // d)), "d": d, "dtype": dtype,
                "residual": rng.random() < 0.7, "codes": codes}
    if op == "quant":
        cols = _spread(rng, 256, 14336, 32)
        rows = _spread(rng, 256, 8192, 8)
        return {"op": op, "n": _spread(rng, 1, max(1, min(64, (1 << 28) // (rows * cols)))), "rows": rows,
                "cols": cols, "group": rng.choice([32, 64, 128])}
    m = rng.choice([4, 8, 12, 16, 32, 64, 128])
    k = rng.randint(1, min(m, 8))
    d = _spread(rng, 512, 4096, 32)
    f = _spread(rng, 512, max(544, min(14336, 450_000_000 // (m * d))) // 32 * 32, 32)
    shared = rng.choice([0, 0, 1, 2])
    top = max(1, min(4096, int(2.0e12 / (6.0 * d * f * (k + shared)))))
    return {"op": op, "T": _spread(rng, 1, top), "d": d, "f": f, "m": m, "k": k, "shared": shared,
            "f_shared": f if shared else 0, "group": rng.choice([32, 64, 128]),
            "act": rng.choice(["swiglu", "swiglu", "relu"]), "renorm": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, gen, std=1.0):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32).mul_(std)


def _pack(v, group):
    """Codes and scales of one matrix [rows, cols] fp32, as the module's description says."""
    rows, cols = v.shape
    ng = -(-cols // group)
    v = torch.nn.functional.pad(v, (0, ng * group - cols)).view(rows, ng, group)
    mant, ex = torch.frexp(v.abs().amax(2) / 7)
    scale = torch.ldexp(torch.round(mant * 32) / 32, ex)
    scale = torch.where(scale >= 2.0 ** -126, scale, torch.ones_like(scale))
    q = (torch.round(v / scale[:, :, None]) + 8).to(torch.int32).view(rows, -1)[:, :cols].reshape(rows, cols // 8, 8)
    word = torch.zeros(rows, cols // 8, dtype=torch.int32, device=v.device)
    for col, nib in enumerate(ORDER):
        word |= q[:, :, col] << (4 * nib)
    return word.view(torch.uint8), scale.to(torch.bfloat16).t().contiguous()


def _weights(gen, n, rows, cols, group):
    codes = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, -(-cols // group), rows, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        codes[i], scales[i] = _pack(_randn((rows, cols), gen, cols ** -0.5), group)
    return codes, scales


def _inputs(case, seed):
    gen = _generator(seed)
    if case["op"] == "norm":
        dt = TORCH[case["dtype"]]
        shape = (case["rows"], case["d"])
        return {"x": _randn(shape, gen, 0.5).to(dt),
                # a residual stream: rows of unlike sizes, a few large channels
                "residual": (_randn(shape, gen) * torch.exp(_randn((case["rows"], 1), gen, 0.5))
                             * torch.exp(_randn((1, case["d"]), gen, 0.5))).to(dt) if case["residual"] else None,
                "weight": (1 + _randn((case["d"],), gen, 0.2)).to(dt), "eps": 1e-5}
    if case["op"] == "quant":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        w = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
        for i in range(n):
            w[i] = _randn((rows, cols), gen, cols ** -0.5)
        return {"w": w}
    T, d, f, m, k, ns, fs, g = (case[key] for key in ("T", "d", "f", "m", "k", "shared", "f_shared", "group"))
    w_router = _randn((m, d), gen, d ** -0.5).to(torch.bfloat16)
    bias = -0.4 * torch.log(1 + torch.randperm(m, device="cuda", generator=gen).float())
    x = _randn((T + T // 8 + 64, d), gen).to(torch.bfloat16)
    # tokens whose k-th and next logit lie within 1e-3 would be routed by the order of a sum: others in their place
    top = torch.sort(x.double() @ w_router.double().t() + bias.double(), 1, descending=True)[0]
    close = top[:, k - 1] - top[:, k] < 1e-3 if k < m else torch.zeros(len(x), dtype=torch.bool, device="cuda")
    x = x[torch.argsort(close.to(torch.int32), stable=True)[:T]].contiguous()
    s = {"x": x, "w_router": w_router, "bias": bias, "group": g}
    for name, n, rows, cols in (("gate", m, f, d), ("up", m, f, d), ("down", m, d, f), ("sh_gate", ns, fs, d),
                                ("sh_up", ns, fs, d), ("sh_down", ns, d, fs)):
        if n and not (name.endswith("up") and case["act"] == "relu"):
            s[name], s[name + "_scale"] = _weights(gen, n, rows, cols, g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] == "experts":
        import sparse_mixture_experts_08_b200 as moe
        s["cfg"] = moe.make_config(case["T"], case["d"], case["f"], case["m"], case["k"], n_shared=case["shared"],
                                   f_shared=case["f_shared"], act=moe.SWIGLU if case["act"] == "swiglu" else moe.RELU,
                                   renormalize=case["renorm"])
        s["ws"] = moe.w4_workspace(s["cfg"])
    return s


# ---------------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if case["op"] == "norm":
        return _norm_own(s, case) if own else _norm(s, case)
    if case["op"] == "quant":
        return _quant_own(s, case) if own else _quant(s, case)
    return _experts_own(s, case) if own else _experts(s, case)


def _norm_own(s, case):
    import sparse_mixture_experts_08_b200 as moe
    x = s["x"]
    total = torch.empty_like(x) if case["residual"] else None
    y = torch.empty_like(x)
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if case["codes"] else None
    scales = torch.empty(x.shape[0], dtype=torch.float32, device=x.device) if case["codes"] else None
    moe.moe_add_rmsnorm(x, s["residual"], s["weight"], s["eps"], y, sum_out=total, codes=codes, scales=scales)
    out = {"y": y}
    if case["residual"]:
        out["sum"] = total
    if case["codes"]:
        out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scales
    return out


def _norm(s, case):
    x = s["x"].float()
    if case["residual"]:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {"y": y.to(s["x"].dtype)}
    if case["residual"]:
        out["sum"] = x.to(s["x"].dtype)
    if case["codes"]:
        top = y.abs().amax(1)
        scales = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        out["codes"], out["scales"] = (y / scales[:, None]).to(torch.float8_e4m3fn), scales
    return out


def _quant_own(s, case):
    import sparse_mixture_experts_08_b200 as moe
    n, rows, cols = s["w"].shape
    codes = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, -(-cols // case["group"]), rows, dtype=torch.bfloat16, device="cuda")
    values = torch.empty_like(s["w"])
    moe.moe_quantize_w4(s["w"], case["group"], codes, scales)
    moe.moe_dequantize_w4(codes, scales, case["group"], values)
    return {"values": values, "scales": scales}


def _quant(s, case):
    group = case["group"]
    n, rows, cols = s["w"].shape
    ng = -(-cols // group)
    v = s["w"].float()
    if ng * group != cols:
        v = torch.nn.functional.pad(v, (0, ng * group - cols))
    v = v.view(n, rows, ng, group)
    mant, ex = torch.frexp(v.abs().amax(3) / 7)
    scale = torch.ldexp(torch.round(mant * 32) / 32, ex)
    scale = torch.where(scale >= 2.0 ** -126, scale, torch.ones_like(scale))
    values = (torch.round(v / scale[..., None]) * scale[..., None]).to(torch.bfloat16)
    return {"values": values.view(n, rows, ng * group)[:, :, :cols].contiguous(),
            "scales": scale.to(torch.bfloat16).transpose(1, 2).contiguous()}


def _experts_own(s, case):
    import sparse_mixture_experts_08_b200 as moe
    out = torch.empty_like(s["x"])
    moe.moe_layer_forward_w4(s["cfg"], s["x"], s["w_router"], s["bias"], s, out, s["ws"])
    return out


def _unpack(codes, scales, group):
    """One matrix's values [rows, cols] in fp32."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    shift = torch.tensor([4 * nib for nib in ORDER], dtype=torch.int32, device=codes.device)
    q = ((codes.view(torch.int32)[:, :, None] >> shift) & 15).view(rows, cols).float() - 8
    return q * scales.t().float().repeat_interleave(group, 1)[:, :cols]


def _ffn(x, s, pre, e, case):
    w = lambda name: _unpack(s[pre + name][e], s[pre + name + "_scale"][e], case["group"])  # noqa: E731
    h = x @ w("gate").t()
    if case["act"] == "swiglu":
        h = h * torch.sigmoid(h) * (x @ w("up").t())
    else:
        h = torch.relu(h)
    return h @ w("down").t()


def _experts(s, case):
    x = s["x"].float()
    logits = x @ s["w_router"].float().t() + s["bias"]
    chosen = torch.topk(logits, case["k"], 1)[1]
    gate = torch.gather(torch.softmax(logits, 1), 1, chosen)
    if case["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    order = torch.argsort(chosen.reshape(-1), stable=True)
    token, weight = order // case["k"], gate.reshape(-1)[order]
    out = torch.zeros_like(x)
    start = 0
    for e, count in enumerate(torch.bincount(chosen.reshape(-1), minlength=case["m"]).tolist()):
        if count:
            at = token[start:start + count]
            out.index_add_(0, at, _ffn(x[at], s, "", e, case) * weight[start:start + count, None])
            start += count
    for e in range(case["shared"]):
        out += _ffn(x, s, "sh_", e, case)
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------- work, 64 bits

def work(case):
    if case["op"] == "norm":
        n, es = case["rows"] * case["d"], 4 if case["dtype"] == "f32" else 2
        b = n * es * (2 + 2 * case["residual"]) + case["d"] * es
        if case["codes"]:
            b += n + 4 * case["rows"]
        return {"bytes": b, "flops": n * (5 + case["residual"] + 2 * case["codes"])}
    if case["op"] == "quant":
        n = case["n"] * case["rows"] * case["cols"]
        # bf16 weights in; codes and scales are what a program keeps; bf16 values out
        kept = n // 2 + 2 * case["n"] * case["rows"] * -(-case["cols"] // case["group"])
        return {"bytes": 4 * n + kept, "flops": 4 * n}
    T, d, f, m, k, ns, fs, g = (case[key] for key in ("T", "d", "f", "m", "k", "shared", "f_shared", "group"))
    mats = 3 if case["act"] == "swiglu" else 2
    active = m * (1 - (1 - k / m) ** T)  # experts that some token chooses, were all alike
    per = lambda width: mats * d * width * (0.5 + 2.0 / g)  # noqa: E731
    tasks = T * k
    return {"bytes": int(active * per(f) + ns * per(fs) + 2 * m * d + 4 * m + 4 * T * d),
            "flops": 2 * mats * d * (tasks * f + ns * T * fs) + 2 * T * d * m}


def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        r = s["x"].to(f64)
        if s["residual"] is not None:
            r = r.add(s["residual"].to(f64))
        rms = r.pow(2).sum(1).div(case["d"]).add(s["eps"]).sqrt()
        y = r.div(rms[:, None]).mul(s["weight"].to(f64))
        out = {"y": y}
        if case["residual"]:
            out["sum"] = r
        if case["codes"]:
            scale = y.abs().max(1).values.div(E4M3_MAX)
            scale[scale == 0] = 1
            out["scales"] = scale
            # E4M3's grid around v: steps of 2^(e - 3) in [2^e, 2^(e + 1)), of 2^-9 below 2^-6
            v = y / scale[:, None]
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            out["codes"] = torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)
        return out
    if case["op"] == "quant":
        w, g = s["w"], case["group"]
        values, scales = torch.empty(w.shape, dtype=f64, device=w.device), []
        for c0 in range(0, case["cols"], g):
            v = w[:, :, c0:c0 + g].to(f64)
            a = v.abs().max(2).values / 7
            unit = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -1000))) - 4)
            a = torch.round(a / unit) * unit
            a[a < 2.0 ** -126] = 1
            values[:, :, c0:c0 + g] = torch.round(v / a[:, :, None]) * a[:, :, None]
            scales.append(a)
        return {"values": values, "scales": torch.stack(scales, 1)}
    x, T, m, k, g = s["x"].to(f64), case["T"], case["m"], case["k"], case["group"]

    def matrix(name, e):
        b = s[name][e].to(torch.int64)  # four bytes a word, two columns four places apart in each
        rows, cols = b.shape[0], 2 * b.shape[1]
        b = b.view(rows, cols // 8, 4)
        v = torch.empty(rows, cols // 8, 8, dtype=f64, device=b.device)
        v[:, :, 0], v[:, :, 2] = b[:, :, 0] % 16, b[:, :, 0] // 16
        v[:, :, 4], v[:, :, 6] = b[:, :, 1] % 16, b[:, :, 1] // 16
        v[:, :, 1], v[:, :, 3] = b[:, :, 2] % 16, b[:, :, 2] // 16
        v[:, :, 5], v[:, :, 7] = b[:, :, 3] % 16, b[:, :, 3] // 16
        v = v.view(rows, cols) - 8
        for i, c0 in enumerate(range(0, cols, g)):
            v[:, c0:c0 + g] *= s[name + "_scale"][e, i].to(f64)[:, None]
        return v

    def expert(rows, pre, e):
        a = rows.mm(matrix(pre + "gate", e).t())
        if case["act"] == "swiglu":
            a = a / (1 + torch.exp(-a)) * rows.mm(matrix(pre + "up", e).t())
        else:
            a = a.clamp_min(0)
        return a.mm(matrix(pre + "down", e).t())

    z = x.mm(s["w_router"].to(f64).t()) + s["bias"].to(f64)
    p = torch.exp(z - z.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    # the k largest, ties to the lower index
    keep = torch.zeros_like(p).scatter_(1, torch.sort(z, stable=True, dim=1, descending=True)[1][:, :k], 1.0)
    p = p * keep
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    out = torch.zeros(T, case["d"], dtype=f64, device=x.device)
    for e in range(m):
        rows = torch.nonzero(keep[:, e])[:, 0]
        if len(rows):
            out[rows] += p[rows, e][:, None] * expert(x[rows], "", e)
    for e in range(case["shared"]):
        out += expert(x, "sh_", e)
    return out
