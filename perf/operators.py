"""Cases, plain forms and exact values of the W8A8 and mixture-of-experts operators.

Operators (`op` of a case):
  quantize_int8  rows of T to 8-bit codes with one scale per row
  int8_mm        product of two such matrices, scaled per token and channel
  qqmm_int8      the two in one call: x in T against an 8-bit weight
  moe            a whole mixture-of-experts layer: router, experts, weighted sum
  moe_experts    the experts of that layer for given indices and weights

`run` computes the plain form (elementary torch operations in 32 bits) or, with
`own` set, makes the library's calls.  Expert weights are group-quantized in
the library's formats: affine codes of 2..8 bits with a scale and bias per
group, or FP4 (E2M1) codes with E8M0 (group 32) or E4M3 (group 16) scales.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ------------------------------------------------------------------- cases
def _moe(name, op, T, H, I, E, k, fmt, bits, gs, dtype, norm=True, pad=0):
    return {"name": name, "op": op, "T": T, "H": H, "I": I, "E": E, "k": k, "fmt": fmt,
            "bits": bits, "gs": gs, "dtype": dtype, "norm": norm, "pad": pad}


def listed():
    return [
        # a few decode tokens on their way into an 8-bit projection
        {"name": "quantize tokens 7x2048", "op": "quantize_int8", "R": 7, "K": 2048, "dtype": "f16"},
        # the activations of a long prompt (also: a projection's weights, once)
        {"name": "quantize prompt 8192x4096", "op": "quantize_int8", "R": 8192, "K": 4096, "dtype": "bf16"},
        # one decode token through a square projection
        {"name": "int8 mm 1x2048x2048", "op": "int8_mm", "M": 1, "N": 2048, "K": 2048, "dtype": "bf16"},
        # a ragged batch of prompt tokens, output rows of odd length
        {"name": "int8 mm 333x1001x1040", "op": "int8_mm", "M": 333, "N": 1001, "K": 1040, "dtype": "f16"},
        # a prompt through an up projection
        {"name": "int8 mm 8192x8192x2048", "op": "int8_mm", "M": 8192, "N": 8192, "K": 2048, "dtype": "bf16"},
        # a small decode batch through a down projection, x quantized on the way
        {"name": "w8a8 5x2048x8192", "op": "qqmm_int8", "M": 5, "N": 2048, "K": 8192, "dtype": "bf16"},
        # a prompt chunk through a square projection
        {"name": "w8a8 1000x4096x4096", "op": "qqmm_int8", "M": 1000, "N": 4096, "K": 4096, "dtype": "f16"},
        # one token through a layer of many small experts: latency
        _moe("moe 1 token, 8 of 64, 4-bit", "moe", 1, 2048, 768, 64, 8, "affine", 4, 64, "bf16"),
        # a decode batch through the same kind of layer, experts of 1408
        _moe("moe 16 tokens, 8 of 64, 4-bit", "moe", 16, 2048, 1408, 64, 8, "affine", 4, 64, "bf16"),
        # byte-packed 3-bit experts in fp16, weights not renormalised
        _moe("moe 3 tokens, 4 of 16, 3-bit", "moe", 3, 1024, 512, 16, 4, "affine", 3, 32, "f16", norm=False),
        # routing done by the caller, some slots of a padded batch empty
        _moe("experts 11 tokens, 2 of 8, 8-bit", "moe_experts", 11, 2048, 1408, 8, 2, "affine", 8, 128, "bf16", pad=3),
        # FP4 experts, a larger decode batch
        _moe("experts 40 tokens, 2 of 8, fp4", "moe_experts", 40, 2048, 1408, 8, 2, "fp4", 4, 32, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize_int8", "int8_mm", "qqmm_int8", "moe", "moe", "moe_experts"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "quantize_int8":
        return {"op": op, "R": _log(rng, 1, 8192), "K": 16 * _log(rng, 8, 256), "dtype": dtype}
    if op in ("int8_mm", "qqmm_int8"):
        while True:
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 8192),
                 "K": 16 * _log(rng, 8, 512), "dtype": dtype}
            if c["M"] * c["N"] * c["K"] <= 8192 * 8192 * 2048:
                return c
    fmt, bits, gs = rng.choice([("affine", 4, 64), ("affine", 4, 64), ("affine", 4, 32), ("affine", 4, 128),
                                ("affine", 2, 32), ("affine", 3, 64), ("affine", 5, 32), ("affine", 6, 64),
                                ("affine", 8, 64), ("fp4", 4, 32), ("fp4", 4, 16)])
    unit = max(gs, 32)
    while True:
        H, I = unit * _log(rng, 512 // unit, 4096 // unit), unit * _log(rng, 256 // unit, 2816 // unit)
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 64)
        if E * H * I <= 64 * 2048 * 1408 and min(E, T * k) * H * I <= 48 * 2048 * 1408:
            break
    pad = rng.randint(0, T * k // 4) if op == "moe_experts" else 0
    c = _moe("", op, T, H, I, E, k, fmt, bits, gs, dtype, norm=rng.random() < 0.5, pad=pad)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _tokens(g, R, K, dtype):
    """Activations: rows of their own size, a few channels much larger."""
    x = torch.randn((R, K), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((R, 1), generator=g, device=DEV))
    x[:, :: max(1, K // 5)] *= 8.0
    return x.to(dtype)


def _rows_to_int8(x):
    x = x.float()
    s = x.abs().amax(1) / torch.full((x.shape[0],), 127.0, device=x.device)
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), torch.zeros_like(x))
    return q.clamp(-127, 127).to(torch.int8), s


def _pack(codes, bits):
    """Codes [..., K] to a little-endian bit stream [..., K * bits / 8]: eight codes in `bits` bytes."""
    c = codes.to(torch.int64).unflatten(-1, (-1, 8))
    v = (c << (bits * torch.arange(8, device=c.device))).sum(-1, keepdim=True)
    return ((v >> (8 * torch.arange(bits, device=c.device))) & 255).to(torch.uint8).flatten(-2)


def _quantized(g, E, N, K, fmt, bits, gs, dtype):
    """Expert weights N(0, 0.02) in the library's format: (w_q, scales, biases)."""
    parts = []
    for _ in range(E):
        w = (torch.randn((N, K // gs, gs), generator=g, device=DEV) * 0.02).to(dtype).float()
        if fmt == "affine":
            lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
            s = ((hi - lo) / (2 ** bits - 1)).clamp_min(1e-7).to(dtype).float()
            b = lo.to(dtype).float()
            q = torch.round((w - b) / s).clamp(0, 2 ** bits - 1)
            parts.append((_pack(q.flatten(-2), bits), s[..., 0].to(dtype), b[..., 0].to(dtype)))
        else:
            s = w.abs().amax(-1, keepdim=True) / 6
            if gs == 32:
                byte = (torch.round(torch.log2(s)) + 127).clamp(1, 254).to(torch.int32)
                sv, byte = (byte << 23).view(torch.float32), byte.to(torch.uint8)
            else:
                byte = s.to(torch.float8_e4m3fn)
                sv, byte = byte.float().clamp_min(2.0 ** -9), byte.view(torch.uint8)
            mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
            q = torch.bucketize((w / sv).abs(), mid) + 8 * (w < 0)
            parts.append((_pack(q.flatten(-2), 4), byte[..., 0], None))
    return tuple(None if p[0] is None else torch.stack(p) for p in zip(*parts))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, dtype = dict(case), DT[case["dtype"]]
    op = c["op"]
    if op == "quantize_int8":
        return {"case": c, "x": _tokens(g, c["R"], c["K"], dtype)}
    if op in ("int8_mm", "qqmm_int8"):
        w_q, w_s = _rows_to_int8(_normal(g, (c["N"], c["K"]), 0.02, dtype))
        x = _tokens(g, c["M"], c["K"], dtype)
        if op == "qqmm_int8":
            return {"case": c, "x": x, "w_q": w_q, "w_s": w_s}
        x_q, x_s = _rows_to_int8(x)
        return {"case": c, "x_q": x_q, "x_s": x_s, "w_q": w_q, "w_s": w_s}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    f = (c["fmt"], c["bits"], c["gs"], dtype)
    st = {"case": c, "x": _normal(g, (T, H), 1.0, dtype),
          "gate": _quantized(g, E, I, H, *f), "up": _quantized(g, E, I, H, *f),
          "down": _quantized(g, E, H, I, *f)}
    if op == "moe":
        st["w_router"] = _normal(g, (E, H), 2.0 / math.sqrt(H), dtype)
    else:
        l = torch.randn((T, E), generator=g, device=DEV)
        top = torch.sort(l, dim=1, descending=True, stable=True)
        st["indices"] = top.indices[:, :k].to(torch.int32).contiguous()
        st["weights"] = torch.softmax(top.values[:, :k], 1).contiguous()
        if c["pad"]:
            at = torch.randperm(T * k, generator=g, device=DEV)[: c["pad"]]
            st["indices"].view(-1)[at] = -1
    return st


# ------------------------------------------------------------ plain forms
def _unpack(w_q, bits):
    if 8 % bits == 0:
        at = torch.arange(0, 8, bits, device=w_q.device, dtype=torch.uint8)
        return ((w_q[..., None] >> at) & (2 ** bits - 1)).flatten(-2)
    b = w_q.unflatten(-1, (-1, bits)).to(torch.int64)
    v = (b << (8 * torch.arange(bits, device=b.device))).sum(-1, keepdim=True)
    return ((v >> (bits * torch.arange(8, device=b.device))) & (2 ** bits - 1)).flatten(-2)


def _fp4_scale(byte, gs, dtype):
    if gs == 16:
        return byte.view(torch.float8_e4m3fn).float().to(dtype).float()
    s = byte.to(torch.int32)
    return torch.where(s == 0, 0x00400000, s << 23).view(torch.float32).to(dtype).float()


def _dequantize(m, pick, c, dtype):
    """The matrices `pick` of a stack in 32 bits: [P, N, K]."""
    w_q, s, b = (None if t is None else t if pick is None else t[pick] for t in m)
    q = _unpack(w_q, c["bits"]).unflatten(-1, (-1, c["gs"]))
    if c["fmt"] == "affine":
        w = q.float() * s.float()[..., None] + b.float()[..., None]
    else:
        v = torch.tensor(LUT + tuple(-t for t in LUT), device=q.device)[q.long()]
        w = v * _fp4_scale(s, c["gs"], dtype)[..., None]
    return w.flatten(-2)


def _experts(st, indices, weights):
    c, x = st["case"], st["x"]
    T, H, I, E, k, dtype = c["T"], c["H"], c["I"], c["E"], c["k"], st["x"].dtype
    ok = (indices >= 0) & (indices < E)
    at, w = indices.long().clamp(0, E - 1), torch.where(ok, weights, torch.zeros_like(weights))
    xf = x.float()
    if T * k < E:      # each slot's own matrices
        pick = at.flatten()
        xr = xf.repeat_interleave(k, 0)[:, :, None]
        g = torch.bmm(_dequantize(st["gate"], pick, c, dtype), xr)
        u = torch.bmm(_dequantize(st["up"], pick, c, dtype), xr)
        h = g / (1 + torch.exp(-g)) * u
        o = torch.bmm(_dequantize(st["down"], pick, c, dtype), h).view(T, k, H)
        return (o * w[:, :, None]).sum(1).to(dtype)
    # every expert for every token, weighted by the slots that chose it
    g = (xf @ _dequantize(st["gate"], None, c, dtype).view(E * I, H).T).view(T, E, I)
    u = (xf @ _dequantize(st["up"], None, c, dtype).view(E * I, H).T).view(T, E, I)
    wt = torch.zeros((T, E), device=x.device).scatter_add(1, at, w)
    h = g / (1 + torch.exp(-g)) * u * wt[:, :, None]
    d = _dequantize(st["down"], None, c, dtype).transpose(1, 2).reshape(E * I, H)
    return (h.view(T, E * I) @ d).to(dtype)


def _route(st):
    # in 64 bits: the order of two near logits decides which expert runs
    l = st["x"].double() @ st["w_router"].double().T
    top = torch.sort(l, dim=1, descending=True, stable=True)
    k = st["case"]["k"]
    p = torch.softmax(top.values, 1)[:, :k]
    if st["case"]["norm"]:
        p = p / p.sum(1, keepdim=True)
    return top.indices[:, :k].to(torch.int32), p.float()


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import group_wise_affine_quant_b200 as aq
        if op == "quantize_int8":
            return aq.aq_quantize_int8(st["x"])
        if op == "int8_mm":
            return aq.aq_int8_mm(st["x_q"], st["x_s"], st["w_q"], st["w_s"], dtype=DT[c["dtype"]])
        if op == "qqmm_int8":
            return aq.aq_qqmm_int8(st["x"], st["w_q"], st["w_s"])
        if op == "moe":
            return aq.aq_moe(st["x"], st["w_router"], st["gate"], st["up"], st["down"], c["k"],
                             normalize=c["norm"], bits=c["bits"], group_size=c["gs"])
        return aq.aq_moe_experts(st["x"], st["indices"], st["weights"], st["gate"], st["up"],
                                 st["down"], bits=c["bits"], group_size=c["gs"])
    if op == "quantize_int8":
        return _rows_to_int8(st["x"])
    if op in ("int8_mm", "qqmm_int8"):
        x_q, x_s = _rows_to_int8(st["x"]) if op == "qqmm_int8" else (st["x_q"], st["x_s"])
        y = (x_q.float() @ st["w_q"].float().T) * x_s[:, None] * st["w_s"][None, :]
        return y.to(DT[c["dtype"]])
    if op == "moe":
        indices, weights = _route(st)
        return _experts(st, indices, weights), indices, weights
    return _experts(st, st["indices"], st["weights"])


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "quantize_int8":
        n = c["R"] * c["K"]
        return {"bytes": 3 * n + 4 * c["R"], "flops": 4 * n}
    if c["op"] in ("int8_mm", "qqmm_int8"):
        M, N, K = c["M"], c["N"], c["K"]
        x = 2 * M * K if c["op"] == "qqmm_int8" else M * K + 4 * M
        return {"bytes": x + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    slots = T * k - c["pad"]
    experts = E * (1 - (1 - 1 / E) ** slots) if c["op"] == "moe_experts" else E * (1 - (1 - k / E) ** T)
    per = c["bits"] / 8 + (4 if c["fmt"] == "affine" else 1) / c["gs"]
    route = 2 * E * H if c["op"] == "moe" else 0
    return {"bytes": experts * 3 * I * H * per + route + 4 * T * H + 8 * T * k,
            "flops": 6 * slots * I * H + route * T}


# ------------------------------------------------------------------ exact
def _bit(w_q, j):
    return (w_q >> j) & 1


def _matrix64(m, e, c, dtype):
    """Matrix e of a stack in 64 bits, codes read bit by bit."""
    w_q, s = m[0][e], m[1][e]
    bits, gs = c["bits"], c["gs"]
    stream = torch.stack([_bit(w_q, j) for j in range(8)], -1).flatten(1)
    stream = stream.unflatten(1, (-1, bits)).double()
    code = sum(stream[..., j] * 2.0 ** j for j in range(bits))
    if c["fmt"] == "affine":
        s, b = s.double(), m[2][e].double()
        return code * s.repeat_interleave(gs, 1) + b.repeat_interleave(gs, 1)
    sign = torch.where(code >= 8, -1.0, 1.0).double()
    mag = torch.remainder(code, 8)
    ex, man = torch.floor(mag / 2), torch.remainder(mag, 2)
    v = torch.where(ex == 0, man * 0.5, (1 + man / 2) * torch.exp2(ex - 1))
    if gs == 16:
        sv = s.view(torch.float8_e4m3fn).double()
    else:
        sv = torch.exp2(s.double() - 127)
    sv = sv.to(dtype).double()
    return sign * v * sv.repeat_interleave(gs, 1)


def exact(case, seed):
    st = prepare(case, seed)
    c, dtype = case, DT[case["dtype"]]
    op = c["op"]

    def int8_rows(x):
        """Codes (whole numbers of the definition's 32-bit division) and 64-bit scales."""
        peak = torch.maximum(x.double().amax(1), -x.double().amin(1))
        q = torch.round(x.float() / (peak / 127).float().clamp_min(1e-45)[:, None])
        return q.clamp(-127, 127).double(), peak / 127

    if op == "quantize_int8":
        return None, int8_rows(st["x"])[1]
    if op in ("int8_mm", "qqmm_int8"):
        x_q, x_s = int8_rows(st["x"]) if op == "qqmm_int8" else (st["x_q"].double(), st["x_s"].double())
        return torch.mm(x_q * x_s[:, None], (st["w_q"].double() * st["w_s"].double()[:, None]).T)
    x = st["x"].double()
    T, E, k = c["T"], c["E"], c["k"]
    share = torch.zeros((T, E), dtype=torch.float64, device=x.device)
    if op == "moe":
        l = torch.stack([(x * r.double()).sum(1) for r in st["w_router"]], 1)
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        left, chosen = l.clone(), []
        for _ in range(k):
            best = left.argmax(1)
            chosen.append(best)
            left[torch.arange(T, device=x.device), best] = -math.inf
        at = torch.stack(chosen, 1)
        weights = p.gather(1, at)
        if c["norm"]:
            weights = weights / weights.sum(1, keepdim=True)
    else:
        at, weights = st["indices"].long(), st["weights"].double()
    for j in range(k):
        for e in range(E):
            share[:, e] += torch.where(at[:, j] == e, weights[:, j], 0.0)
    y = torch.zeros_like(x)
    for e in range(E):
        rows = torch.nonzero(share[:, e] != 0).flatten()
        if rows.numel() == 0:
            continue
        g = x[rows] @ _matrix64(st["gate"], e, c, dtype).T
        u = x[rows] @ _matrix64(st["up"], e, c, dtype).T
        h = g * torch.sigmoid(g) * u
        y[rows] += share[rows, e][:, None] * (h @ _matrix64(st["down"], e, c, dtype).T)
    return (y, None, weights) if op == "moe" else y
