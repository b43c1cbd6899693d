"""Cases for measuring the products grouped by expert and the microscaled 4-bit
format: grouped products on bf16 weights (forward, and the gradients of the rows and
of the weights), quantisation to blocks of 32 e2m1 codes under a power-of-two scale,
and grouped products on such weights.  `run` computes each in a plain form of
elementary torch operations, or, where `own` is true, through the library's own
entry points.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
BLOCK = 32


# ------------------------------------------------------------------- cases
def _case(name, **c):
    return dict(c, name=name) if name else c


def _product(name, A, E, N, K, *, transpose=False, out="bf16"):
    return _case(name, op="product", A=A, E=E, N=N, K=K, transpose=transpose, out=out)


def _dw(name, A, E, N, K, *, out="bf16"):
    return _case(name, op="dw", A=A, E=E, N=N, K=K, out=out)


def _quant(name, R, K, *, x="bf16", glu="none"):
    return _case(name, op="quant", R=R, K=K, x=x, glu=glu)


def _mx(name, A, E, N, K, *, x="mx", out="bf16"):
    return _case(name, op="mx", A=A, E=E, N=N, K=K, x=x, out=out)


def listed():
    return [
        # one decoded token's down projection: the latency of a short product
        _product("product_token", 8, 128, 2816, 704, out="fp32"),
        # gate|up of the 16384-assignment workload
        _product("product_prefill16k", 16384, 128, 1408, 2816),
        # gradient of the rows in the 4096-assignment workload, through the gate|up weights
        _product("product_dx_prefill4k", 4096, 128, 2816, 1408, transpose=True),
        # few experts with long, odd runs of rows: bound by the matrix cores
        _product("product_few_experts", 16381, 8, 2816, 4096),
        # gradient of the gate|up weights in the 16384-assignment workload
        _dw("dw_prefill16k", 16384, 128, 1408, 2816),
        # few rows, sizes that fill no tile, fp32 gradients
        _dw("dw_odd_fp32", 333, 5, 264, 1000, out="fp32"),
        # the rows of a prompt chunk before a microscaled product
        _quant("quant_chunk", 2048, 2816),
        # the FFN's intermediate of the 16384-assignment workload: product of the gated halves, then codes
        _quant("quant_glu", 16384, 704, glu="gelu"),
        # the decode workload on microscaled weights: bound by reading them
        _mx("mx_decode", 64, 128, 1408, 2816, x="bf16"),
        # the 4096-assignment workload, rows kept in bf16
        _mx("mx_prefill4k_bf16_rows", 4096, 128, 1408, 2816, x="bf16"),
        # the 16384-assignment workload, both sides microscaled
        _mx("mx_prefill16k", 16384, 128, 1408, 2816),
        # few experts with long, odd runs of rows, both sides microscaled
        _mx("mx_few_experts", 16381, 8, 2816, 4096),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, step * int(round(v / step))))


def draw(rng):
    op = rng.choice(["product", "dw", "quant", "mx"])
    if op == "quant":
        R, K = _log_int(rng, 1, 16384), _log_int(rng, 32, 8192, 32)
        glu = rng.choice(["none", "none", "gelu", "silu"])
        return _quant(None, max(1, min(R, 16384 * 704 // K)), K, x=rng.choice(["bf16", "fp32"]), glu=glu)
    top = {"product": (128 * 1408 * 2816, 16381 * 2816 * 4096), "dw": (128 * 1408 * 2816 // 2, 16384 * 1408 * 2816),
           "mx": (128 * 1408 * 2816, 16381 * 2816 * 4096)}[op]
    step = 32 if op == "mx" else 8
    while True:
        A, E = _log_int(rng, 1, 16384), _log_int(rng, 1, 256)
        N, K = _log_int(rng, 64, 4096, 8), _log_int(rng, 64, 4096, step)
        if E * N * K > top[0] or A * N * K > top[1]:
            continue
        out = rng.choice(["bf16", "bf16", "fp32"])
        if op == "product":
            return _product(None, A, E, N, K, transpose=rng.random() < 0.5, out=out)
        if op == "dw":
            return _dw(None, A, E, N, K, out=out)
        return _mx(None, A, E, N, K, x=rng.choice(["bf16", "mx"]), out=out)


def _touched(c):
    """Expected number of experts that A rows touch."""
    return c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** c["A"])


def work(case):
    c = case
    if c["op"] == "quant":  # rows in; codes, scales and the values they stand for out
        R, K, n = c["R"], c["K"], 1 if c["glu"] == "none" else 2
        return {"bytes": R * K * (n * BYTES[c["x"]] + 17 / 32 + 2), "flops": R * K * (8 if n == 1 else 20)}
    A, E, N, K, out = c["A"], c["E"], c["N"], c["K"], BYTES[c["out"]]
    flops = 2 * A * N * K
    if c["op"] == "dw":
        return {"bytes": 2 * A * (N + K) + E * N * K * out, "flops": flops}
    w, x = (2.0, 2.0) if c["op"] == "product" else (17 / 32, 2.0 if c["x"] == "bf16" else 17 / 32)
    return {"bytes": A * K * x + _touched(c) * N * K * w + A * N * out, "flops": flops}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rows(g, A, K):
    """Rows of activations: some channels much larger than the rest."""
    return (_normal(g, A, K) * (0.5 + _normal(g, K).abs())).bfloat16()


def _weights(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):  # an expert at a time: no fp32 copy of all
        w[e] = _normal(g, N, K, std=1.0 / math.sqrt(K))
    return w


def _sizes(case, seed):
    """Rows of each expert: routing with popular and unpopular experts, some without a row."""
    r = np.random.default_rng(int(seed))
    p = np.exp(0.4 * r.standard_normal(case["E"]))
    return [int(n) for n in r.multinomial(case["A"], p / p.sum())]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(c)}
    if c["op"] == "quant":
        width = c["K"] * (1 if c["glu"] == "none" else 2)
        s["x"] = (_normal(g, c["R"], width) * (0.5 + _normal(g, width).abs())).to(TYPES[c["x"]])
        return s
    A, E, N, K = c["A"], c["E"], c["N"], c["K"]
    s["sizes"] = _sizes(c, seed)
    ends = np.cumsum([0] + s["sizes"])
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["x"] = _rows(g, A, K)
    if c["op"] == "dw":
        s["dy"] = _normal(g, A, N, std=0.02, dtype=torch.bfloat16)
    elif c["op"] == "product":
        s["w"] = _weights(g, E, K, N) if c["transpose"] else _weights(g, E, N, K)
    else:
        s["codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device="cuda")
        for e in range(E):
            s["codes"][e], s["scales"][e] = _quantised(_normal(g, N, K, std=1.0 / math.sqrt(K)))
        if c["x"] == "mx":
            s["x"], s["x_scales"] = _quantised(s["x"])
    return s


# ------------------------------------------------------------------ plain
def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantised(v):
    """Codes [..., K / 2] and scales [..., K / 32] of values [..., K]."""
    v = v.double().unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax)[1].long() - 3, -127).clamp(-127, 127)
    a = v.abs() * _power(-s)
    # nearest code, ties to the even one
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).byte()
    code = (code + 8 * torch.signbit(v).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (s + 127).squeeze(-1).byte()


def _values(codes, scales):
    """fp32 values of codes [..., K / 2] and scales [..., K / 32]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    scale = torch.exp2(scales.double() - 127.0).float().unsqueeze(-1)
    return (v.unflatten(-1, (-1, BLOCK)) * scale).flatten(-2)


def _glu(x, kind):
    """act(g) u of rows [g | u], in 64 bits: codes have borders."""
    g, u = x.double().chunk(2, -1)
    if kind == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u


def _plain(s):
    c = s["case"]
    if c["op"] == "quant":
        x = s["x"] if c["glu"] == "none" else _glu(s["x"], c["glu"])
        return {"values": _values(*_quantised(x)).bfloat16()}
    A, E, N, K, t = c["A"], c["E"], c["N"], c["K"], TYPES[c["out"]]
    at = 0
    if c["op"] == "dw":
        out = torch.zeros(E, N, K, dtype=t, device="cuda")
        for e, n in enumerate(s["sizes"]):
            if n:
                out[e] = s["dy"][at:at + n].float().T @ s["x"][at:at + n].float()
            at += n
        return {"dw": out}
    out = torch.empty(A, N, dtype=t, device="cuda")
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        if c["op"] == "product":
            x, w = s["x"][at:at + n].float(), s["w"][e].float()
            w = w if c["transpose"] else w.T
        else:
            x = s["x"][at:at + n]
            x = x.float() if c["x"] == "bf16" else _values(x, s["x_scales"][at:at + n])
            w = _values(s["codes"][e], s["scales"][e]).T
        out[at:at + n] = x @ w
        at += n
    return {"out": out}


def _library(s):
    import bit_gathered_quantized_amd as bgq
    c = s["case"]
    if c["op"] == "quant":
        codes, scales = bgq.mx_quantize(s["x"], glu=None if c["glu"] == "none" else c["glu"])
        return {"values": bgq.mx_dequantize(codes, scales)}
    t = TYPES[c["out"]]
    if c["op"] == "dw":
        return {"dw": bgq.grouped_matmul_dw(s["dy"], s["x"], s["offsets"], out_dtype=t)}
    if c["op"] == "product":
        return {"out": bgq.grouped_matmul(s["x"], s["w"], s["offsets"], transpose=c["transpose"], out_dtype=t)}
    return {"out": bgq.grouped_matmul(s["x"], s["codes"], s["offsets"], x_scales=s.get("x_scales"),
                                      w_scales=s["scales"], out_dtype=t)}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64

    def decoded(codes, scales):
        n = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int64, device=codes.device)
        n[..., 0::2], n[..., 1::2] = codes % 16, codes // 16
        e, m = n // 2 % 4, (n % 2).to(f64)
        size = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * 2.0 ** (e - 1).to(f64))
        size = torch.where(n < 8, size, -size)
        return size * (2.0 ** (scales.to(f64) - 127.0)).repeat_interleave(BLOCK, -1)

    if c["op"] == "quant":
        x = s["x"].to(f64)
        if c["glu"] != "none":
            g, u = x[:, :c["K"]], x[:, c["K"]:]
            z = g if c["glu"] == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g**3)
            x = g * torch.sigmoid(z) * u
        rows = x.reshape(c["R"], -1, BLOCK)
        top = torch.floor(torch.log2(rows.abs().amax(-1, keepdim=True))) - 2.0
        unit = 2.0 ** top.clamp(-127.0, 127.0)
        a = (rows / unit).abs()
        step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(f64)
        near = (torch.round(a / step) * step).clamp(max=6.0)  # torch rounds halves to even
        return {"values": (torch.sign(rows) * near * unit).reshape(c["R"], c["K"])}
    if c["op"] == "dw":
        out = torch.zeros(c["E"], c["N"], c["K"], dtype=f64, device="cuda")
    else:
        out = torch.empty(c["A"], c["N"], dtype=f64, device="cuda")
    x = s["x"] if c["op"] != "mx" or c["x"] == "bf16" else decoded(s["x"], s["x_scales"])
    edges = s["offsets"].tolist()
    for e in range(c["E"]):
        rows = slice(edges[e], edges[e + 1])
        if edges[e] == edges[e + 1]:
            continue
        if c["op"] == "dw":
            torch.mm(s["dy"][rows].to(f64).t(), x[rows].to(f64), out=out[e])
            continue
        if c["op"] == "mx":
            w = decoded(s["codes"][e], s["scales"][e]).t()
        else:
            w = s["w"][e].to(f64)
            w = w if c["transpose"] else w.t()
        out[rows] = x[rows].to(f64) @ w
    return {"dw" if c["op"] == "dw" else "out": out}
