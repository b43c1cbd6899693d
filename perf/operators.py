"""Cases for measuring the operators around the routed expert FFN: the block
norms (before and after a block, with its gate and residual scale), the router
(norm, product and top-k) and the whole mixture-of-experts layer for a few
tokens.  `run` computes each in a plain form of elementary torch operations,
or, where `own` is true, through the library's own entry points.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases
def _norm(name, T, H, *, y="bf16", res="bf16", post=True, gate="channel", scale=1.0, pre=True):
    c = dict(op="norm", T=T, H=H, y=y, res=res, post=post, gate=gate, scale=scale, pre=pre)
    return dict(c, name=name) if name else c


def _router(name, T, E, H, k, *, w="fp32"):
    c = dict(op="router", T=T, E=E, H=H, k=k, w=w)
    return dict(c, name=name) if name else c


def _layer(name, T, E, H, I, k, *, gs=64, bits=4, swiglu=False, w="fp32", gate="channel"):
    c = dict(op="layer", T=T, E=E, H=H, I=I, k=k, gs=gs, bits=bits, swiglu=swiglu, w=w, gate=gate)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token: the launch is all that counts
        _norm("norm_token", 1, 2816),
        # a prompt chunk with sizes that fit no vector width, fp32 stream, token gate
        _norm("norm_odd_fp32", 333, 1001, y="fp32", res="fp32", gate="token", scale=0.75),
        # the prompt chunk of the 16384-assignment workload
        _norm("norm_prefill", 2048, 2816, scale=0.5),
        # many long rows: bound by memory alone
        _norm("norm_large", 16384, 4096, gate="none"),
        # a decode batch with the router's weights kept in fp32
        _router("router_decode", 8, 128, 2816, 8),
        # the prompt chunk of the 4096-assignment workload, bf16 weights
        _router("router_prefill4k", 512, 128, 2816, 8, w="bf16"),
        # the prompt chunk of the 16384-assignment workload
        _router("router_prefill16k", 2048, 128, 2816, 8),
        # many experts and an odd token count
        _router("router_many_experts", 4001, 512, 4096, 8, w="bf16"),
        # small layer, many tokens to an expert, groups of 32
        _layer("layer_small", 13, 8, 256, 128, 2, gs=32, gate="none"),
        # one decoded token
        _layer("layer_token", 1, 128, 2816, 704, 8),
        # the decode workload
        _layer("layer_decode", 8, 128, 2816, 704, 8),
        # the largest batch of the few-token form, 8-bit codes, SwiGLU
        _layer("layer_decode16_8bit", 16, 128, 2816, 768, 8, gs=128, bits=8, swiglu=True, w="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "router", "layer"])
    if op == "norm":
        T = _log_int(rng, 1, 16384)
        H = _log_int(rng, 32, 8192)
        H = min(H, 16384 * 4096 // T)
        y, res = rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"])
        if BYTES[y] + BYTES[res] > 4:
            T = max(1, T // 2)
        post = rng.random() < 0.7
        return _norm(None, T, H, y=y, res=res, post=post, gate=rng.choice(["none", "channel", "token"]),
                     scale=round(rng.uniform(0.25, 2.0), 3), pre=rng.random() < 0.7 or not post)
    if op == "router":
        H = 64 * rng.randint(2, 64)
        E = _log_int(rng, 8, 512)
        T = min(_log_int(rng, 1, 8192), 4001 * 512 * 4096 // (E * H * 2))
        return _router(None, T, E, H, rng.randint(1, min(E, 16)), w=rng.choice(["bf16", "fp32"]))
    while True:
        gs = rng.choice([32, 64, 128])
        step = max(gs, 64)
        H, I = step * rng.randint(2, 4096 // step), step * rng.randint(1, 1536 // step)
        E, T, bits = _log_int(rng, 4, 256), rng.randint(1, 16), rng.choice([4, 8])
        k = rng.randint(1, min(E, 10))
        c = _layer(None, T, E, H, I, k, gs=gs, bits=bits, swiglu=rng.random() < 0.5,
                   w=rng.choice(["bf16", "fp32"]), gate=rng.choice(["none", "channel", "token"]))
        w, top = work(c), work(listed()[-1])
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and E * H * I <= 128 * 2816 * 1024:
            return c


def _touched(c):
    """Expected number of experts that T tokens of k distinct experts touch."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] == "norm":
        row = BYTES[c["y"]] + 2 * BYTES[c["res"]] + (BYTES[c["res"]] if c["pre"] else 0)
        side = 2 * H * ((1 if c["post"] else 0) + (1 if c["pre"] else 0))
        side += {"none": 0, "channel": 4 * H, "token": 4 * T}[c["gate"]]
        return {"bytes": T * H * row + side, "flops": 10 * T * H}
    E, k = c["E"], c["k"]
    router = T * H * 2 + E * H * BYTES[c["w"]]
    if c["op"] == "router":
        return {"bytes": router + T * E * 4 + T * k * 4, "flops": 2 * T * E * H}
    I, gs, bits = c["I"], c["gs"], c["bits"]
    expert = 3 * H * I * bits / 8 + 2 * 2 * 3 * H * I / gs
    return {"bytes": _touched(c) * expert + router + 3 * T * H * 2, "flops": 6 * T * k * H * I + 2 * T * E * H}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _gate(g, kind, T, H):
    if kind == "none":
        return None
    if kind == "channel":
        return 0.5 + 0.3 * _normal(g, H)
    return torch.sigmoid(_normal(g, T, 1))


def _codes(g, E, rows, words):
    return torch.randint(-2**31, 2**31, (E, rows, words), generator=g, device="cuda", dtype=torch.int32)


def _stream(g, T, H, dtype=torch.bfloat16):
    """Rows of a residual stream: some channels much larger than the rest."""
    return (_normal(g, T, H) * (1.0 + 2.0 * _normal(g, H).abs())).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    T, H = c["T"], c["H"]
    s = {"case": dict(c)}
    if c["op"] == "norm":
        s["y"] = _normal(g, T, H, std=3.0, dtype=TYPES[c["y"]])
        s["residual"] = _stream(g, T, H, TYPES[c["res"]])
        s["post"] = (1.0 + 0.2 * _normal(g, H)).bfloat16() if c["post"] else None
        s["gate"] = _gate(g, c["gate"], T, H)
        s["pre"] = (1.0 + 0.2 * _normal(g, H)).bfloat16() if c["pre"] else None
        return s
    E, k = c["E"], c["k"]
    s["x"] = _stream(g, T, H)
    s["router"] = _normal(g, E, H, std=1.5 / math.sqrt(H), dtype=TYPES[c["w"]])
    if c["op"] == "router":
        return s
    I, gs, bits = c["I"], c["gs"], c["bits"]
    s["expert_scale"] = 0.5 + torch.rand(E, generator=g, device="cuda")
    mid, std = (8, 0.02) if bits == 4 else (128, 0.02 / 16)
    for name, rows, cols in (("gateup", 2 * I, H), ("down", H, I)):
        s["w_" + name] = _codes(g, E, rows, cols * bits // 32)
        s["s_" + name] = _normal(g, E, rows, cols // gs, std=std).abs().bfloat16()
        s["b_" + name] = -mid * s["s_" + name]
    s["norm"] = (1.0 + 0.2 * _normal(g, H)).bfloat16()
    s["post"] = (1.0 + 0.2 * _normal(g, H)).bfloat16()
    s["gate"] = _gate(g, c["gate"], T, H)
    s["pre"] = (1.0 + 0.2 * _normal(g, H)).bfloat16()
    if own:  # the handle that a program keeps beside its weights
        import bit_gathered_quantized_amd as bgq
        s["layer"] = bgq.MoeLayer(s["router"], k, s["w_gateup"], s["s_gateup"], s["b_gateup"], s["w_down"],
                                  s["s_down"], s["b_down"], norm_weight=s["norm"], expert_scale=s["expert_scale"],
                                  post_weight=s["post"], pre_weight=s["pre"], swiglu=c["swiglu"], eps=EPS)
    return s


# ------------------------------------------------------------------ plain
def _rms(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _tail(y, residual, post, gate, scale, pre, out_type):
    z = y.float()
    if post is not None:
        z = _rms(z) * post.float()
    if gate is not None:
        z = z * gate
    out = residual.float() * scale + z
    got = {"out": out.to(out_type)}
    if pre is not None:
        got["normed"] = (_rms(out) * pre.float()).to(out_type)
    return got


def _top(logits, k, expert_scale):
    """The k largest in descending order, the lower index first on ties."""
    val, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    p = torch.exp(val - val[:, :1])
    p = p / p.sum(-1, keepdim=True)
    return ids, p if expert_scale is None else p * expert_scale[ids]


def _dequantised(words, scale, bias, bits):
    """fp32 weights [..., rows, cols] of packed codes [..., rows, cols * bits / 32]."""
    shift = torch.arange(0, 32, bits, device=words.device, dtype=torch.int32)
    q = ((words.unsqueeze(-1) >> shift) & (2**bits - 1)).flatten(-2).float()
    q = q.unflatten(-1, (scale.shape[-1], -1))
    return (q * scale.float().unsqueeze(-1) + bias.float().unsqueeze(-1)).flatten(-2)


def _act(v, swiglu):
    if swiglu:
        return v / (1.0 + torch.exp(-v))
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _plain_layer(s):
    c = s["case"]
    T, k, I, bits = c["T"], c["k"], c["I"], c["bits"]
    x = s["x"].float()
    n = _rms(x) * s["norm"].float()
    # the choice of experts is a border: logits in 64 bits
    xd = s["x"].double()
    logits = (xd @ s["router"].double().T) * torch.rsqrt((xd * xd).mean(-1, keepdim=True) + EPS)
    ids, p = _top(logits, k, s["expert_scale"].double())
    flat, p = ids.reshape(-1), p.float()
    rows = n.repeat_interleave(k, 0).unsqueeze(-1)
    w = _dequantised(s["w_gateup"][flat], s["s_gateup"][flat], s["b_gateup"][flat], bits)
    gu = torch.matmul(w, rows).squeeze(-1)
    h = _act(gu[:, :I], c["swiglu"]) * gu[:, I:]
    w = _dequantised(s["w_down"][flat], s["s_down"][flat], s["b_down"][flat], bits)
    y = torch.matmul(w, h.unsqueeze(-1)).squeeze(-1).reshape(T, k, -1)
    f = (y * p.unsqueeze(-1)).sum(1)
    return _tail(f, s["x"], s["post"], s["gate"], 1.0, s["pre"], torch.bfloat16)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _tail(s["y"], s["residual"], s["post"], s["gate"], c["scale"], s["pre"], TYPES[c["res"]])
    if c["op"] == "router":
        x = s["x"].float()
        logits = (x @ s["router"].float().T) * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        # no ids: two logits nearer than 32 bits can tell apart may change places.  The
        # weights, in order of their logits, do not jump when they do.
        return {"logits": logits, "weights": _top(logits, c["k"], None)[1]}
    return _plain_layer(s)


def _library(s):
    import bit_gathered_quantized_amd as bgq
    c = s["case"]
    if c["op"] == "norm":
        got = bgq.block_norm(s["y"], s["residual"], post_weight=s["post"], gate=s["gate"], residual_scale=c["scale"],
                             pre_weight=s["pre"], eps=EPS)
        return {"out": got} if s["pre"] is None else {"out": got[0], "normed": got[1]}
    if c["op"] == "router":
        logits, _, weights = bgq.router_forward(s["x"], s["router"], c["k"], eps=EPS)
        return {"logits": logits, "weights": weights}
    out, normed = s["layer"](s["x"], residual=s["x"], gate=s["gate"])
    return {"out": out, "normed": normed}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64

    def unit(v):
        return v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()

    def finish(y, residual, scale):
        z = y if s["post"] is None else unit(y) * s["post"].to(f64)
        z = z if s["gate"] is None else z * s["gate"].to(f64)
        out = scale * residual.to(f64) + z
        return {"out": out} if s["pre"] is None else {"out": out, "normed": unit(out) * s["pre"].to(f64)}

    if c["op"] == "norm":
        return finish(s["y"].to(f64), s["residual"], c["scale"])
    logits = unit(s["x"].to(f64)) @ s["router"].to(f64).T
    top, ids = logits.topk(c["k"], dim=-1)
    p = torch.softmax(top, -1)
    if c["op"] == "router":
        return {"logits": logits, "weights": p}
    n = unit(s["x"].to(f64)) * s["norm"].to(f64)
    p = p * s["expert_scale"].to(f64)[ids]
    per = 32 // c["bits"]

    def matrix(name, e):
        words = s["w_" + name][e].to(torch.int64) & 0xFFFFFFFF
        cols = words.shape[-1] * per
        q = torch.empty(words.shape[0], cols, dtype=f64, device=words.device)
        for i in range(per):
            q[:, i::per] = ((words // 2 ** (c["bits"] * i)) % 2 ** c["bits"]).to(f64)
        sc = s["s_" + name][e].to(f64).repeat_interleave(c["gs"], -1)
        return sc * q + s["b_" + name][e].to(f64).repeat_interleave(c["gs"], -1)

    f = torch.zeros_like(n)
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (n[t] @ matrix("gateup", e).T).split(c["I"], -1)
        if c["swiglu"]:
            a = gate * torch.sigmoid(gate)
        else:
            a = gate * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate**3))
        f.index_add_(0, t, ((a * up) @ matrix("down", e).T) * p[t, j].unsqueeze(-1))
    return finish(f, s["x"], 1.0)
