"""The whole layer (moe_layer_forward, MoeLayer): refusals on the CPU, values on the
GPU against the formulas in 64 bits.

Bounds of the few-token form, u = 2^-24.  n and h are kept as bf16 hi + lo, each
within r = 2^-17 of itself.  A matmul output is off by r sum |W n| from its operand,
and by its fp32 sums: codes enter as 16 + q, so the terms' magnitudes add up to
M = sum_c |n_c| (31 |s_c| + |b_c|) plus the 16 |s_c| |n_c| taken off again, and a
chain of at most 64 products, 2 K / 32 chains, 8 shares rounds each of them at
most 64 + 2 K / 32 + 16 times.  h = act(g) u carries 1.13 |u| dg + |act(g)| du and
2^-20 of itself (hardware exponential and reciprocal).  y sums w_j times that.
The norms and the residual follow as in the block norm.  As a whole (2-norm) a
result without norms is within 3 r + 100 u of itself: n, h and the square root
law for sums."""
import ctypes
import math

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.layer import MoeLayerDesc, MoeNorm

U, R = 2.0 ** -24, 2.0 ** -17
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# --------------------------------------------------------------- refusals
def host_args(p, tail=None, **kw):
    d = MoeLayerDesc(flags=1, router_flags=1, eps=1e-6, router_weight=0x10000, w_gateup=0x10000, s_gateup=0x10000,
                     b_gateup=0x10000, w_down=0x10000, s_down=0x10000, b_down=0x10000)
    for k, v in kw.items():
        setattr(d, k, v)
    n = MoeNorm(T=p.T, H=p.H, residual=0x20000, out=0x30000, normed=0x40000, residual_stride=p.H, out_stride=p.H,
                normed_stride=p.H, eps=1e-6, gate_scale=1.0, residual_scale=1.0)
    for k, v in (tail or {}).items():
        setattr(n, k, v)
    return d, n


def host_call(p, d, n, x=0x50000, ws=0x60000, nbytes=None):
    L = bgq.lib()
    nbytes = L.moe_layer_workspace_bytes(ctypes.byref(p)) if nbytes is None else nbytes
    return L.moe_layer_forward(ctypes.byref(p), None if d is None else ctypes.byref(d), x,
                               None if n is None else ctypes.byref(n), ws, nbytes, None)


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("kw,tail,status", [
    (dict(flags=2), None, -3), (dict(router_flags=4), None, -3), (dict(norm_type=5), None, -3),
    (dict(router_type=5), None, -3), (dict(eps=-1.0), None, -2), (dict(router_weight=None), None, -1),
    (dict(w_gateup=None), None, -1), (dict(b_down=None), None, -1), (dict(router_weight=0x10008), None, -4),
    (dict(norm_weight=0x10008), None, -4), (dict(s_gateup=0x10008), None, -4), (dict(topk_ids=0x10002), None, -4),
    (dict(expert_scale=0x10002), None, -4), ({}, dict(T=5), -2), ({}, dict(H=128), -2), ({}, dict(out=None, normed=None), -1),
    ({}, dict(out=0x30008), -4), ({}, dict(residual_stride=260), -4), ({}, dict(post_weight=0x10002, flags=1), -4),
    ({}, dict(gate=0x10008, gate_stride_h=1), -4), ({}, dict(stream_type=9), -3), ({}, dict(out_stride=8), -2)])
def test_host_checks(T, kw, tail, status):
    p = bgq.problem(T, 2, 8, 256, 128)
    assert host_call(p, *host_args(p, tail, **kw)) == status


def test_host_checks_of_the_problem():
    p = bgq.problem(4, 2, 8, 256, 128)
    d, n = host_args(p)
    assert host_call(p, None, n) == -1 and host_call(p, d, None) == -1 and host_call(p, d, n, x=None) == -1
    assert host_call(p, d, n, x=0x50008) == -4 and host_call(p, d, n, ws=0x60080) == -4
    assert host_call(p, d, n, ws=None) == -5 and host_call(p, d, n, nbytes=64) == -5
    for bad, status in ((bgq.problem(4, 2, 8, 256, 128, bgq.MOE_F_FP32_OUT), -3), (bgq.problem(4, 65, 128, 256, 128), -3),
                        (bgq.problem(4, 2, 8, 256, 128, bits=3), -3), (bgq.problem(4, 2, 8, 4160, 128), -3),
                        (bgq.problem(4, 2, 8, 250, 128), -2)):
        assert bgq.lib().moe_layer_workspace_bytes(ctypes.byref(bad)) == 0
        assert host_call(bad, *host_args(bad), nbytes=1 << 30) == status
    none = bgq.problem(0, 2, 8, 256, 128)
    d, n = host_args(none)
    assert host_call(none, d, n, x=None, ws=None, nbytes=0) == 0


# ----------------------------------------------------------------- values
def make(E, H, I, gs=64, bits=4, wt=F32, seed=0, centred=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = dict(router=(r(E, H) * (1.5 / math.sqrt(H))).to(wt), expert_scale=0.5 + torch.rand(E, generator=g, device="cuda"),
             norm=(1 + 0.2 * r(H)).to(wt), post=(1 + 0.2 * r(H)).bfloat16(), pre=(1 + 0.2 * r(H)).bfloat16())
    mid, std = (8, 0.02) if bits == 4 else (128, 0.02 / 16)
    for name, rows, cols in (("gateup", 2 * I, H), ("down", H, I)):
        w["w_" + name] = torch.randint(-2**31, 2**31, (E, rows, cols * bits // 32), generator=g, device="cuda",
                                       dtype=torch.int32)
        w["s_" + name] = (std * r(E, rows, cols // gs)).abs().bfloat16()
        w["b_" + name] = -mid * w["s_" + name] if centred else (0.05 * r(E, rows, cols // gs)).bfloat16()
    w.update(E=E, H=H, I=I, gs=gs, bits=bits, r=r)
    return w


def layer_of(w, k, **kw):
    return bgq.MoeLayer(w["router"], k, w["w_gateup"], w["s_gateup"], w["b_gateup"], w["w_down"], w["s_down"],
                        w["b_down"], **kw)


def tokens(w, T):
    return (w["r"](T, w["H"]) * (1 + w["r"](w["H"]).abs())).bfloat16()


def dense(w, name, e):
    """(W, magnitude of its terms) of one expert in 64 bits, from the codes byte by byte."""
    bits, gs = w["bits"], w["gs"]
    by = w["w_" + name][e].contiguous().view(torch.uint8)
    q = torch.stack([by & 15, by >> 4], -1).flatten(-2) if bits == 4 else by
    s = w["s_" + name][e].to(F64).repeat_interleave(gs, -1)
    b = w["b_" + name][e].to(F64).repeat_interleave(gs, -1)
    return s * q.to(F64) + b, 47 * s.abs() + b.abs() if bits == 4 else 255 * s.abs() + b.abs()


def reference(w, x, k, ids, *, norm=True, router_norm=True, scaled=True, swiglu=False, eps=1e-6):
    """(logits, weights, y, bound of y) in 64 bits for the chosen ids."""
    xd = x.to(F64)
    rms = (xd.square().mean(-1, keepdim=True) + eps).sqrt()
    logits = (xd / rms if router_norm else xd) @ w["router"].to(F64).T
    p = torch.softmax(torch.gather(logits, 1, ids.long()), -1)
    if scaled:
        p = p * w["expert_scale"].to(F64)[ids.long()]
    n = xd / rms * w["norm"].to(F64) if norm else xd
    dn = n.abs() * (R + (48 * U if norm else 0))
    H, I = w["H"], w["I"]
    y, dy = torch.zeros(x.shape[0], H, dtype=F64, device="cuda"), torch.zeros(x.shape[0], H, dtype=F64, device="cuda")
    cg, cd = U * (80 + H / 16), U * (80 + I / 16)
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        W, M = dense(w, "gateup", e)
        gu = n[t] @ W.T
        dgu = dn[t] @ W.abs().T + cg * (n[t].abs() @ M.T)
        g, u, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
        act = g * torch.sigmoid(g) if swiglu else 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g**3)))
        h = act * u
        dh = 1.13 * u.abs() * dg + act.abs() * du + 1.13 * dg * du + h.abs() * (R + 2.0 ** -20)
        W, M = dense(w, "down", e)
        v = h @ W.T
        dv = dh @ W.abs().T + cd * (h.abs() @ M.T)
        pt = p[t, j].unsqueeze(-1)
        y.index_add_(0, t, pt * v)
        dy.index_add_(0, t, pt * (dv + v.abs() * U * (k + 40)))
    return logits, p, y, dy


def check_routing(logits, ids, weights, p):
    """The ids are those of the largest logits, up to what 32 bits can tell apart."""
    k = ids.shape[1]
    mine = torch.gather(logits, 1, ids.long())
    best = logits.sort(-1, descending=True).values[:, :k]
    assert bool(((mine - best).abs() <= 1e-5).all())
    assert all(len(set(row)) == k for row in ids.tolist())
    assert torch.allclose(weights.double(), p, rtol=1e-4, atol=0)


def run_case(T, E, H, I, k, *, gs=64, bits=4, wt=F32, swiglu=False, norm=True, router_norm=True, scaled=True, centred=True,
             seed=0):
    w = make(E, H, I, gs, bits, wt, seed, centred)
    x = tokens(w, T)
    layer = layer_of(w, k, norm=norm, norm_weight=w["norm"] if norm else None, router_norm=router_norm,
                     expert_scale=w["expert_scale"] if scaled else None, swiglu=swiglu)
    out = torch.empty(T, H, device="cuda")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    weights = torch.empty(T, k, device="cuda")
    # any contents of the workspace
    ws = torch.full((max(layer.workspace_bytes(T), 1),), 0xFF, dtype=torch.uint8, device="cuda")
    layer(x, out=out, ids=ids, weights=weights, workspace=ws)
    torch.cuda.synchronize()
    logits, p, y, dy = reference(w, x, k, ids, norm=norm, router_norm=router_norm, scaled=scaled, swiglu=swiglu)
    check_routing(logits, ids, weights, p)
    err = (out.double() - y).abs()
    worst, rel = float((err / dy).max()), float(torch.linalg.norm(err) / torch.linalg.norm(y))
    print(f"T={T} E={E} H={H} I={I} k={k} gs={gs} bits={bits}: worst error / bound {worst:.3f}, overall {rel:.2e}", flush=True)
    assert worst <= 1.0
    return rel, w, layer, x


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,H,I,k", [
    (1, 1, 64, 64, 1), (1, 8, 256, 128, 2), (5, 8, 256, 128, 2), (13, 4, 320, 192, 3), (16, 2, 64, 64, 2),
    (16, 3, 128, 576, 1), (9, 16, 1088, 320, 5), (16, 40, 640, 1152, 8), (7, 64, 512, 64, 16), (2, 300, 192, 128, 9),
    (16, 1024, 64, 64, 64), (3, 5, 4096, 4096, 2), (16, 6, 2176, 2112, 4)])
@pytest.mark.parametrize("bits", [4, 8])
def test_sizes(T, E, H, I, k, bits):
    rel, *_ = run_case(T, E, H, I, k, bits=bits, seed=T + E)
    assert rel <= 3 * R + 100 * U


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("gs,bits,I", [(64, 4, 704), (128, 8, 768), (32, 4, 704)])
def test_decode_geometry(T, gs, bits, I):
    rel, *_ = run_case(T, 128, 2816, I, 8, gs=gs, bits=bits, seed=T)
    assert rel <= 3 * R + 100 * U


@pytest.mark.gpu
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("swiglu", [False, True])
def test_variants(gs, bits, swiglu):
    """Formats, activations, biases of their own, no norm, no router norm, no expert scale."""
    run_case(6, 12, 640, 384, 3, gs=gs, bits=bits, swiglu=swiglu, centred=False, wt=BF)
    run_case(6, 12, 640, 384, 3, gs=gs, bits=bits, swiglu=swiglu, norm=False, router_norm=False, scaled=False)


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("gate", [None, "channel", "token", 0.5])
def test_tail(stream, gate):
    """Post norm, gate, residual and the next norm around the layer equal the block
    norm of the layer's own output."""
    T, w = 11, make(16, 512, 256, seed=7)
    x = tokens(w, T)
    g = {None: None, "channel": w["r"](512), "token": w["r"](T, 1)}.get(gate, gate)
    res = x.to(stream)
    y = layer_of(w, 4, norm_weight=w["norm"])(x, out=torch.empty(T, 512, device="cuda"))
    want = bgq.block_norm(y, res, post_weight=w["post"], gate=g, residual_scale=0.8, pre_weight=w["pre"])
    layer = layer_of(w, 4, norm_weight=w["norm"], post_weight=w["post"], pre_weight=w["pre"])
    got = layer(x, residual=res, gate=g, residual_scale=0.8)
    for a, b in zip(got, want):
        # the same arithmetic but for the order of the sums of squares (2 * 40 u)
        assert a.dtype is stream
        step = torch.finfo(stream).eps
        assert bool(((a.double() - b.double()).abs() <= (step + 80 * U) * b.double().abs() + 1e-6).all())
    # in place on the residual, which is x itself
    if stream is BF:
        x2 = x.clone()
        out, normed = layer(x2, residual=x2, gate=g, residual_scale=0.8, out=x2)
        assert torch.equal(out, got[0]) and torch.equal(normed, got[1]) and out.data_ptr() == x2.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [17, 100])
@pytest.mark.parametrize("norm", [True, False])
def test_many_tokens_equal_the_operators_in_turn(T, norm):
    w = make(16, 512, 256, seed=8)
    x, gate = tokens(w, T), w["r"](512)
    layer = layer_of(w, 4, norm=norm, norm_weight=w["norm"] if norm else None, expert_scale=w["expert_scale"],
                     post_weight=w["post"], pre_weight=w["pre"])
    ids, weights = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    out, normed = layer(x, residual=x, gate=gate, ids=ids, weights=weights)
    n = bgq.block_norm(x, pre_weight=w["norm"], want_out=False) if norm else x
    _, i, p = bgq.router_forward(x, w["router"], 4, expert_scale=w["expert_scale"])
    assert torch.equal(i, ids) and torch.equal(p, weights)
    y = bgq.expert_ffn_forward(n, i, p, w["w_gateup"], w["s_gateup"], w["b_gateup"], w["w_down"], w["s_down"],
                               w["b_down"], fp32_out=True)
    want = bgq.block_norm(y, x, post_weight=w["post"], gate=gate, pre_weight=w["pre"])
    assert torch.equal(out, want[0]) and torch.equal(normed, want[1])
    again, normed2 = layer(x, residual=x, gate=gate)
    assert torch.equal(again, out) and torch.equal(normed2, normed)


@pytest.mark.gpu
def test_few_and_many_tokens_agree():
    """The first 16 of 40 tokens alone: within the bf16 roundings of n and h of the
    larger batch (2^-9 each at most, three of them, and the output's own)."""
    w = make(32, 704, 320, seed=9)
    x = tokens(w, 40)
    layer = layer_of(w, 4, norm_weight=w["norm"])
    many = layer(x, out=torch.empty(40, 704, device="cuda"))[:16].double()
    few = layer(x[:16].contiguous(), out=torch.empty(16, 704, device="cuda")).double()
    rel = float(torch.linalg.norm(few - many) / torch.linalg.norm(few))
    print(f"few against many tokens: {rel:.2e}")
    assert rel <= 3 * 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 16])
def test_repeats_streams_and_rows(T):
    """The same bits again, on another stream, and in two calls at once with their own
    workspaces; a token's bits do not depend on the order of the tokens."""
    rel, w, layer, x = run_case(T, 64, 1408, 448, 6, seed=10)
    want = layer(x, residual=x)
    torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(layer(x, residual=x), want)
    streams = [torch.cuda.Stream() for _ in range(4)]
    x2 = x.flip(0).contiguous()
    torch.cuda.synchronize()
    got = [layer(x2 if i % 2 else x, residual=x2 if i % 2 else x, stream=streams[i % 4]) for i in range(24)]
    torch.cuda.synchronize()
    assert all(torch.equal(g.flip(0) if i % 2 else g, want) for i, g in enumerate(got))


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T", [1, 11, 16, 40])
def test_in_place(T, norm):
    """out, or normed, is x itself, which is the residual as well."""
    w = make(12, 320, 192, seed=T)
    layer = layer_of(w, 3, norm=norm, norm_weight=w["norm"] if norm else None, post_weight=w["post"], pre_weight=w["pre"])
    x = tokens(w, T)
    out, normed = layer(x, residual=x, gate=w["post"])
    a = x.clone()
    o, n = layer(a, residual=a, gate=w["post"], out=a)
    assert o is a and torch.equal(a, out) and torch.equal(n, normed)
    b = x.clone()
    o, n = layer(b, residual=b, gate=w["post"], normed=b)
    assert n is b and torch.equal(o, out) and torch.equal(b, normed)


@pytest.mark.gpu
def test_same_experts_for_every_token():
    """All tokens alike: each chosen expert has two full tiles, the others none."""
    w = make(24, 256, 192, seed=11)
    x = tokens(w, 1).expand(16, 256).contiguous()
    layer = layer_of(w, 3, norm_weight=w["norm"])
    ids = torch.empty(16, 3, dtype=torch.int32, device="cuda")
    out = layer(x, out=torch.empty(16, 256, device="cuda"), ids=ids)
    assert all(torch.equal(out[0], o) for o in out) and bool((ids == ids[0]).all())
    one = layer(x[:1].contiguous(), out=torch.empty(1, 256, device="cuda"))
    # one token's logits come from the form for one token: the weights' last bits
    assert torch.allclose(out[0].double(), one[0].double(), rtol=0, atol=float(20 * U * out.abs().max()))


@pytest.mark.gpu
def test_ties_zero_and_nan_tokens():
    w = make(10, 256, 128, seed=12)
    w["router"][7] = w["router"][2]
    x = tokens(w, 4)
    x[1] = 0
    x[2, 3] = float("nan")
    layer = layer_of(w, 10, norm_weight=w["norm"], pre_norm=True)
    ids = torch.empty(4, 10, dtype=torch.int32, device="cuda")
    out, normed = layer(x, residual=x, ids=ids)
    order = ids[0].tolist()
    assert order.index(2) + 1 == order.index(7)
    assert ids[1].tolist() == list(range(10))
    assert bool((out[1] == 0).all()) and bool((normed[1] == 0).all())
    assert bool(torch.isnan(out[2]).all()) and sorted(ids[2].tolist()) == list(range(10))
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isfinite(out[3]).all())
    alone = layer(x[3:].contiguous(), residual=x[3:].contiguous())[0]
    assert torch.allclose(alone.float(), out[3:].float(), rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 16, 24])
def test_graph_replays(T):
    w = make(64, 704, 192, seed=13)
    x, k = tokens(w, T), 6
    layer = layer_of(w, k, norm_weight=w["norm"], post_weight=w["post"], pre_weight=w["pre"])
    ws = torch.empty(layer.workspace_bytes(T), dtype=torch.uint8, device="cuda")
    out, normed = torch.empty_like(x), torch.empty_like(x)
    layer(x, residual=x, out=out, normed=normed, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, residual=x, out=out, normed=normed, workspace=ws)
    for rep in range(4):
        x.copy_(tokens(w, T))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = layer(x, residual=x)
        assert torch.equal(out, eager[0]) and torch.equal(normed, eager[1]), rep
        _ = (x.float() * 2).sum()


@pytest.mark.gpu
def test_no_tokens_and_places_outside():
    w = make(8, 256, 128, seed=14)
    layer = layer_of(w, 2, pre_norm=True)
    out, normed = layer(torch.empty(0, 256, dtype=BF, device="cuda"))
    assert out.shape == normed.shape == (0, 256)
    T, big = 6, torch.full((3, 9, 288), 7.0, device="cuda")
    x = tokens(w, T)
    want = layer(x, out=torch.empty(T, 256, device="cuda"), normed=torch.empty(T, 256, device="cuda"))
    view, view2 = big[0, 1:7, 16:272], big[1, 2:8, 0:256]
    layer(x, out=view, normed=view2)
    assert torch.equal(view, want[0]) and torch.equal(view2, want[1])
    view.fill_(7.0)
    view2.fill_(7.0)
    assert bool((big == 7.0).all())
    # the workspace: nothing past its end
    n = layer.workspace_bytes(T)
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    layer(x, workspace=ws[:n])
    assert bool((ws[n:] == 0xA5).all())
    with pytest.raises(bgq.MoeError):
        layer(x, workspace=ws[:n - 256])


@pytest.mark.gpu
def test_binding_refusals():
    w = make(8, 256, 128, seed=15)
    layer, x = layer_of(w, 2), tokens(w, 4)
    bad = [dict(x=x.float()), dict(x=x[:, :128]), dict(x=x.T), dict(residual=x[:3]), dict(gate=torch.zeros(3, device="cuda")),
           dict(out=torch.empty(4, 255, device="cuda")), dict(normed=x.clone()), dict(ids=torch.zeros(4, 2, device="cuda")),
           dict(weights=torch.zeros(4, 3, device="cuda")), dict(workspace=torch.zeros(1 << 20, device="cuda")),
           dict(residual=x.half()), dict(residual=x.float(), out=x.clone())]
    for kw in bad:
        args = dict(x=x)
        args.update(kw)
        with pytest.raises(ValueError):
            layer(args.pop("x"), **args)
    for k, kw in [(9, {}), (0, {}), (2, dict(norm=False, norm_weight=w["norm"])), (2, dict(norm_weight=w["norm"][:100])),
                  (2, dict(expert_scale=w["expert_scale"].double())), (2, dict(post_weight=w["post"], pre_weight=w["pre"].float()))]:
        with pytest.raises(ValueError):
            layer_of(w, k, **kw)
    for name in ("w_gateup", "s_gateup", "b_down", "router"):
        cut = dict(w)
        cut[name] = w[name][:, :-8]
        with pytest.raises(ValueError):
            layer_of(cut, 2)
