"""The whole router (moe_router_forward): refusals on the CPU, values on the GPU.

logits against the product in 64 bits.  Products are exact, so an output is off
by its fp32 sums alone: a chain of L additions of terms that sum to S in
magnitude is within L u S (u = 2^-24).  A thread of the few-token form adds at
most 8 ceil(H / 2048) products, 6 lanes and 4 waves; an MFMA of the tiled form
adds 32 products to its accumulator, ceil(H / 256) times per wave and three
times as often for fp32 weights, then 8 waves.  The mean of squares is within
the same share of itself (half of it in the root), four more roundings follow.
ids and weights against the returned logits: the ids exactly, the weights within
the exponentials (2 u each way), a sum of k, a quotient and a product."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.layer import MOE_R_NORM, MoeRouter

U = 2.0 ** -24


def host_router(**kw):
    r = MoeRouter(T=4, H=256, E=8, k=2, eps=1e-6, x_stride=256, weight=0x10000, flags=MOE_R_NORM)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -2), (dict(H=0), -2), (dict(H=96), -2), (dict(H=16448), -3), (dict(E=0), -2), (dict(E=1025), -3),
    (dict(k=0), -2), (dict(k=9), -2), (dict(E=128, k=65), -3), (dict(weight_type=2), -3), (dict(flags=2), -3),
    (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(x_stride=255), -2), (dict(x_stride=260), -4),
    (dict(x_stride=1 << 23), -2), (dict(weight=None), -1), (dict(weight=0x10008), -4), (dict(expert_scale=0x10002), -4),
    (dict(T=1 << 30, E=8), -2)])
def test_host_checks(kw, status):
    r = host_router(**kw)
    assert bgq.lib().moe_router_forward(ctypes.byref(r), 0x20000, 0x30000, 0x40000, 0x50000, None) == status


def test_host_checks_of_outputs():
    f, r = bgq.lib().moe_router_forward, ctypes.byref(host_router())
    assert f(None, 0x20000, 0x30000, 0x40000, 0x50000, None) == -1
    assert f(r, None, 0x30000, 0x40000, 0x50000, None) == -1
    assert f(r, 0x20000, None, 0x40000, 0x50000, None) == -1
    assert f(r, 0x20000, 0x30000, None, 0x50000, None) == -1
    assert f(r, 0x20000, 0x30000, 0x40000, None, None) == -1
    assert f(r, 0x20008, 0x30000, 0x40000, 0x50000, None) == -4
    assert f(r, 0x20000, 0x30002, 0x40000, 0x50000, None) == -4
    assert f(ctypes.byref(host_router(T=0, weight=None)), None, None, None, None, None) == 0


def make(T, E, H, wt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda") * (1 + torch.randn(H, generator=g, device="cuda").abs())
    w = torch.randn(E, H, generator=g, device="cuda") * (2.0 / math.sqrt(H))
    return x.bfloat16(), w.to(wt), 0.5 + torch.rand(E, generator=g, device="cuda")


def check(x, w, k, scale, got, norm=True, eps=1e-6):
    logits, ids, weights = got
    T, H = x.shape
    xd, wd = x.double(), w.double()
    rstd = torch.rsqrt(xd.square().mean(-1, keepdim=True) + eps) if norm else torch.ones(T, 1, device="cuda").double()
    ref = rstd * (xd @ wd.T)
    size = rstd * (xd.abs() @ wd.abs().T)
    if T <= 8:
        L = 8 * math.ceil(H / 2048) + 10
    else:
        L = 32 * math.ceil(H / 256) * (3 if w.dtype is torch.float32 else 1) + 8
    err, bound = (logits.double() - ref).abs(), U * (L * size + (L / 2 + 4) * ref.abs()) + 1e-30
    # signs are as good as random: the root of the number of roundings for the whole
    rel = float(torch.linalg.norm(err) / torch.linalg.norm(size)) if T else 0.0
    print(f"worst error / bound {float((err / bound).max()):.3f}, overall {rel:.2e} of the terms", flush=True)
    assert bool((err <= bound).all())
    assert rel <= U * math.sqrt(L)
    lo = logits.cpu().numpy()
    order = np.argsort(-lo, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), order)
    chosen = torch.gather(logits.double(), 1, ids.long())
    p = torch.softmax(chosen, -1)
    if scale is not None:
        p = p * scale.double()[ids.long()]
    # exp(l - m) of a rounded difference: |l - m| u more
    spread = (chosen - chosen[:, :1]).abs()
    assert bool(((weights.double() - p).abs() <= U * (k + 12 + 2 * spread) * p + 1e-37).all())


@pytest.mark.gpu
@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H,k", [
    (1, 128, 2816, 8), (2, 8, 256, 2), (3, 1, 64, 1), (5, 128, 4096, 8), (8, 60, 2816, 6), (16, 1000, 704, 64),
    (15, 33, 16384, 5), (17, 128, 2816, 8), (64, 16, 64, 16), (100, 129, 192, 3), (333, 31, 1088, 7),
    (2048, 128, 2816, 8), (2049, 200, 512, 8), (1000, 1024, 256, 10), (70, 8, 16384, 2)])
def test_sizes(wt, T, E, H, k):
    x, w, scale = make(T, E, H, wt)
    check(x, w, k, None, bgq.router_forward(x, w, k))
    check(x, w, k, scale, bgq.router_forward(x, w, k, expert_scale=scale))


@pytest.mark.gpu
@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H,k", [(1037, 1024, 128, 8), (257, 1000, 64, 3), (4201, 128, 192, 8), (8321, 100, 64, 4),
                                     (129, 70, 320, 2)])
def test_large_tiles_and_their_order(wt, T, E, H, k):
    """Batches of the largest tiles, with four and with eight waves, grouped by XCD
    (with blocks past the batch) and not."""
    x, w, scale = make(T, E, H, wt)
    check(x, w, k, None, bgq.router_forward(x, w, k))
    check(x, w, k, scale, bgq.router_forward(x, w, k, expert_scale=scale))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 300])
def test_without_norm_strided_rows_and_given_outputs(T):
    x, w, scale = make(T, 24, 320, torch.float32, seed=3)
    view = x[:, 64:256]  # rows 320 apart, starting on 128 bytes
    wv = w[:, 64:256].contiguous()
    big = torch.full((T + 2, 24), 5.0, device="cuda")
    got = bgq.router_forward(view, wv, 4, norm=False, logits=big[1:T + 1])
    check(view, wv, 4, None, got, norm=False)
    assert bool((big[0] == 5.0).all()) and bool((big[T + 1] == 5.0).all())
    assert got[0].data_ptr() == big[1:].data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 40])
def test_ties_zeros_and_nan(T):
    x, w, _ = make(T, 64, 256, torch.bfloat16, seed=4)
    w[10] = w[3]
    w[50] = w[3]
    x[1] = 0
    x[2, 5] = float("nan")
    logits, ids, weights = bgq.router_forward(x, w, 64)
    assert torch.equal(logits[:, 3], logits[:, 10]) or bool(torch.isnan(logits[2, 3]))
    order = ids[0].tolist()
    assert order.index(3) < order.index(10) < order.index(50)
    assert bool((logits[1] == 0).all()) and ids[1].tolist() == list(range(64))
    assert torch.allclose(weights[1], torch.full((64,), 1 / 64, device="cuda"), rtol=70 * U, atol=0)
    assert bool(torch.isnan(logits[2]).all())  # NaN ranks as -inf: the ids are still experts
    assert sorted(ids[2].tolist()) == list(range(64))


@pytest.mark.gpu
def test_no_tokens_stream_and_graph():
    x, w, scale = make(24, 128, 2816, torch.float32, seed=5)
    e = bgq.router_forward(x[:0], w, 8)
    assert e[0].shape == (0, 128) and e[1].shape == e[2].shape == (0, 8)
    want = bgq.router_forward(x, w, 8, expert_scale=scale)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = bgq.router_forward(x, w, 8, expert_scale=scale, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    outs = [torch.empty_like(t) for t in want]
    with torch.cuda.graph(g):
        bgq.router_forward(x, w, 8, expert_scale=scale, logits=outs[0], ids=outs[1], weights=outs[2])
    for _ in range(3):
        x.copy_(torch.randn(24, 2816, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        eager = bgq.router_forward(x, w, 8, expert_scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


@pytest.mark.gpu
def test_binding_refusals():
    x, w, scale = make(4, 8, 128, torch.bfloat16)
    for args, kw in [((x.float(), w, 2), {}), ((x, w[:, :64].contiguous(), 2), {}), ((x, w.T, 2), {}),
                     ((x, w.half(), 2), {}), ((x, w, 9), {}), ((x, w, 2), dict(expert_scale=scale[:7])),
                     ((x, w, 2), dict(expert_scale=scale.double())),
                     ((x, w, 2), dict(logits=torch.empty(4, 9, device="cuda"))),
                     ((x, w, 2), dict(ids=torch.empty(4, 2, device="cuda"))), ((x[0], w, 2), {})]:
        with pytest.raises(ValueError):
            bgq.router_forward(*args, **kw)
    with pytest.raises(bgq.MoeError):
        bgq.router_forward(x[:, :96].contiguous(), w[:, :96].contiguous(), 2)
