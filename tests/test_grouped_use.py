"""The grouped products and microscaled values as a program uses them: together after a router, in
captured graphs, on other streams, with offsets that are not in order, past 32-bit addresses."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from grouped_util import F64, U, check, decode, encode, gradient, offsets_of, product, random_mx

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMS = ["bf16", "transposed", "mx", "bf16 mx"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)


def operands(form, g, A, E, N, K):
    """(positional arguments, named ones, x and w in values)."""
    if form in ("bf16", "transposed"):
        x, w = normal(g, A, K), normal(g, E, N, K)
        if form == "bf16":
            return (x, w), {}, x, w
        return (x, w.transpose(1, 2).contiguous()), dict(transpose=True), x, w
    wc, ws = random_mx(g, E, N, K)
    if form == "mx":
        xc, xs = random_mx(g, A, K)
        return (xc, wc), dict(x_scales=xs, w_scales=ws), decode(xc, xs), decode(wc, ws)
    x = normal(g, A, K)
    return (x, wc), dict(w_scales=ws), x, decode(wc, ws)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 128, 64), (7, 8, 2, 256, 96), (300, 16, 4, 192, 160)])
@pytest.mark.parametrize("kind", ["mx", "bf16 mx"])
def test_experts_after_a_router(T, E, k, H, I, kind):
    """Router, order, rows of the experts, both products with the gated values quantised between them.  Each
    step is checked against 64 bits on what the step before it gave, so that no rounding to 4 bits that falls
    to the other side hides an error."""
    g = gen(T + H)
    x, router = normal(g, T, H), normal(g, E, H)
    wg, wd = normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5)
    _, ids, weights = bgq.router_forward(x, router, k)
    order = bgq.sort_build_tiles(ids, E)
    offsets, perm = order["offsets"], order["perm"].long()
    rows = x[perm // k]
    gq, dq = bgq.mx_quantize(wg), bgq.mx_quantize(wd)
    assert all(torch.equal(a, b) for a, b in zip(gq + dq, encode(wg.to(F64)) + encode(wd.to(F64))))
    wgv, wdv = decode(*gq), decode(*dq)
    if kind == "mx":
        rc, rs = bgq.mx_quantize(rows)
        gate_up = bgq.grouped_matmul(rc, gq[0], offsets, x_scales=rs, w_scales=gq[1], out_dtype=F32)
        check(gate_up, *product(decode(rc, rs), wgv, offsets), H)
    else:
        gate_up = bgq.grouped_matmul(rows, gq[0], offsets, w_scales=gq[1], out_dtype=F32)
        check(gate_up, *product(rows, wgv, offsets), H)
    hc, hs = bgq.mx_quantize(gate_up, glu="silu")
    gate, up = gate_up.to(F64).chunk(2, -1)
    h = gate * torch.sigmoid(gate) * up
    # the codes of h, or of a value within 2^-14 of it (sigmoid in fp32)
    low, high = decode(*encode(h * (1 - 2.0 ** -14))), decode(*encode(h * (1 + 2.0 ** -14)))
    hv = decode(hc, hs)
    assert bool(((hv >= torch.minimum(low, high)) & (hv <= torch.maximum(low, high))).all())
    y = bgq.grouped_matmul(hc, dq[0], offsets, x_scales=hs, w_scales=dq[1])
    ref, size = product(hv, wdv, offsets)
    check(y, ref, size, I)
    out = (y.float()[order["inv_perm"].long()].view(T, k, H) * weights[..., None]).sum(1)
    mean = (ref[order["inv_perm"].long()].view(T, k, H) * weights.to(F64)[..., None])
    room = (size[order["inv_perm"].long()].view(T, k, H) * weights.to(F64)[..., None]).sum(1)
    # a rounding of each y, k products and sums in fp32, and y's own sums
    assert bool(((out.to(F64) - mean.sum(1)).abs() <= (2.0 ** -8 * mean.abs()).sum(1) + U * (I + 16 + 2 * k) * room).all())


@pytest.mark.parametrize("T,E,k,H,I", [(5, 4, 2, 64, 40), (200, 8, 2, 128, 72)])
def test_experts_forward_and_backward(T, E, k, H, I):
    """Two products with a square between them, L = sum(y c): the gradients of rows and weights that the
    grouped products give are the ones of the formula in 64 bits (autograd, on what bf16 holds of each step)."""
    g = gen(T)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.int()
    order = bgq.sort_build_tiles(ids, E)
    offsets, A = order["offsets"], T * k
    x, w1, w2, c = normal(g, A, H), normal(g, E, I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5), normal(g, A, H)
    z = bgq.grouped_matmul(x, w1, offsets, out_dtype=F32)
    check(z, *product(x, w1, offsets), H)
    h = (z * z).to(BF)
    y = bgq.grouped_matmul(h, w2, offsets)
    check(y, *product(h, w2, offsets), I)
    dh = bgq.grouped_matmul(c, w2, offsets, transpose=True, out_dtype=F32)
    dw2 = bgq.grouped_matmul_dw(c, h, offsets, out_dtype=F32)
    dz = (2 * z * dh).to(BF)
    dx = bgq.grouped_matmul(dz, w1, offsets, transpose=True, out_dtype=F32)
    dw1 = bgq.grouped_matmul_dw(dz, x, offsets, out_dtype=F32)
    most = int(order["counts"].max())
    hp, zp = h.to(F64).requires_grad_(), dz.to(F64)
    w2p = w2.to(F64).requires_grad_()
    (product(hp, w2p, offsets)[0] * c.to(F64)).sum().backward()
    xp, w1p = x.to(F64).requires_grad_(), w1.to(F64).requires_grad_()
    (product(xp, w1p, offsets)[0] * zp).sum().backward()
    check(dh, hp.grad, product(c, w2.transpose(1, 2), offsets)[1], H)
    check(dw2, w2p.grad, gradient(c, h, offsets)[1], most)
    check(dx, xp.grad, product(dz, w1.transpose(1, 2), offsets)[1], I)
    check(dw1, w1p.grad, gradient(dz, x, offsets)[1], most)


def test_captured_calls():
    """Two graphs, replayed in turn with eager work between, on new values and new offsets in the same memory."""
    g = gen(1)
    sizes, N, K = [130, 0, 7, 40], 264, 288
    A, E = sum(sizes), len(sizes)
    x, w, dy = normal(g, A, K), normal(g, E, N, K), normal(g, A, N)
    big = normal(g, 3000, 64)
    offsets, one = offsets_of(sizes), offsets_of([3000])
    wq = bgq.mx_quantize(w)
    need = bgq.grouped_dw_workspace_bytes(3000, 1, 64, 64)
    assert need > 0
    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def forward():
        xq = bgq.mx_quantize(x)
        return [bgq.grouped_matmul(x, w, offsets), bgq.grouped_matmul(xq[0], wq[0], offsets, x_scales=xq[1], w_scales=wq[1]),
                bgq.grouped_matmul(x, wq[0], offsets, w_scales=wq[1]), bgq.mx_dequantize(*xq)]

    def backward(space):
        return [bgq.grouped_matmul(dy, w, offsets, transpose=True), bgq.grouped_matmul_dw(dy, x, offsets, out_dtype=F32),
                bgq.grouped_matmul_dw(big, big, one, workspace=space, out_dtype=F32)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        forward(), backward(spaces[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in (forward, lambda: backward(spaces[0]), lambda: backward(spaces[1])):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    for turn in range(4):
        n = 177 - 40 * turn
        offsets.copy_(offsets_of([n // 2, 3, n - n // 2 - 3, 0][:E]))
        for t in (x, dy, big):
            t.copy_(normal(gen(10 + turn), *t.shape))
        for o in outs:
            for t in o:
                t.fill_(9.0)
        for graph in graphs:
            graph.replay()
        want = [forward(), backward(None), backward(None)]
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            for p, q in zip(a, b):
                rows = slice(0, n) if p.shape[0] == A and p is not outs[0][3] else slice(None)
                assert torch.equal(p[rows], q[rows])
                if rows.stop:
                    assert bool((p[n:] == 9).all())  # rows of no expert


@pytest.mark.parametrize("form", FORMS)
def test_other_streams_two_at_once(form):
    """Calls on two streams at a time, given and current ones, are bit for bit those on the default stream."""
    g = gen(2)
    sizes = [70, 1, 0, 300, 33]
    offsets = offsets_of(sizes)
    args, kw, _, _ = operands(form, g, sum(sizes), len(sizes), 328, 1056)
    want = bgq.grouped_matmul(*args, offsets, **kw)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(6):
        outs.append(bgq.grouped_matmul(*args, offsets, stream=a, **kw))
        with torch.cuda.stream(b):
            outs.append(bgq.grouped_matmul(*args, offsets, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)


def test_gradients_and_codes_on_two_streams():
    g = gen(3)
    dy, x, offsets = normal(g, 4000, 136), normal(g, 4000, 128), offsets_of([1500, 0, 2500])
    want, codes = bgq.grouped_matmul_dw(dy, x, offsets), bgq.mx_quantize(x)
    need = bgq.grouped_dw_workspace_bytes(4000, 3, 136, 128)
    assert need > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in streams]  # NaN, whatever it held
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s, ws in zip(streams, spaces):
            outs.append((bgq.grouped_matmul_dw(dy, x, offsets, workspace=ws, stream=s), bgq.mx_quantize(x, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(want, d) and torch.equal(codes[0], q[0]) and torch.equal(codes[1], q[1]) for d, q in outs)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_of_another_device():
    x, w = normal(gen(4), 40, 64).to("cuda:1"), normal(gen(5), 24, 64).to("cuda:1")
    with torch.cuda.device(0):
        got, q = bgq.grouped_matmul(x, w), bgq.mx_quantize(x)
        assert got.device == x.device == q[0].device
        assert torch.equal(got.cpu(), bgq.grouped_matmul(x.to("cuda:0"), w.to("cuda:0")).cpu())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("A,E,N,K", [(700, 5, 200, 96), (12, 9, 72, 1024), (40, 6, 264, 288)])
def test_offsets_out_of_order(form, A, E, N, K):
    """Rows may be missing or wrong, but nothing outside out is written and nothing outside x and w read."""
    g = gen(A + N)
    args, kw, _, _ = operands(form, g, A, E, N, K)
    around = torch.full((A + 400, N), 5.0, dtype=F32, device="cuda")
    out = around[200:200 + A]
    for seed in range(8):
        c = torch.Generator().manual_seed(seed)
        offsets = torch.randint(-3, A + 3, (E + 1,), generator=c)
        offsets[torch.randint(0, E + 1, (2,), generator=c)] = torch.tensor([2 ** 31 - 1, -2 ** 31])
        bgq.grouped_matmul(*args, offsets.int().cuda(), out=out, **kw)
        assert bool((around[:200] == 5).all()) and bool((around[200 + A:] == 5).all())
        assert bool(out.isfinite().all())
        if form == "bf16":
            dw = bgq.grouped_matmul_dw(out.to(BF), args[0], offsets.int().cuda(), out_dtype=F32)
            assert bool(dw.isfinite().all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("A,E,N,K,starts", [(3, 1, 64, 1024, None), (32, 128, 72, 1024, None), (900, 2, 520, 520, [0, 300, 900])])
def test_same_bits_again(form, A, E, N, K, starts):
    K = (K + 31) // 32 * 32
    g = gen(A)
    args, kw, _, _ = operands(form, g, A, E, N, K)
    offsets = torch.tensor(starts or [A * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    first = bgq.grouped_matmul(*args, offsets, out_dtype=F32, **kw)
    for _ in range(5):
        assert torch.equal(first, bgq.grouped_matmul(*args, offsets, out_dtype=F32, **kw))


# more of w than the caches keep, rows few and many; codes of many rows an expert
@pytest.mark.parametrize("form,sizes,N,K", [
    ("bf16", [1] * 64, 1408, 1024), ("transposed", [1] * 64, 1408, 1024), ("transposed", [70, 30] * 32, 1408, 1024),
    ("mx", [1, 0] * 96, 1408, 2048), ("bf16 mx", [2, 0] * 96, 1408, 2048), ("mx", [40, 9] * 48, 1408, 2048),
    ("mx", [400, 1], 520, 1056), ("bf16 mx", [300, 200], 264, 416), ("bf16 mx", [250, 300], 72, 96), ("mx", [250, 300], 72, 160),
    ("bf16 mx", [3, 5], 40, 32), ("mx", [3, 5], 40, 32), ("mx", [70] * 3, 1408, 1024),
])
def test_large_weights_and_codes(form, sizes, N, K):
    g = gen(N + K)
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(*args, offsets, **kw), *product(x, w, offsets), K)


@pytest.mark.parametrize("sizes,N,K", [([3, 0, 2], 40, 64), ([200, 70, 5], 136, 96), ([2, 1], 24, 1024)])
def test_scales_at_the_ends(sizes, N, K):
    """Scale bytes from 0 to 255, products of the smallest with the largest; a value's NaN reaches its row or column alone."""
    g = gen(N)
    A, E = sum(sizes), len(sizes)
    offsets = offsets_of(sizes)
    for xb, wb in ((0, 254), (254, 0), (20, 230), (1, 252)):
        xc, wc = random_mx(g, A, K)[0], random_mx(g, E, N, K)[0]
        xs = torch.full((A, K // 32), xb, dtype=torch.uint8, device="cuda")
        ws = torch.full((E, N, K // 32), wb, dtype=torch.uint8, device="cuda")
        got = bgq.grouped_matmul(xc, wc, offsets, x_scales=xs, w_scales=ws, out_dtype=F32)
        check(got, *product(decode(xc, xs), decode(wc, ws), offsets), K)
        x = bgq.mx_dequantize(xc, xs)
        if bool(x.isfinite().all()) and wb < 253:
            check(bgq.grouped_matmul(x, wc, offsets, w_scales=ws, out_dtype=F32), *product(x, decode(wc, ws), offsets), K)
    xc, xs = random_mx(g, A, K)
    wc, ws = random_mx(g, E, N, K)
    xs[1, -1], ws[0, 5, 0] = 255, 255
    xc[1, -16:], wc[0, 5, :16] = 0, 0  # as quantised: all of the block stands for NaN
    got = bgq.grouped_matmul(xc, wc, offsets, x_scales=xs, w_scales=ws, out_dtype=F32)
    nan = torch.zeros(A, N, dtype=torch.bool, device="cuda")
    nan[:sizes[0], 5] = True
    mixed = bgq.grouped_matmul(bgq.mx_dequantize(*random_mx(g, A, K)), wc, offsets, w_scales=ws, out_dtype=F32)
    assert torch.equal(mixed.isnan(), nan)
    nan[1] = True
    assert torch.equal(got.isnan(), nan)
    ref, size = product(decode(xc, xs), decode(wc, ws), offsets)
    check(got[~nan], ref[~nan], size[~nan], K)


# many rows: 448 tiles of 256 x 256 and more, 512 rows an expert and more
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("form", ["bf16", "transposed", "mx"])
@pytest.mark.parametrize("sizes,N,K", [([9001, 0, 6970], 2040, 288), ([14000], 2056, 160), ([3, 6000, 0, 5000, 70, 1, 300, 257, 4500], 1784, 1056)])
def test_many_rows(sizes, N, K, form, out):
    g = gen(N + K)
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    assert sum(sizes) >= 512 * len(sizes) and (sum(sizes) // 256 + len(sizes) // 2) * -(-N // 256) >= 448
    check(bgq.grouped_matmul(*args, offsets, out_dtype=out, **kw), *product(x, w, offsets), K)
    if sizes[0] == 9001:  # rows behind the last, offsets that fall
        given = torch.full((sum(sizes), N), 5.0, dtype=out, device="cuda")
        bgq.grouped_matmul(*args, offsets_of([9000, 0, 6000]), out=given, **kw)
        assert bool((given[15000:] == 5).all())
        falling = torch.tensor([20000, 3, 15000, -4], dtype=torch.int32, device="cuda")
        assert bool(bgq.grouped_matmul(*args, falling, out=given, **kw).isfinite().all())


# few rows: wide columns of workgroups (more than 512 narrow ones), their last one in part
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("form", ["bf16", "mx", "bf16 mx"])
@pytest.mark.parametrize("sizes,N,K", [([1] * 8, 1408, 1024), ([64], 4040, 1152), ([3, 0, 17, 1], 2504, 1056), ([0, 2], 4096, 2080)])
def test_few_rows(sizes, N, K, form, out):
    g = gen(N + K)
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(*args, offsets, out_dtype=out, **kw), *product(x, w, offsets), K)


@pytest.mark.parametrize("sizes,K", [([3, 0, 2], 64), ([300, 70], 128), ([2, 1], 1024)])
def test_codes_past_bf16(sizes, K):
    """Against bf16 rows 6 * 2^127 counts as infinity, 1.5 * 2^126 as itself."""
    g = gen(K)
    A, E, N = sum(sizes), len(sizes), 24
    x = normal(g, A, K).abs() + 2.0 ** -6
    codes = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    codes[0, 5, 0], codes[0, 6, 3], codes[0, 7, K // 2 - 1] = 0x07, 0xF0, 0x03
    scales = torch.full((E, N, K // 32), 254, dtype=torch.uint8, device="cuda")
    scales[0, 7] = 253
    got = bgq.grouped_matmul(x * 2.0 ** -10, codes, offsets_of(sizes), w_scales=scales, out_dtype=F32)
    n = sizes[0]
    assert bool((got[:n, 5] == torch.inf).all()) and bool((got[:n, 6] == -torch.inf).all())
    assert torch.equal(got[:n, 7].to(F64), x[:n, K - 2].to(F64) * 1.5 * 2.0 ** 116)
    got[:n, 5:8] = 0
    assert not got.any()


@pytest.mark.parametrize("sizes,N,K", [([3, 0, 2], 40, 64), ([200, 70, 5], 136, 96), ([2, 1], 24, 1024)])
def test_subnormal_and_not_finite_bf16(sizes, N, K):
    """x of bf16's subnormals against large w; infinities and NaN in a row or column stay there."""
    g = gen(K)
    A, E, offsets = sum(sizes), len(sizes), offsets_of(sizes)
    x = (torch.randint(-127, 128, (A, K), generator=g, device="cuda").double() * 2.0 ** -133).to(BF)
    w = normal(g, E, N, K) * 2.0 ** 120
    dy = normal(g, A, N) * 2.0 ** 120
    for got, ref in ((bgq.grouped_matmul(x, w, offsets, out_dtype=F32), product(x, w, offsets)),
                     (bgq.grouped_matmul(x, w.transpose(1, 2).contiguous(), offsets, transpose=True, out_dtype=F32), product(x, w, offsets))):
        check(got, *ref, K)
    check(bgq.grouped_matmul_dw(dy, x, offsets, out_dtype=F32), *gradient(dy, x, offsets), max(sizes))
    x, w = normal(g, A, K), normal(g, E, N, K)
    x[1, 3], w[0, 5, 2] = torch.inf, torch.nan
    bad = torch.zeros(A, N, dtype=torch.bool, device="cuda")
    bad[:sizes[0], 5], bad[1] = True, True
    for got in (bgq.grouped_matmul(x, w, offsets), bgq.grouped_matmul(x, w.transpose(1, 2).contiguous(), offsets, transpose=True)):
        assert bool(got[:sizes[0], 5].isnan().all())
        ref = product(x, w, offsets)[0]
        assert torch.equal(got[1].isnan(), ref[1].isnan()) and torch.equal(got[1].isinf(), ref[1].isinf())
        assert bool(got[~bad].isfinite().all())
    dy, x = normal(g, A, N), normal(g, A, K)
    x[1, 3] = torch.nan
    dw = bgq.grouped_matmul_dw(dy, x, offsets)
    assert bool(dw[0, :, 3].isnan().all()) and int(dw.isnan().sum()) == N


def test_rows_past_32_bits():
    """Rows of x and out 8 and 16 MB apart, experts of w 3 GB apart."""
    g = gen(6)
    A, N, K = 600, 72, 96
    x = torch.empty(A, 1 << 22, dtype=BF, device="cuda")[:, :K]
    x.copy_(normal(g, A, K))
    sizes = [290, 310, 0]
    w = torch.empty(3 * 1500000000, dtype=BF, device="cuda").as_strided((3, N, K), (1500000000, 104, 1))
    w.copy_(normal(g, 3, N, K))
    out = torch.empty(A, 1 << 22, dtype=F32, device="cuda")[:, 8:8 + N]
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(x, w, offsets, out=out), *product(x, w, offsets), K)
    few = offsets_of([0, 0, 40])
    check(bgq.grouped_matmul(x[560:], w, few, out=out[560:]), *product(x[560:], w, few), K)
    turned = w.as_strided((3, K, N), (1500000000, 80, 1))
    turned.copy_(normal(g, 3, K, N))
    check(bgq.grouped_matmul(x, turned, offsets, transpose=True, out=out), *product(x, turned.transpose(1, 2), offsets), K)
    dy = torch.empty(A, 1 << 22, dtype=BF, device="cuda")[:, 64:64 + N]
    dy.copy_(normal(g, A, N))
    check(bgq.grouped_matmul_dw(dy, x, offsets), *gradient(dy, x, offsets), 310)


def test_a_long_sum_past_32_bits():
    """w [K, N] with rows 8 MB apart: one expert's K rows pass 32 bits."""
    g = gen(7)
    K, N = 1000, 40
    w = torch.empty(1, K, 1 << 22, dtype=BF, device="cuda")[:, :, :N]
    w.copy_(normal(g, 1, K, N))
    x = normal(g, 20, K)
    check(bgq.grouped_matmul(x, w, transpose=True), *product(x, w.transpose(1, 2), offsets_of([20])), K)


def test_last_expert_past_32_bits():
    """Codes of 1024 experts, 8 GB, and a gradient of 5 GB: experts at both ends."""
    g = gen(8)
    E, N, K = 1024, 4096, 4096
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    for e in (0, E - 1):
        codes[e], scales[e] = random_mx(g, N, K)
    sizes = torch.zeros(E, dtype=torch.long)
    for n in (3, 200):
        sizes[0] = sizes[-1] = n
        offsets, x = offsets_of(sizes.tolist()), normal(g, 2 * n, K)
        ends = torch.tensor([0, n, 2 * n], dtype=torch.int32)
        pair = decode(codes[[0, E - 1]], scales[[0, E - 1]])
        check(bgq.grouped_matmul(x, codes, offsets, w_scales=scales), *product(x, pair, ends), K)
        xc, xs = random_mx(g, 2 * n, K)
        check(bgq.grouped_matmul(xc, codes, offsets, x_scales=xs, w_scales=scales), *product(decode(xc, xs), pair, ends), K)
    del codes, scales
    dy, x = normal(g, 90, 8192), normal(g, 90, 8192)
    dw = bgq.grouped_matmul_dw(dy, x, offsets_of([40] + [0] * 38 + [50]))
    ends = torch.tensor([0, 40, 90], dtype=torch.int32)
    check(dw[[0, 39]], *gradient(dy, x, ends), 50)
    assert not dw[1].any() and not dw[38].any()


def test_codes_past_32_bits():
    """2^33 values: rows at the start and the end."""
    R, K = 8192 + 8, 1 << 20
    x = torch.zeros(R, K, dtype=BF, device="cuda")
    g = gen(9)
    for r in (0, R - 1):
        x[r] = normal(g, K)
    codes, scales = bgq.mx_quantize(x)
    for r in (0, R - 1):
        want = encode(x[r].to(F64))
        assert torch.equal(codes[r], want[0]) and torch.equal(scales[r], want[1])
    assert not codes[R // 2].any() and not scales[R // 2].any()
    x[R - 1] = 7.0
    bgq.mx_dequantize(codes, scales, out=x)
    assert torch.equal(x[R - 1].to(F64), decode(codes[R - 1], scales[R - 1]))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("A,N,K", [(1, 1 << 20, 32), (2, 16, 1 << 20), (40, 8, 1 << 18)])
def test_longest_dimensions(form, A, N, K):
    g = gen(A)
    args, kw, x, w = operands(form, g, A, 1, N, K)
    for starts in (None, offsets_of([A])):
        check(bgq.grouped_matmul(*args, starts, out_dtype=F32, **kw), *product(x, w, offsets_of([A])), K)


@pytest.mark.parametrize("A,N,K", [(3, 1 << 20, 8), (3, 8, 1 << 20), (70, 8, 1 << 17)])
def test_longest_dimensions_of_a_gradient(A, N, K):
    g = gen(N)
    dy, x = normal(g, A, N), normal(g, A, K)
    check(bgq.grouped_matmul_dw(dy, x), *gradient(dy, x, offsets_of([A])), A)


@pytest.mark.parametrize("form", FORMS)
def test_millions_of_rows(form):
    g = gen(11)
    sizes, N, K = [1, 0, 2000003, 900000], 8, 32
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(*args, offsets, **kw), *product(x, w, offsets), K)


def test_a_gradient_of_millions_of_rows():
    g = gen(12)
    sizes = [1, 0, 2000003, 900000]
    dy, x, offsets = normal(g, sum(sizes), 8), normal(g, sum(sizes), 16), offsets_of(sizes)
    assert bgq.grouped_dw_workspace_bytes(sum(sizes), 4, 8, 16) > 0
    check(bgq.grouped_matmul_dw(dy, x, offsets, out_dtype=F32), *gradient(dy, x, offsets), max(sizes))


@pytest.mark.parametrize("A,N,K", [(1, 72, 1024), (33, 200, 1056), (50, 2504, 1120)])
def test_few_rows_of_one_matrix(A, N, K):
    """Without offsets, rows strided, fp32 rows of out on 16 bytes alone."""
    g = gen(A)
    wide = torch.full((A, K + 40), torch.nan, dtype=BF, device="cuda")
    x = wide[:, 8:8 + K]
    x.copy_(normal(g, A, K))
    w = normal(g, N, K)
    wc, ws = random_mx(g, N, K)
    xc, xs = random_mx(g, A, K)
    out = torch.full((A, N + 12), 3.0, dtype=F32, device="cuda")
    for args, kw, xv, wv in (((x, w), {}, x, w), ((x, wc), dict(w_scales=ws), x, decode(wc, ws)),
                             ((xc, wc), dict(x_scales=xs, w_scales=ws), decode(xc, xs), decode(wc, ws))):
        bgq.grouped_matmul(*args, out=out[:, 4:4 + N], **kw)
        check(out[:, 4:4 + N], *product(xv, wv[None], offsets_of([A])), K)
        assert bool((out[:, :4] == 3).all()) and bool((out[:, 4 + N:] == 3).all())


def test_strided_rows_with_codes():
    g = gen(13)
    sizes, N, K = [200, 3], 136, 416
    x = torch.full((203, K + 16), torch.nan, dtype=BF, device="cuda")[:, 8:8 + K]
    x.copy_(normal(g, 203, K))
    wc, ws = random_mx(g, 2, N, K)
    offsets, one = offsets_of(sizes), x[:1].expand(203, K)
    check(bgq.grouped_matmul(x, wc, offsets, w_scales=ws), *product(x, decode(wc, ws), offsets), K)
    check(bgq.grouped_matmul(one, wc, offsets, w_scales=ws), *product(one, decode(wc, ws), offsets), K)
    w = normal(g, 2, 1, K).expand(2, N, K)  # rows of w all the same, stride 0
    check(bgq.grouped_matmul(x, w, offsets), *product(x, w, offsets), K)
    dy = normal(g, 1, N).expand(203, N)
    check(bgq.grouped_matmul_dw(dy, x, offsets), *gradient(dy, x, offsets), 200)
