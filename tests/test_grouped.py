"""Products grouped by expert on the GPU, against 64 bits."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from grouped_util import F64, check, decode, gradient, offsets_of, product, random_mx

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)


# rows of the experts, N, K
SIZES = [
    ([1], 8, 8), ([0, 3, 0], 64, 64), ([5, 0, 1, 17], 136, 72), ([128], 128, 128), ([129, 0, 127, 1], 264, 200),
    ([16] * 7, 72, 1000), ([300, 2, 65], 1000, 264), ([0, 0, 0], 16, 32), ([1] * 70 + [0] * 60, 40, 96),
    ([3, 0, 0, 1] * 75, 24, 64), ([0] * 1023 + [2], 16, 40), ([1000, 777], 520, 2816), ([40] * 9, 2816, 704),
    ([2000], 384, 512), ([1], 72, 4096), ([3, 0, 16, 1], 200, 1096), ([64], 1000, 1152), ([17, 0, 40], 136, 2056),
    ([70, 30] * 32, 1408, 1024), ([1, 0] * 32, 1408, 1024),
]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("sizes,N,K", SIZES)
def test_values(sizes, N, K, transpose, out):
    g = gen(len(sizes) + N + K)
    A, E = sum(sizes), len(sizes)
    x, w = normal(g, A, K), normal(g, E, N, K)
    offsets = offsets_of(sizes)
    got = bgq.grouped_matmul(x, w.transpose(1, 2).contiguous() if transpose else w, offsets, transpose=transpose, out_dtype=out)
    assert got.shape == (A, N) and got.dtype is out
    check(got, *product(x, w, offsets), K)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("xm", [False, True])
@pytest.mark.parametrize("sizes,N,K", [(s, n, (k + 31) // 32 * 32) for s, n, k in SIZES])
def test_microscaled_values(sizes, N, K, xm, out):
    g = gen(len(sizes) + N + K)
    A, E = sum(sizes), len(sizes)
    wc, ws = random_mx(g, E, N, K)
    offsets = offsets_of(sizes)
    if xm:
        xc, xs = random_mx(g, A, K)
        x, got = decode(xc, xs), bgq.grouped_matmul(xc, wc, offsets, x_scales=xs, w_scales=ws, out_dtype=out)
    else:
        x = normal(g, A, K)
        got = bgq.grouped_matmul(x, wc, offsets, w_scales=ws, out_dtype=out)
    assert got.shape == (A, N) and got.dtype is out
    check(got, *product(x, decode(wc, ws), offsets), K)


@pytest.mark.parametrize("form", ["bf16", "transposed", "mx", "bf16 mx"])
def test_rows_of_no_expert(form):
    """They are not written, and what they and their neighbours hold touches no other row."""
    g = gen(5)
    sizes, N, K = [4, 0, 131, 20], 72, 96
    first, A = 3, 3 + sum(sizes) + 9
    offsets = offsets_of(sizes, first)
    inside = slice(first, first + sum(sizes))
    out = torch.full((A, N), 7.0, dtype=F32, device="cuda")
    if "mx" in form:
        wc, ws = random_mx(g, 4, N, K)
        kw, w, wv = dict(w_scales=ws), wc, decode(wc, ws)
    else:
        wv = normal(g, 4, N, K)
        kw, w = (dict(transpose=True), wv.transpose(1, 2).contiguous()) if form == "transposed" else ({}, wv)
    x = normal(g, A, K)
    x[:first] = x[inside.stop:] = torch.nan
    x[first + 50] = torch.nan
    xv = x
    if form == "mx":
        xc, xs = bgq.mx_quantize(x)
        x, xv = xc, decode(xc, xs)
        kw["x_scales"] = xs
    assert bgq.grouped_matmul(x, w, offsets, out=out, **kw) is out
    ref, size = product(xv, wv, offsets)
    assert bool((out[:first] == 7).all()) and bool((out[inside.stop:] == 7).all())
    assert bool(out[first + 50].isnan().all())
    good = [r for r in range(inside.start, inside.stop) if r != first + 50]
    check(out[good], ref[good], size[good], K)


@pytest.mark.parametrize("transpose", [False, True])
def test_strides(transpose):
    """Rows of x and out inside wider tensors, w a half of packed rows, columns of rows past the end NaN."""
    g = gen(6)
    sizes, N, K = [30, 1, 200], 136, 104
    A, offsets = sum(sizes), offsets_of(sizes)
    x = torch.full((A, K + 24), torch.nan, dtype=BF, device="cuda")
    x[:, 16:16 + K] = normal(g, A, K)
    rows, cols = (K, N) if transpose else (N, K)
    w = torch.full((3, 2 * rows, cols + 8), torch.nan, dtype=BF, device="cuda")
    w[:, rows:, :cols] = normal(g, 3, rows, cols)
    view = w[:, rows:, :cols]
    out = torch.full((A, N + 40), 3.0, dtype=F32, device="cuda")
    bgq.grouped_matmul(x[:, 16:16 + K], view, offsets, transpose=transpose, out=out[:, 8:8 + N])
    check(out[:, 8:8 + N], *product(x[:, 16:16 + K], view.transpose(1, 2) if transpose else view, offsets), K)
    assert bool((out[:, :8] == 3).all()) and bool((out[:, 8 + N:] == 3).all())


def test_one_matrix_and_repeated_rows():
    g = gen(7)
    x, w = normal(g, 50, 72), normal(g, 40, 72)
    check(bgq.grouped_matmul(x, w, out_dtype=F32), *product(x, w[None], offsets_of([50])), 72)
    check(bgq.grouped_matmul(x, w[None]), *product(x, w[None], offsets_of([50])), 72)
    same = x[:1].expand(50, 72)  # row stride 0
    assert torch.equal(bgq.grouped_matmul(same, w), bgq.grouped_matmul(same.contiguous(), w))
    shared = w[None].expand(2, 40, 72)  # expert stride 0
    assert torch.equal(bgq.grouped_matmul(x, shared, offsets_of([20, 30])), bgq.grouped_matmul(x, w))
    wc, ws = bgq.mx_quantize(normal(g, 40, 64))
    check(bgq.grouped_matmul(x[:, :64], wc, w_scales=ws), *product(x[:, :64], decode(wc, ws)[None], offsets_of([50])), 64)
    assert bgq.grouped_matmul(x[:0], w).shape == (0, 40)


GRADS = [([1], 8, 8), ([0, 3, 0], 64, 64), ([5, 0, 1, 17], 136, 72), ([64, 65, 63, 0, 128], 128, 264), ([300, 2, 65], 1000, 40),
         ([0, 0], 16, 24), ([1] * 70 + [0] * 60, 40, 96), ([1000, 777], 264, 520), ([0] * 1023 + [2], 16, 8),
         ([5000], 72, 200), ([1500, 0, 2500, 3], 136, 128)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("sizes,N,K", GRADS)
def test_gradient_values(sizes, N, K, out):
    g = gen(len(sizes) + N + K)
    A = sum(sizes)
    dy, x = normal(g, A + 5, N), normal(g, A + 5, K)
    dy[:2], x[:2], dy[A + 2:], x[A + 2:] = torch.nan, torch.nan, torch.nan, torch.nan  # of no expert
    offsets = offsets_of(sizes, 2)
    got = bgq.grouped_matmul_dw(dy, x, offsets, out_dtype=out)
    assert got.shape == (len(sizes), N, K) and got.dtype is out
    check(got, *gradient(dy, x, offsets), max(sizes))


def test_gradient_cases_split():
    """The last two of GRADS cut an expert's rows; others do not."""
    need = [bgq.grouped_dw_workspace_bytes(sum(s) + 5, len(s), N, K) for s, N, K in GRADS]
    assert need[-1] > 0 and need[-2] > 0 and not any(need[:6])


def test_gradient_strides_and_no_rows():
    g = gen(8)
    dy, x = normal(g, 90, 200), normal(g, 90, 120)
    offsets = offsets_of([20, 70])
    out = torch.empty(2, 104, 64, dtype=F32, device="cuda")
    bgq.grouped_matmul_dw(dy[:, 48:152], x[:, 24:88], offsets, out=out)
    check(out, *gradient(dy[:, 48:152], x[:, 24:88], offsets), 70)
    one = bgq.grouped_matmul_dw(dy[:, :8], x[:, :8])
    check(one, *gradient(dy[:, :8], x[:, :8], offsets_of([90])), 90)
    out.fill_(5.0)
    empty = bgq.grouped_matmul_dw(dy[:0, 48:152], x[:0, 24:88], offsets_of([0, 0]), out=out)
    assert empty is out and not out.any()


def test_gradients_by_formula_and_by_differences():
    """L = sum (out * c) + sum (out^2) / 2: dL/dx = dL/dout w, dL/dw = dL/dout^T x, and both against differences of L."""
    g = gen(9)
    sizes, N, K = [7, 0, 12], 24, 40
    offsets = offsets_of(sizes)
    A = sum(sizes)
    x, w = normal(g, A, K), normal(g, 3, N, K, std=0.2)
    c = normal(g, A, N)

    def loss(x, w):
        y = product(x, w, offsets)[0]
        return (y * c.to(F64)).sum() + y.square().sum() / 2

    y = bgq.grouped_matmul(x, w, offsets, out_dtype=F32)
    dy = (c.float() + y).to(BF)
    dx = bgq.grouped_matmul(dy, w, offsets, transpose=True, out_dtype=F32)
    dw = bgq.grouped_matmul_dw(dy, x, offsets, out_dtype=F32)
    check(dx, *product(dy, w.transpose(1, 2), offsets), N)
    check(dw, *gradient(dy, x, offsets), max(sizes))
    # dy is rounded to bf16, half a step of 2^-8 a term; L is quadratic, so central differences are exact
    h, half = 2.0 ** -6, 2.0 ** -9 * 2
    for r, k in ((0, 0), (6, 39), (7, 13), (18, 5)):
        d = torch.zeros(A, K, dtype=F64, device="cuda")
        d[r, k] = h
        slope = (loss(x.to(F64) + d, w) - loss(x.to(F64) - d, w)) / (2 * h)
        e = 0 if r < 7 else 2
        room = half * (dy[r].to(F64).abs() * w[e, :, k].to(F64).abs()).sum() + 1e-6
        assert abs(float(dx[r, k]) - float(slope)) <= float(room)
    for e, n, k in ((0, 0, 0), (0, 23, 39), (2, 11, 17)):
        d = torch.zeros(3, N, K, dtype=F64, device="cuda")
        d[e, n, k] = h
        slope = (loss(x, w.to(F64) + d) - loss(x, w.to(F64) - d)) / (2 * h)
        rows = slice(0, 7) if e == 0 else slice(7, 19)
        room = half * (dy[rows, n].to(F64).abs() * x[rows, k].to(F64).abs()).sum() + 1e-6
        assert abs(float(dw[e, n, k]) - float(slope)) <= float(room)
    assert not dw[1].any()


def test_binding_refusals():
    g = gen(10)
    x, w, offsets = normal(g, 20, 64), normal(g, 2, 32, 64), offsets_of([10, 10])
    wc, ws = bgq.mx_quantize(w)
    xc, xs = bgq.mx_quantize(x)
    bad = [
        lambda: bgq.grouped_matmul(x, w), lambda: bgq.grouped_matmul(x, w[0], offsets), lambda: bgq.grouped_matmul(x.float(), w, offsets),
        lambda: bgq.grouped_matmul(x, w.float(), offsets), lambda: bgq.grouped_matmul(x[:, :56], w, offsets),
        lambda: bgq.grouped_matmul(x, w, offsets.long()), lambda: bgq.grouped_matmul(x, w, offsets[:2]),
        lambda: bgq.grouped_matmul(x, w, offsets.cpu()), lambda: bgq.grouped_matmul(x, w, offsets, out_dtype=torch.float16),
        lambda: bgq.grouped_matmul(x, w.transpose(1, 2), offsets, transpose=True),
        lambda: bgq.grouped_matmul(x, w, offsets, out=torch.empty(20, 40, dtype=BF, device="cuda")),
        lambda: bgq.grouped_matmul(x, w, offsets, out=torch.empty(20, 32, dtype=BF, device="cuda"), out_dtype=F32),
        lambda: bgq.grouped_matmul(x, wc, offsets), lambda: bgq.grouped_matmul(x, wc, offsets, w_scales=ws, transpose=True),
        lambda: bgq.grouped_matmul(x, wc, offsets, w_scales=ws[:, :16]), lambda: bgq.grouped_matmul(xc, wc, offsets, w_scales=ws),
        lambda: bgq.grouped_matmul(xc, w, offsets, x_scales=xs), lambda: bgq.grouped_matmul(xc, wc, offsets, x_scales=xs[:10], w_scales=ws),
        lambda: bgq.grouped_matmul(x, wc[:, ::2], offsets, w_scales=ws[:, ::2]),
        lambda: bgq.grouped_matmul_dw(x, x[:10], offsets), lambda: bgq.grouped_matmul_dw(x.float(), x, offsets),
        lambda: bgq.grouped_matmul_dw(x, x, offsets, out=torch.empty(2, 64, 32, dtype=BF, device="cuda")),
        lambda: bgq.mx_quantize(x.half()), lambda: bgq.mx_quantize(x[:, :40]), lambda: bgq.mx_quantize(x[:, :32], glu="gelu"),
        lambda: bgq.mx_quantize(x, glu="relu"), lambda: bgq.mx_quantize(x, codes=xc[:10]), lambda: bgq.mx_quantize(x.t()),
        lambda: bgq.mx_dequantize(xc, xs[:10]), lambda: bgq.mx_dequantize(xc.int(), xs),
        lambda: bgq.mx_dequantize(xc, xs, out=torch.empty(20, 32, dtype=BF, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: bgq.grouped_matmul(x[:, 4:60], w[:, :, 4:60], offsets), lambda: bgq.grouped_matmul(x, w[:, :30], offsets)):
        with pytest.raises(bgq.MoeError):
            call()
