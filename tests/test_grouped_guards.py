"""Grouped products and the weights' gradient with operands amid values that are not finite and results amid marked memory:
offsets in any order, paths that cut an expert's rows or keep a block of x.  What is read beside x, w, dy or their scales
and reaches a result shows as NaN; what is written beside a result changes a mark."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from grouped_util import check, decode, gradient, offsets_of, product, random_mx
from test_grouped_use import FORMS, gen, normal

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 300  # rows


def amid(t, fill, pad=8):
    """t's rows inside a wider and longer tensor of `fill` (pad 0: only longer)."""
    wide = torch.full((t.shape[0] + 2 * GUARD, t.shape[1] + 2 * pad), fill, dtype=t.dtype, device="cuda")
    view = wide[GUARD:GUARD + t.shape[0], pad:pad + t.shape[1]]
    view.copy_(t)
    return view


def weights_amid(w):
    wide = torch.full((w.shape[0] + 2, w.shape[1] + 40, w.shape[2] + 16), torch.nan, dtype=w.dtype, device="cuda")
    view = wide[1:-1, 16:16 + w.shape[1], 8:8 + w.shape[2]]
    view.copy_(w)
    return view


def codes_amid(codes, scales):
    """Codes between codes of 6, scales between NaN's."""
    rows = lambda t, fill: amid(t.flatten(0, -2), fill, 0).view(t.shape)
    return rows(codes, 0x77), rows(scales, 255)


def operands(form, g, A, E, N, K):
    if form in ("bf16", "transposed"):
        x, w = amid(normal(g, A, K), torch.nan), normal(g, E, N, K)
        if form == "bf16":
            return (x, weights_amid(w)), {}, x, w
        return (x, weights_amid(w.transpose(1, 2))), dict(transpose=True), x, w
    wc, ws = codes_amid(*random_mx(g, E, N, K))
    if form == "mx":
        xc, xs = codes_amid(*random_mx(g, A, K))
        return (xc, wc), dict(x_scales=xs, w_scales=ws), decode(xc, xs), decode(wc, ws)
    x = amid(normal(g, A, K), torch.nan)
    return (x, wc), dict(w_scales=ws), x, decode(wc, ws)


class Marked:
    """A result inside memory of ones that no call writes."""

    def __init__(self, *shape, dtype, pad=0):
        last = shape[-1] + 2 * pad
        lead = shape[0] + 2 * GUARD if len(shape) == 2 else shape[0] + 2
        self.all = torch.full((lead,) + shape[1:-1] + (last,), 1.0, dtype=dtype, device="cuda")
        skip = GUARD if len(shape) == 2 else 1
        self.inside = (slice(skip, skip + shape[0]), Ellipsis, slice(pad, pad + shape[-1]))
        self.out = self.all[self.inside]

    def untouched(self):
        around = self.all.clone()
        around[self.inside] = 1.0
        return bool((around == 1.0).all())


def disordered(A, E, seed):
    c = torch.Generator().manual_seed(seed)
    offsets = torch.randint(-3, A + 3, (E + 1,), generator=c)
    offsets[torch.randint(0, E + 1, (2,), generator=c)] = torch.tensor([2 ** 31 - 1, -2 ** 31])
    return offsets.int().cuda()


SHAPES = [(700, 5, 200, 96), (12, 9, 72, 1024), (40, 6, 264, 288), (3000, 3, 328, 544), (900, 4, 136, 1056)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("A,E,N,K", SHAPES)
def test_products(A, E, N, K, form, out):
    g = gen(A + N)
    args, kw, x, w = operands(form, g, A, E, N, K)
    sizes = [A // E] * (E - 1)
    offsets = offsets_of(sizes + [A - sum(sizes)])
    m = Marked(A, N, dtype=out, pad=8)
    bgq.grouped_matmul(*args, offsets, out=m.out, **kw)
    check(m.out, *product(x, w, offsets), K)
    assert m.untouched()
    for seed in range(6):
        m.out.fill_(2.0)
        bgq.grouped_matmul(*args, disordered(A, E, seed), out=m.out, **kw)
        assert bool(m.out.isfinite().all()) and m.untouched()


# many tiles of 256 x 256
@pytest.mark.parametrize("form", ["bf16", "transposed", "mx"])
def test_products_of_many_rows(form):
    g = gen(3)
    A, E, N, K = 15971, 3, 2040, 672
    args, kw, x, w = operands(form, g, A, E, N, K)
    offsets = offsets_of([9001, 0, 6970])
    m = Marked(A, N, dtype=F32, pad=8)
    bgq.grouped_matmul(*args, offsets, out=m.out, **kw)
    check(m.out, *product(x, w, offsets), K)
    assert m.untouched()
    for seed in range(3):
        m.out.fill_(2.0)
        bgq.grouped_matmul(*args, disordered(A, E, seed), out=m.out, **kw)
        assert bool(m.out.isfinite().all()) and m.untouched()


def space(A, E, N, K):
    """A workspace between marks, filled with NaN."""
    need = bgq.grouped_dw_workspace_bytes(A, E, N, K)
    if not need:
        return None, None
    marked = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    marked[256:256 + need] = 255
    return marked, marked[256:256 + need]


def gradient_call(dy, x, offsets, dtype):
    E, N, K = offsets.numel() - 1, dy.shape[1], x.shape[1]
    m = Marked(E, N, K, dtype=dtype)
    marked, ws = space(dy.shape[0], E, N, K)
    bgq.grouped_matmul_dw(dy, x, offsets, out=m.out, workspace=ws)
    assert m.untouched()
    assert ws is None or bool((marked[:256] == 7).all()) and bool((marked[-256:] == 7).all())
    return m.out


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("A,E,N,K,splits", [(700, 5, 200, 96, False), (4000, 3, 136, 128, True), (6000, 1, 264, 72, True), (40, 9, 72, 600, False)])
def test_gradients(A, E, N, K, splits, out):
    g = gen(A + N)
    dy, x = amid(normal(g, A, N), torch.nan), amid(normal(g, A, K), torch.nan)
    assert (bgq.grouped_dw_workspace_bytes(A, E, N, K) > 0) == splits
    sizes = [A // (E + 1)] * (E - 1)
    offsets = offsets_of(sizes + [A - sum(sizes)])
    check(gradient_call(dy, x, offsets, out), *gradient(dy, x, offsets), max(sizes + [A - sum(sizes)]))
    for seed in range(6):
        assert bool(gradient_call(dy, x, disordered(A, E, seed), out).isfinite().all())


# A block of x stays in LDS for up to three blocks of dy from n k E = 6144 tiles on (128 columns of dy, 256 of x).  Experts of one
# to three stages of 64 rows keep it, longer ones read it again; columns that fill no tile on either side.
LENGTHS = [0, 1, 64, 65, 128, 129, 192, 193, 400, 17, 0, 257, 63, 127, 191, 256]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("N,K,first", [(1400, 2312, 0), (1288, 2568, 5), (1672, 2056, 11)])
def test_gradients_that_keep_x(N, K, first, out):
    g = gen(N)
    E = 64
    assert -(-N // 128) * -(-K // 256) * E >= 6144 and N % 384
    sizes = [LENGTHS[(first + e * 7) % len(LENGTHS)] for e in range(E)]
    A = sum(sizes)
    dy, x = amid(normal(g, A, N), torch.nan), amid(normal(g, A, K), torch.nan)
    offsets = offsets_of(sizes)
    dw = gradient_call(dy, x, offsets, out)
    for e in range(0, E, 8):  # 64-bit values of eight experts at a time
        check(dw[e:e + 8], *gradient(dy, x, offsets[e:e + 9]), max(sizes))
    again = gradient_call(dy, x, offsets, out)
    assert torch.equal(dw, again)
    for seed in range(3):
        assert bool(gradient_call(dy, x, disordered(A, E, seed), out).isfinite().all())
