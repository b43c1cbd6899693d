"""Outputs on memory that a call reads or writes otherwise: refused on the host, before anything is
enqueued.  Tensors that lie between each other's rows are taken."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.grouped import MoeGrouped, MoeGroupedGrad, MoeMx

P = 0x1000000
UNSUPPORTED = -3

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run on made-up addresses")


def mx(f, **kw):
    q = MoeMx(R=10, K=96, type=0, values=P, codes=2 * P, scales=3 * P, stride=96)
    for k, v in kw.items():
        setattr(q, k, v)
    return getattr(bgq.lib(), f)(ctypes.byref(q), None)


# values: 10 rows of 192 bytes; codes 480 bytes, scales 30
OVERLAPS = [
    dict(codes=P), dict(scales=P), dict(codes=P + 9 * 192 + 176), dict(codes=P - 464), dict(scales=P + 10 * 192 - 1), dict(scales=P - 29),
    dict(scales=2 * P), dict(scales=2 * P + 479), dict(scales=2 * P - 29), dict(type=1, codes=P + 3824),
    dict(stride=4096, codes=P + 9 * 8192 + 176), dict(stride=4096, scales=P + 8192 - 29), dict(stride=4096, scales=P + 8192 + 191),
]
APART = [
    dict(codes=P + 10 * 192), dict(codes=P - 480), dict(scales=P + 10 * 192), dict(scales=P - 30), dict(scales=2 * P + 480),
    dict(scales=2 * P - 30), dict(type=1, codes=P + 3840), dict(stride=4096, codes=P + 192), dict(stride=4096, codes=P + 8 * 8192 + 7712),
    dict(stride=4096, scales=P + 192), dict(stride=4096, scales=P + 8192 - 30),
]


@pytest.mark.parametrize("f", ["moe_mx_quantize", "moe_mx_dequantize"])
@pytest.mark.parametrize("kw", OVERLAPS)
def test_microscaled_overlaps_are_refused(f, kw):
    assert mx(f, **kw) == UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("f", ["moe_mx_quantize", "moe_mx_dequantize"])
@pytest.mark.parametrize("kw", APART)
def test_microscaled_neighbours_are_taken(f, kw):
    assert mx(f, **kw) == -6  # it reaches the launch, for which there is no GPU


def test_gated_rows_count_whole():
    """A row of [g | u] is 2 K values."""
    assert mx("moe_mx_quantize", flags=1, stride=192, codes=P + 9 * 384 + 368) == UNSUPPORTED
    assert mx("moe_mx_quantize", flags=1, stride=200, scales=P + 383) == UNSUPPORTED


@pytest.mark.gpu
def test_binding_refuses_codes_over_values():
    x = torch.randn(40, 96, device="cuda").bfloat16()
    raw = x.view(torch.uint8)
    before = x.clone()
    codes, scales = bgq.mx_quantize(x)
    for call in (lambda: bgq.mx_quantize(x, codes=raw.flatten()[:40 * 48].view(40, 48)),
                 lambda: bgq.mx_quantize(x, scales=raw.flatten()[64:64 + 120].view(40, 3)),
                 lambda: bgq.mx_quantize(x, codes=codes, scales=codes.flatten()[:120].view(40, 3)),
                 lambda: bgq.mx_dequantize(raw.flatten()[:40 * 48].view(40, 48), scales, out=x)):
        with pytest.raises(bgq.MoeError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    # codes and scales in the gaps of values' rows are taken
    wide = torch.zeros(40, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, :96] = x
    gap = wide[0, 96:].view(torch.uint8)  # 320 bytes
    one = bgq.mx_quantize(wide[:2, :96], codes=gap[:96].view(2, 48), scales=gap[96:102].view(2, 3))
    assert torch.equal(one[0], codes[:2]) and torch.equal(one[1], scales[:2])


def product(**kw):
    g = MoeGrouped(A=10, E=4, N=64, K=96, x_type=0, w_type=0, out_type=0, offsets=P, x=2 * P, w=3 * P, out=4 * P, x_stride=96, w_stride=96,
                   w_expert_stride=64 * 96, out_stride=64)
    for k, v in kw.items():
        setattr(g, k, v)
    return bgq.lib().moe_grouped_matmul(ctypes.byref(g), None)


MX = dict(w_type=2, w_scales=5 * P)  # codes 4 * 64 * 48 bytes, scales 4 * 64 * 3
MX2 = dict(MX, x_type=2, x_scales=6 * P)  # codes 10 * 48, scales 10 * 3
W = 4 * 64 * 96 * 2


@pytest.mark.parametrize("kw", [
    dict(out=2 * P + 192), dict(out=2 * P + 9 * 192 + 176), dict(out=2 * P - 1264), dict(out=3 * P + W - 16), dict(out=3 * P - 16),
    dict(x_stride=4096, out=2 * P + 8192 - 16, out_stride=4096), dict(x_stride=4096, out_stride=2048, out=2 * P + 80),
    dict(offsets=4 * P + 1276), dict(offsets=4 * P - 16), dict(w_stride=960, w_expert_stride=96, out_stride=960, out=3 * P + 736),
    dict(w_stride=192, w_expert_stride=0, out_stride=192, out=3 * P + 64), dict(MX, out=3 * P + 12272), dict(MX, out=5 * P + 752),
    dict(MX2, out=2 * P + 464), dict(MX2, out=6 * P + 16), dict(out_type=1, out=2 * P - 2544),
    dict(x_stride=0, out=2 * P + 176), dict(flags=1, out=3 * P + 64 * 4),
])
def test_products_refuse_overlaps(kw):
    assert product(**kw) == UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(out=2 * P + 1920), dict(out=2 * P - 1280), dict(out=3 * P + W), dict(out=3 * P - 1280), dict(out_type=1, out=2 * P - 2560),
    dict(x_stride=4096, out_stride=4096, out=2 * P + 192), dict(x_stride=4096, out_stride=4096, out=2 * P - 128),
    dict(x_stride=4096, out_stride=2048, out=2 * P + 192), dict(offsets=4 * P + 1280), dict(offsets=4 * P - 20),
    dict(w_stride=960, w_expert_stride=96, out_stride=960, out=3 * P + 768), dict(w_stride=192, w_expert_stride=0, out_stride=192, out=3 * P + 192),
    dict(MX, out=3 * P + 12288), dict(MX, out=5 * P + 768), dict(MX2, out=2 * P + 480), dict(MX2, out=6 * P + 32),
    dict(x_stride=0, out=2 * P + 192), dict(x=3 * P), dict(w_expert_stride=(1 << 62)),
])
def test_products_take_neighbours(kw):
    assert product(**kw) == -6


def grad(ws=7 * P, ws_bytes=1 << 40, **kw):
    g = MoeGroupedGrad(A=10, E=4, N=64, K=96, out_type=0, offsets=P, dy=2 * P, x=3 * P, dw=4 * P, dy_stride=64, x_stride=96)
    for k, v in kw.items():
        setattr(g, k, v)
    return bgq.lib().moe_grouped_matmul_dw(ctypes.byref(g), ws, ws_bytes, None)


SPLIT = dict(A=4000, E=1)  # runs of rows, so a workspace


@pytest.mark.parametrize("kw", [
    dict(dw=2 * P + 1264), dict(dw=2 * P - W + 16), dict(dw=3 * P + 1904), dict(dw=3 * P - W + 16), dict(offsets=4 * P + W - 4),
    dict(out_type=1, dw=3 * P - 2 * W + 16), dict(dy_stride=65536, dw=2 * P + 9 * 131072 + 112), dict(A=0, offsets=4 * P + 16),
    dict(SPLIT, ws=4 * P), dict(SPLIT, dw=7 * P + 512), dict(SPLIT, ws=2 * P + 512), dict(SPLIT, ws=3 * P + 512), dict(SPLIT, offsets=7 * P + 4),
])
def test_gradients_refuse_overlaps(kw):
    assert grad(**kw) == UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(dw=2 * P + 1280), dict(dw=2 * P - W), dict(dw=3 * P + 1920), dict(dw=3 * P - W), dict(offsets=4 * P + W), dict(x=2 * P),
    dict(dy_stride=65536, dw=2 * P + 128), dict(ws=4 * P), SPLIT,
])
def test_gradients_take_neighbours(kw):
    assert grad(**kw) == -6


@pytest.mark.gpu
def test_binding_refuses_results_over_operands():
    g = torch.Generator(device="cuda").manual_seed(0)
    both = torch.randn(40, 256, generator=g, device="cuda").bfloat16()
    x, w, before = both[:, :64], torch.randn(96, 64, generator=g, device="cuda").bfloat16(), both.clone()
    for call in (lambda: bgq.grouped_matmul(x[1:], w[:64], out=both[:-1, :64]), lambda: bgq.grouped_matmul(x, w, out=both[:, 56:152]),
                 lambda: bgq.grouped_matmul_dw(both[:, :32], both[:, 64:96], out=both.flatten()[:1024].view(1, 32, 32))):
        with pytest.raises(bgq.MoeError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(both, before)
    # beside x in the same rows
    want = bgq.grouped_matmul(x, w)
    assert torch.equal(bgq.grouped_matmul(x, w, out=both[:, 64:160]), want) and torch.equal(both[:, :64], before[:, :64])
    assert torch.equal(both[:, 160:], before[:, 160:])
