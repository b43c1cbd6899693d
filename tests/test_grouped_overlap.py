"""Outputs on memory that a call reads or writes otherwise: refused on the host, before anything is
enqueued.  Tensors that lie between each other's rows are taken."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.grouped import MoeMx

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
