"""Products grouped by expert and microscaled values: refusals, on the CPU (every call
fails a check of the host before anything is enqueued)."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.grouped import MoeGrouped, MoeGroupedGrad, MoeMx

P = 0x10000


def product(**kw):
    g = MoeGrouped(A=10, E=4, N=64, K=96, x_type=0, w_type=0, out_type=0, offsets=P, x=2 * P, w=3 * P, out=4 * P,
                   x_stride=96, w_stride=96, w_expert_stride=64 * 96, out_stride=64)
    for k, v in kw.items():
        setattr(g, k, v)
    return bgq.lib().moe_grouped_matmul(ctypes.byref(g), None)


MX = dict(w_type=2, w_scales=5 * P)
MX2 = dict(MX, x_type=2, x_scales=6 * P)


@pytest.mark.parametrize("kw,status", [
    (dict(A=-1), -2), (dict(A=1 << 30), -2), (dict(E=0), -2), (dict(E=1025), -3), (dict(N=0), -2), (dict(N=60), -2),
    (dict(K=0), -2), (dict(K=100), -2), (dict(N=(1 << 20) + 8), -3), (dict(K=(1 << 20) + 8), -3),
    (dict(x_type=1), -3), (dict(x_type=2), -3), (dict(w_type=1), -3), (dict(w_type=3), -3), (dict(out_type=2), -3),
    (dict(flags=2), -3), (dict(MX, flags=1), -3), (dict(MX, K=72), -2), (dict(MX2, K=104), -2),
    (dict(x_stride=-8), -2), (dict(x_stride=100), -2), (dict(x_stride=(1 << 22) + 8), -2), (dict(w_stride=-8), -2),
    (dict(w_stride=97), -2), (dict(w_expert_stride=-8), -2), (dict(w_expert_stride=100), -2), (dict(out_stride=63), -2),
    (dict(out_stride=56), -2), (dict(out_stride=68), -2), (dict(out_type=1, out_stride=66), -2),
    (dict(A=(1 << 30) - 1, N=1 << 20), -2), (dict(A=20000, E=512, N=1 << 20), -2), (dict(MX, A=190 * 512, E=512, N=1 << 18, K=32), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(offsets=None), -1), (dict(MX, w_scales=None), -1),
    (dict(MX2, x_scales=None), -1),
    (dict(x=2 * P + 8), -4), (dict(w=3 * P + 2), -4), (dict(out=4 * P + 4), -4), (dict(offsets=P + 2), -4),
    (dict(out=2 * P), -3), (dict(out=3 * P), -3),
])
def test_product_refuses(kw, status):
    assert product(**kw) == status


def test_product_without_rows():
    assert product(A=0, x=None, w=None, out=None, offsets=None) == 0
    assert bgq.lib().moe_grouped_matmul(None, None) == -1


def grad(ws=7 * P, ws_bytes=1 << 40, **kw):
    g = MoeGroupedGrad(A=10, E=4, N=64, K=96, out_type=0, offsets=P, dy=2 * P, x=3 * P, dw=4 * P, dy_stride=64, x_stride=96)
    for k, v in kw.items():
        setattr(g, k, v)
    return bgq.lib().moe_grouped_matmul_dw(ctypes.byref(g), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(A=-1), -2), (dict(A=1 << 30), -2), (dict(E=0), -2), (dict(E=1025), -3), (dict(N=60), -2), (dict(K=100), -2),
    (dict(N=(1 << 20) + 8), -3), (dict(E=1024, N=1 << 20, K=1 << 20), -2), (dict(out_type=2), -3),
    (dict(dy_stride=-8), -2), (dict(x_stride=97), -2), (dict(x_stride=(1 << 22) + 8), -2),
    (dict(dy=None), -1), (dict(x=None), -1), (dict(dw=None), -1), (dict(offsets=None), -1), (dict(A=0, dw=None), -1),
    (dict(dy=2 * P + 8), -4), (dict(x=3 * P + 8), -4), (dict(dw=4 * P + 8), -4), (dict(offsets=P + 1), -4),
    (dict(dw=2 * P), -3), (dict(dw=3 * P), -3),
    (dict(A=1 << 16, ws=None), -5), (dict(A=1 << 16, ws_bytes=1 << 10), -5), (dict(A=1 << 16, ws=7 * P + 128), -4),
])
def test_gradient_refuses(kw, status):
    assert grad(**kw) == status
    assert bgq.lib().moe_grouped_matmul_dw(None, None, 0, None) == -1


def test_gradient_workspace():
    assert bgq.grouped_dw_workspace_bytes(333, 5, 264, 1000) == 0
    assert bgq.grouped_dw_workspace_bytes(16384, 128, 1408, 2816) == 0  # tiles enough
    need = bgq.grouped_dw_workspace_bytes(1 << 16, 1, 64, 96)
    assert need > 0 and need % (64 * 96 * 4) == 0
    assert bgq.grouped_dw_workspace_bytes(1 << 16, 1, 64, 100) == 0  # refused sizes


def mx(f="moe_mx_quantize", **kw):
    q = MoeMx(R=10, K=96, type=0, values=P, codes=2 * P, scales=3 * P, stride=96)
    for k, v in kw.items():
        setattr(q, k, v)
    return getattr(bgq.lib(), f)(ctypes.byref(q), None)


@pytest.mark.parametrize("f", ["moe_mx_quantize", "moe_mx_dequantize"])
@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=(1 << 20) + 32, stride=1 << 21), -3), (dict(type=2), -3),
    (dict(flags=3), -3), (dict(flags=4), -3), (dict(R=1 << 33), -2), (dict(stride=64), -2), (dict(stride=100), -2),
    (dict(type=1, stride=98), -2), (dict(stride=1 << 31), -2), (dict(values=None), -1), (dict(codes=None), -1),
    (dict(scales=None), -1), (dict(values=P + 8), -4), (dict(codes=2 * P + 4), -4),
])
def test_microscaled_refuses(f, kw, status):
    assert mx(f, **kw) == status


def test_microscaled_flags_and_empty():
    assert mx(flags=1, stride=96) == -2  # a row is [g | u]
    assert mx("moe_mx_dequantize", flags=1, stride=192) == -3
    assert mx(R=0, values=None, codes=None, scales=None) == 0
    assert bgq.lib().moe_mx_quantize(None, None) == bgq.lib().moe_mx_dequantize(None, None) == -1


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: bgq.grouped_matmul(x, x), lambda: bgq.grouped_matmul_dw(x, x), lambda: bgq.mx_quantize(x),
                 lambda: bgq.mx_dequantize(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_structures_match_the_header():
    assert ctypes.sizeof(MoeGrouped) == 112 and ctypes.sizeof(MoeGroupedGrad) == 72 and ctypes.sizeof(MoeMx) == 56
