"""Grouped products and microscaled values: the documented limits on sizes, to the last size that is taken and the
first that is refused.  A call whose sizes are taken goes on to the check of its alignment (nothing is enqueued)."""
import ctypes

import pytest

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.grouped import MoeGrouped, MoeGroupedGrad, MoeMx

P = 0x10000
SHAPE, ALIGN = -2, -4


@pytest.mark.parametrize("f", ["moe_mx_quantize", "moe_mx_dequantize"])
@pytest.mark.parametrize("K", [32, 96, 704, 2816, 1 << 20, (1 << 20) - 32])
def test_microscaled_rows(f, K):
    """R K < 2^34."""
    most = (2 ** 34 - 1) // K
    for R, status in ((most, ALIGN), (most + 1, SHAPE)):
        q = MoeMx(R=R, K=K, type=0, values=P + 8, codes=2 * P, scales=3 * P, stride=K)
        assert getattr(bgq.lib(), f)(ctypes.byref(q), None) == status


@pytest.mark.parametrize("f", ["moe_mx_quantize", "moe_mx_dequantize"])
def test_microscaled_stride(f):
    for stride, status in ((1 << 30, ALIGN), ((1 << 30) + 8, SHAPE)):
        q = MoeMx(R=2, K=64, type=0, values=P + 8, codes=2 * P, scales=3 * P, stride=stride)
        assert getattr(bgq.lib(), f)(ctypes.byref(q), None) == status


@pytest.mark.parametrize("E,N,strip", [(1, 1 << 20, 128), (1, 40, 128), (8, 1 << 20, 128), (1024, 1 << 17, 32)])
def test_product_sizes(E, N, strip):
    """(A / strip + E) ceil(N / 32) < 2^24, strips of 32 rows up to 192 rows an expert, else of 128."""
    units = -(-N // 32)
    most = min(((2 ** 24 - 1) // units - E) * strip + strip - 1, 2 ** 30 - 1)
    assert (most + 1 <= 192 * E) == (strip == 32)
    for A, status in ((most, ALIGN), (most + 1, SHAPE)):
        g = MoeGrouped(A=A, E=E, N=N, K=8, x_type=0, w_type=0, out_type=0, offsets=P, x=2 * P + 8, w=3 * P, out=4 * P, x_stride=8,
                       w_stride=8, w_expert_stride=8, out_stride=N)
        assert bgq.lib().moe_grouped_matmul(ctypes.byref(g), None) == status


def test_gradient_sizes():
    """E ceil(N / 64) ceil(K / 64) < 2^31 - 1."""
    for E, N, K, status in ((8, (1 << 20) - 64, 1 << 20, ALIGN), (8, 1 << 20, 1 << 20, SHAPE), (1024, 1 << 17, 1 << 16, SHAPE),
                            (1023, 1 << 17, 1 << 16, ALIGN)):
        g = MoeGroupedGrad(A=2, E=E, N=N, K=K, out_type=0, offsets=P, dy=2 * P + 8, x=3 * P, dw=4 * P, dy_stride=N, x_stride=K)
        assert bgq.lib().moe_grouped_matmul_dw(ctypes.byref(g), None, 0, None) == status
