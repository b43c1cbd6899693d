"""Microscaled 4-bit values on the GPU: codes and scales bit for bit."""
import math

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from grouped_util import F64, decode, encode

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rows(seed, R, K, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, K, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (R, K // 32), generator=g, device="cuda").float()
                                                                  ).repeat_interleave(32, -1)
    return x.to(dtype)


def same(got, ref):
    return all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (7, 352), (1, 2816), (130, 704), (1000, 96), (65, 1056)])
def test_codes(R, K, dtype):
    x = rows(R + K, R, K, dtype)
    got = bgq.mx_quantize(x)
    assert got[0].shape == (R, K // 2) and got[1].shape == (R, K // 32)
    assert same(got, encode(x.to(F64)))
    for out in (BF, F32):
        v = bgq.mx_dequantize(*got, out_dtype=out)
        assert v.dtype is out and torch.equal(v.to(F64), decode(*got))


def test_borders():
    """Every value between two codes, one step below and above, in every binade that fp32 holds, subnormals too."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0], dtype=F32)
    near = torch.cat([ties, torch.nextafter(ties, torch.tensor(0.0)), torch.nextafter(ties, torch.tensor(9.0))])
    near = torch.cat([near, -near])
    block = torch.zeros(3, 32)
    block.view(-1)[:90] = near
    for e in range(-150, 126):
        x = (block.double() * 2.0 ** e).float()
        x[:, -1] = 2.0 ** (e + 2) if e + 2 >= -149 else 0.0  # the block's largest, or its like
        x = x.cuda()
        assert same(bgq.mx_quantize(x), encode(x.to(F64))), e


def test_zeros_and_what_is_not_finite():
    x = torch.zeros(5, 96, device="cuda")
    x[1, 40], x[2, 3], x[3, 70], x[4, 95] = math.nan, math.inf, -math.inf, -0.0
    x[1:4] += torch.linspace(-1, 1, 96, device="cuda")
    for t in (x, x.to(BF)):
        codes, scales = bgq.mx_quantize(t)
        assert same((codes, scales), encode(t.to(F64)))
        assert scales.tolist()[0] == [0, 0, 0] and scales[1, 1] == scales[2, 0] == scales[3, 2] == 255
        v = bgq.mx_dequantize(codes, scales)
        assert torch.equal(v.isnan(), decode(codes, scales).isnan()) and int(v.isnan().sum()) == 96
    big = torch.full((1, 32), torch.finfo(F32).max, device="cuda")
    assert same(bgq.mx_quantize(big), encode(big.to(F64)))


def test_every_code_under_every_scale():
    codes = (torch.arange(16, device="cuda") | (15 - torch.arange(16, device="cuda")) << 4).to(torch.uint8).expand(256, 16).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].contiguous()
    ref = decode(codes, scales)
    for out in (BF, F32):
        v = bgq.mx_dequantize(codes, scales, out_dtype=out)
        assert torch.equal(v.isnan(), ref.isnan())
        assert torch.equal(v[:255], ref[:255].to(out))  # past the range: infinity


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("glu", ["gelu", "silu"])
@pytest.mark.parametrize("R,K", [(1, 32), (37, 352), (300, 704)])
def test_gated(R, K, glu, dtype):
    """act(g) u in fp32.  The exponent of the sigmoid's exponential is off by at most 5 u of itself (five
    roundings), the exponential by that times its size, up to 150 where fp32 holds it, and ln 2, the other
    steps by a few u: e = 2^-14 relative covers 150 * 5 u * ln 2 + 8 u.  So a code may be that of any value
    in v (1 +- e), and the scale too; few values lie that near to a border."""
    g = torch.Generator(device="cuda").manual_seed(R + K)
    x = (torch.randn(R, 2 * K, generator=g, device="cuda") * 2).to(dtype)
    a, u = x.to(F64).chunk(2, -1)
    z = a if glu == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
    v = a * torch.sigmoid(z) * u
    codes, scales = bgq.mx_quantize(x, glu=glu)
    got = decode(codes, scales)
    e = 2.0 ** -14
    low, high = decode(*encode(v * (1 - e))), decode(*encode(v * (1 + e)))
    clean = (low == high)
    assert bool((got == low)[clean].all()) and float(clean.double().mean()) > 0.99
    rest = got[~clean]
    assert bool(((rest >= torch.minimum(low, high)[~clean]) & (rest <= torch.maximum(low, high)[~clean])).all())
    assert same((codes, scales), bgq.mx_quantize(x, glu=glu))


def test_strided_rows_shapes_and_outputs():
    x = rows(3, 40, 256, BF)
    view = x[:, 64:160]
    codes = torch.full((40, 48), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 3), 9, dtype=torch.uint8, device="cuda")
    got = bgq.mx_quantize(view, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales and same(got, encode(view.to(F64)))
    wide = torch.full((40, 112), 5.0, device="cuda")
    bgq.mx_dequantize(codes, scales, out=wide[:, 8:104])
    assert torch.equal(wide[:, 8:104].to(F64), decode(codes, scales))
    assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 104:] == 5).all())
    w = x.view(4, 10, 256)
    assert same(bgq.mx_quantize(w), [t.view(4, 10, -1) for t in bgq.mx_quantize(x)])
    assert bgq.mx_quantize(x[:0])[0].shape == (0, 128) and bgq.mx_dequantize(*bgq.mx_quantize(x[:0])).shape == (0, 256)
    packed = [t.view(d) for t, d in zip(got, (torch.float4_e2m1fn_x2, torch.float8_e8m0fnu))]
    assert torch.equal(bgq.mx_dequantize(*packed), bgq.mx_dequantize(*got))
