"""Arguments of a block norm: tensors that lie on one another (exactly the same rows
are written in place, the same address in any other way is refused) and gates that are
numbers."""
import ctypes

import numpy as np
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd import layer as layer_module
from bit_gathered_quantized_amd.layer import MoeLayerDesc, MoeNorm

Y, RES, OUT, NORMED = 0x10000, 0x20000, 0x30000, 0x40000


def norm(**kw):
    n = MoeNorm(T=4, H=64, eps=1e-6, residual_scale=1.0, gate_scale=1.0, y_stride=64, residual_stride=64, out_stride=64,
                normed_stride=64, residual=RES, out=OUT, normed=NORMED)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


REFUSED = [dict(out=OUT, normed=OUT), dict(out=RES, residual_stride=72), dict(normed=RES, out_stride=72, residual_stride=72),
           dict(normed=RES, normed_type=1), dict(out=RES, residual_stride=0)]
OF_Y = [dict(out=Y, y_stride=72), dict(out=Y, y_type=1), dict(normed=Y, normed_type=1), dict(normed=Y, y_stride=0),
        dict(normed=Y, normed_stride=128)]


@pytest.mark.parametrize("kw", REFUSED + OF_Y)
def test_block_norm_refuses(kw):
    assert bgq.lib().moe_block_norm(ctypes.byref(norm(**kw)), Y, None) == -3


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("kw", REFUSED)
def test_layer_refuses(T, kw):
    p = bgq.problem(T, 2, 8, 64, 64)
    d = MoeLayerDesc(flags=1, router_flags=1, eps=1e-6, router_weight=0x50000, w_gateup=0x50000, s_gateup=0x50000,
                     b_gateup=0x50000, w_down=0x50000, s_down=0x50000, b_down=0x50000)
    t = norm(T=T, **kw)
    assert bgq.lib().moe_layer_forward(ctypes.byref(p), ctypes.byref(d), 0x60000, ctypes.byref(t), 0x70000, 1 << 30,
                                       None) == -3


@pytest.mark.parametrize("kw", [dict(out=RES, residual_stride=72, out_stride=72), dict(out=Y), dict(normed=Y), dict(normed=RES),
                                dict(out=RES, normed=Y), dict(out=None, normed=Y), dict(T=1, out=Y, y_stride=99),
                                dict(out=Y, residual=None), dict(residual=Y, out=Y)])
def test_block_norm_takes_the_same_rows(kw):
    """Refused by the next check alone, that of the gate's alignment."""
    n = norm(**kw)
    n.gate, n.gate_type = 0x50002, 1
    assert bgq.lib().moe_block_norm(ctypes.byref(n), Y, None) == -4


@pytest.mark.parametrize("gate", [0.5, 2, np.float32(0.25), np.float64(0.125), np.int64(3), True])
def test_a_gate_may_be_any_number(gate):
    n = MoeNorm(gate_scale=1.0)
    layer_module._gate(n, gate, torch.device("cpu"), 4, 64)
    assert n.gate_scale == float(gate) and not n.gate


def test_a_gate_must_be_a_number_or_a_tensor():
    with pytest.raises((TypeError, ValueError)):
        layer_module._gate(MoeNorm(), "wide", torch.device("cpu"), 4, 64)
