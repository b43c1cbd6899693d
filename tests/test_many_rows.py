"""Batches of more rows than one dimension of a launch holds (2^32 threads: 2^22 rows
of a workgroup of 1024, 2^24 of 256, 2^26 of a wave), and their refusals."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd import layer as layer_module
from bit_gathered_quantized_amd.layer import MOE_R_NORM, MoeRouter


def test_router_refuses_more_tokens_than_a_launch_holds():
    most = (1 << 30) - 64
    for T, x, status in ((most + 1, 0x20000, -2), (1 << 30, 0x20000, -2), (2**31 - 1, 0x20000, -2), (most, None, -1)):
        r = MoeRouter(T=T, H=64, E=1, k=1, eps=1e-6, x_stride=64, weight=0x10000, flags=MOE_R_NORM)
        assert bgq.lib().moe_router_forward(ctypes.byref(r), x, 0x30000, 0x40000, 0x50000, None) == status


@pytest.mark.parametrize("T", [2**31, 2**32 + 5])
def test_block_norm_refuses_rows_past_31_bits(T, monkeypatch):
    monkeypatch.setattr(layer_module, "_device", lambda t, name: t.device)
    y = torch.zeros(1, 1, dtype=torch.bfloat16).expand(T, 1)
    with pytest.raises(ValueError, match="rows"):
        bgq.block_norm(y, want_out=False, pre_norm=True)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [((1 << 22) + 9, 1030), ((1 << 24) + 5, 3), ((1 << 26) + 13, 8)])
def test_block_norm(T, H):
    """out = gate_t y with the same y in every row: bf16 products, one rounding."""
    g = torch.Generator(device="cuda").manual_seed(H)
    y = torch.randn(1, H, generator=g, device="cuda").bfloat16()
    gate = torch.randn(T, 1, generator=g, device="cuda")
    out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    bgq.block_norm(y.expand(T, H), gate=gate, out=out[1:T + 1])
    for at in range(0, T, 1 << 20):
        n = min(1 << 20, T - at)
        assert torch.equal(out[1 + at:1 + at + n], (gate[at:at + n] * y.float()).bfloat16()), at
    assert bool((out[0] == 7.0).all()) and bool((out[T + 1] == 7.0).all())


@pytest.mark.gpu
def test_topk():
    T, E = (1 << 26) + 3, 3
    logits = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids, weights = bgq.router_topk(logits, 1)
    assert torch.equal(ids[:, 0].long(), logits.argmax(-1)) and bool((weights == 1.0).all())


@pytest.mark.parametrize("T,k,H,I,kw,fits", [
    ((1 << 22) - 1, 1, 4096, 64, {}, True), (1 << 22, 1, 4096, 64, {}, False),        # combine: T H / 4 threads
    (1 << 24, 8, 64, 4096, {}, False), ((1 << 24) - 64, 1, 64, 4096, {}, True),      # gate|up: tiles of 64 rows by 128 columns
    ((1 << 24) - 64, 1, 64, 4096, dict(bits=8), False),                              # tiles of 32 rows
    ((1 << 23) - 1024, 1, 64, 4096, dict(bits=8), True),
    (1 << 25, 1, 64, 64, dict(flags=2), True), (1 << 29, 1, 64, 64, dict(flags=2), False)])
def test_expert_ffn_refuses_sizes_past_a_launch(T, k, H, I, kw, fits):
    """What fits goes on to the next check, that of the workspace."""
    p = bgq.problem(T, k, 8, H, I, **kw)
    some = ctypes.c_void_p(0x10000)
    st = bgq.lib().moe_expert_ffn_forward(ctypes.byref(p), *[some] * 9, some, some, 0, None)
    assert st == (-5 if fits else -2)
