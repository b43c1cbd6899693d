"""The handle of the whole layer (MoeLayer): what it holds and what it refuses when
it is made.  On the CPU the device checks are put aside; nothing is launched."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd import layer as layer_module

E, H, I, K, GS = 8, 256, 128, 2, 64


@pytest.fixture
def on_cpu(monkeypatch):
    """Lets MoeLayer.__init__ take host tensors."""
    def ptr(t, name, itemsize=None, shape=None):
        if t.element_size() != itemsize or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(name)
        return ctypes.c_void_p(t.data_ptr())
    monkeypatch.setattr(layer_module, "_device", lambda t, name: t.device)
    monkeypatch.setattr(bgq, "_dev_ptr", ptr)


def weights(dev="cpu", seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = dict(router_weight=0.1 * r(E, H), expert_scale=1 + 0.1 * r(E).abs(), norm_weight=1 + 0.1 * r(H),
             post_weight=1 + 0.1 * r(H), pre_weight=1 + 0.1 * r(H))
    for name, rows, cols in (("gateup", 2 * I, H), ("down", H, I)):
        w["w_" + name] = torch.randint(-2**31, 2**31, (E, rows, cols // 8), generator=g, dtype=torch.int32)
        w["s_" + name] = (0.02 * r(E, rows, cols // GS)).abs().bfloat16()
        w["b_" + name] = -8 * w["s_" + name]
    return {n: t.to(dev) for n, t in w.items()}


def make(w, **kw):
    names = ("w_gateup", "s_gateup", "b_gateup", "w_down", "s_down", "b_down")
    rest = {n: t for n, t in w.items() if n not in names and n != "router_weight"}
    return bgq.MoeLayer(w["router_weight"], K, *(w[n] for n in names), **{**rest, **kw})


def addresses(layer):
    """The device pointers that a call of the handle passes on, by field."""
    found = {}
    for d in (layer._desc, layer._tail):
        found.update({n: getattr(d, n) for n, t in d._fields_ if t is ctypes.c_void_p and getattr(d, n)})
    return found


FLOATS = ("router_weight", "expert_scale", "norm_weight", "post_weight", "pre_weight")


def test_handle_owns_what_it_points_to(on_cpu):
    """A module's .to(), .bfloat16() and the like give its parameters other memory
    under the same tensor object; the handle keeps the memory that it was made of."""
    w = weights()
    w.update({n: torch.nn.Parameter(w[n]) for n in FLOATS})
    layer = make(w)
    before = addresses(layer)
    assert set(before) >= {"router_weight", "norm_weight", "expert_scale", "post_weight", "pre_weight", "w_gateup", "b_down"}
    for n, t in w.items():
        t.data = t.data.clone() if n not in FLOATS else t.data.double()
    held = {t.data_ptr() for t in layer._keep if t is not None}
    assert addresses(layer) == before and set(before.values()) <= held


@pytest.mark.gpu
def test_calls_after_the_parameters_moved():
    w = weights("cuda")
    w.update({n: torch.nn.Parameter(w[n]) for n in FLOATS})
    layer = make(w)
    x = torch.randn(5, H, device="cuda").bfloat16()
    want = layer(x, residual=x)
    torch.cuda.synchronize()
    sizes = {n: t.numel() * t.element_size() for n, t in w.items()}
    for t in w.values():
        t.data = t.data.clone()
    # what the allocator hands out next would lie where the weights lay
    junk = [torch.full((s,), 0x7F, dtype=torch.uint8, device="cuda") for s in sizes.values() for _ in range(3)]
    got = layer(x, residual=x)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 3 * len(sizes)


@pytest.mark.parametrize("kw", [{}, dict(bits=8), dict(flags=2), dict(group_size=32, flags=4)])
@pytest.mark.parametrize("E_,H_,I_,k", [(128, 2816, 704, 8), (8, 256, 128, 2), (64, 64, 1024, 16)])
def test_workspace_of_a_batch_serves_every_smaller_one(E_, H_, I_, k, kw):
    """A program sizes one workspace for its largest batch."""
    sizes = [bgq.lib().moe_layer_workspace_bytes(ctypes.byref(bgq.problem(T, k, E_, H_, I_, **kw))) for T in range(1, 80)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


ALL = FLOATS + ("w_gateup", "s_gateup", "b_gateup", "w_down", "s_down", "b_down")


@pytest.mark.parametrize("name", [n for n in ALL if n != "expert_scale"])
def test_refuses_weights_off_16_bytes(on_cpu, name):
    """When the handle is made, by name: a call would refuse them too."""
    w = weights()
    t = w[name]
    flat = torch.empty(t.numel() + 16, dtype=t.dtype)
    w[name] = flat[4:4 + t.numel()].view(t.shape)  # 8 or 16 bytes on
    if t.element_size() == 4:
        w[name] = flat[2:2 + t.numel()].view(t.shape)
    assert w[name].data_ptr() % 16 == 8
    with pytest.raises(ValueError, match=f"{name} must start on 16 bytes"):
        make(w)


@pytest.mark.parametrize("name", ["s_gateup", "b_gateup", "s_down", "b_down"])
def test_refuses_float16_scales(on_cpu, name):
    """They would be read as bf16 bits."""
    w = weights()
    w[name] = w[name].half()
    with pytest.raises(ValueError, match=f"{name} must hold bfloat16"):
        make(w)


def test_takes_other_types_of_the_same_bits(on_cpu):
    w = weights()
    for n in ("s_gateup", "b_gateup", "s_down", "b_down"):
        w[n] = w[n].view(torch.int16)
    w["w_gateup"] = w["w_gateup"].view(torch.float32)
    make(w)
