"""Norms around a block (moe_block_norm): refusals on the CPU, values on the GPU
against the formulas in 64 bits.

The bound of a value is what fp32 arithmetic and one rounding can do.  With
u = 2^-24 and a thread's chain of at most 64 fused steps, 6 exchanges and 4 wave
sums of positive terms, a mean of squares is within 76 u and its inverse root
within 40 u; z takes three more products, out one sum.  Hence
    e_out  = u (48 |z| + 4 |residual_scale residual|)            before rounding
    e_norm = |w| / rms (e_out + |out| (rms(e_out) / rms + 48 u)) before rounding
plus half a step of the type, eps / 2 relative, for what is rounded to bf16
(fp32 stores add nothing)."""
import ctypes

import pytest
import torch

import bit_gathered_quantized_amd as bgq
from bit_gathered_quantized_amd.layer import MoeNorm

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def host_norm(**kw):
    n = MoeNorm(T=4, H=64, eps=1e-6, residual_scale=1.0, gate_scale=1.0, y_stride=64, residual_stride=64,
                out_stride=64, normed_stride=64, residual=0x10000, out=0x20000, normed=0x30000)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def host_call(n, y=0x40000):
    return bgq.lib().moe_block_norm(None if n is None else ctypes.byref(n), y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -2), (dict(H=0), -2), (dict(H=16385), -3), (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2),
    (dict(y_type=2), -3), (dict(stream_type=-1), -3), (dict(normed_type=7), -3), (dict(weight_type=2), -3),
    (dict(gate_type=2), -3), (dict(flags=2), -3), (dict(out=None, normed=None), -1),
    (dict(y_stride=-1), -2), (dict(residual_stride=-64), -2), (dict(out_stride=63), -2), (dict(normed_stride=0), -2),
    (dict(gate=0x50000, gate_stride_h=2), -2), (dict(gate=0x50000, gate_stride_t=-1), -2),
    (dict(out=0x20001), -4), (dict(normed=0x30001), -4), (dict(residual=0x10001), -4),
    (dict(stream_type=1, out=0x20002), -4), (dict(post_weight=0x50001, flags=1), -4),
    (dict(pre_weight=0x50002, weight_type=1), -4), (dict(gate=0x50002, gate_type=1), -4),
])
def test_host_checks(kw, status):
    assert host_call(host_norm(**kw)) == status


def test_host_checks_of_y():
    assert host_call(None) == -1
    assert host_call(host_norm(), None) == -1
    assert host_call(host_norm(), 0x40001) == -4
    assert host_call(host_norm(y_type=1), 0x40002) == -4
    assert host_call(host_norm(T=0, out=None, normed=None), None) == 0  # no rows: nothing is touched


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        bgq.block_norm(torch.zeros(2, 64))


def reference(y, residual, *, post, post_weight, gate, residual_scale, pre, pre_weight, offset, eps):
    """(out, normed) in 64 bits and the bounds of both before rounding."""
    d = torch.float64
    z = y.to(d)
    if post:
        z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt()
        if post_weight is not None:
            z = z * (offset + post_weight.to(d))
    if gate is not None:
        z = z * (gate if isinstance(gate, float) else gate.to(d))
    r = residual_scale * residual.to(d) if residual is not None else torch.zeros_like(z)
    out = r + z
    e_out = U * (48 * z.abs() + 4 * r.abs())
    if not pre:
        return out, None, e_out, None
    rms = (out.square().mean(-1, keepdim=True) + eps).sqrt()
    w = offset + pre_weight.to(d) if pre_weight is not None else torch.ones_like(out)
    e = w.abs() / rms * (e_out + out.abs() * (e_out.square().mean(-1, keepdim=True).sqrt() / rms + 48 * U))
    return out, out / rms * w, e_out, e


def check(got, ref, bound, what):
    half = 0.0 if got.dtype is F32 else torch.finfo(got.dtype).eps / 2
    got = got.double()
    same = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    err = (got - ref).abs()[same]
    # the rounding is of the computed value, which is within `bound` of ref
    allowed = (bound + half * (ref.abs() + bound))[same] + 1e-38
    worst = float((err / allowed).max()) if err.numel() else 0.0
    print(f"{what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def make(T, H, yt, st, wt, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gates = {None: None, "number": 0.3, "scalar": r(1), "channel": r(H), "token": r(T, 1), "full": r(T, H),
             "channel16": r(H).bfloat16()}
    return dict(y=(3 * r(T, H)).to(yt), residual=(2 * r(T, H) * (1 + r(H).abs())).to(st),
                post_weight=(1 + 0.2 * r(H)).to(wt), pre_weight=(1 + 0.2 * r(H)).to(wt), gate=gates[gate])


def run_case(T, H, yt=BF, st=BF, wt=BF, gate="channel", post=True, pre=True, offset=0.0, scale=0.7, eps=1e-6, nt=None,
             seed=0):
    d = make(T, H, yt, st, wt, gate, seed)
    pw, nw = (d["post_weight"] if post else None), (d["pre_weight"] if pre else None)
    normed = torch.empty(T, H, dtype=nt, device="cuda") if nt else None
    got = bgq.block_norm(d["y"], d["residual"], post_weight=pw, gate=d["gate"], residual_scale=scale, pre_weight=nw,
                         weight_offset=offset, eps=eps, normed=normed)
    torch.cuda.synchronize()
    out, norm, e_out, e_norm = reference(d["y"], d["residual"], post=post, post_weight=pw, gate=d["gate"],
                                         residual_scale=scale, pre=pre, pre_weight=nw, offset=offset, eps=eps)
    o, m = got if pre else (got, None)
    assert o.dtype is st
    check(o, out, e_out, "out")
    if pre:
        check(m, norm, e_norm, "normed")


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [
    (1, 2816), (1, 1), (3, 2), (5, 7), (2, 63), (7, 64), (9, 1001), (4, 2047), (33, 2048), (5, 2056), (8, 4096),
    (3, 4104), (2, 8192), (2, 16384), (3, 16383), (5000, 64), (4099, 2040), (513, 704), (1025, 504), (1024, 1024), (2, 8200)])
def test_sizes(T, H):
    run_case(T, H)


@pytest.mark.gpu
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("H", [256, 333])
def test_types(yt, st, wt, H):
    run_case(17, H, yt, st, wt, offset=1.0)
    run_case(17, H, yt, st, wt, nt=F32 if st is BF else BF)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [None, "number", "scalar", "channel", "token", "full", "channel16"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_parts(gate, post, pre):
    run_case(19, 512, gate=gate, post=post, pre=pre)
    run_case(1, 77, gate=gate, post=post, pre=pre)


@pytest.mark.gpu
def test_no_weights_no_residual_and_plain_norm():
    d = make(6, 704, BF, BF, BF, None)
    out, normed = bgq.block_norm(d["y"], post_norm=True, pre_norm=True)
    ref = reference(d["y"], None, post=True, post_weight=None, gate=None, residual_scale=1.0, pre=True,
                    pre_weight=None, offset=0.0, eps=1e-6)
    check(out, ref[0], ref[2], "out")
    check(normed, ref[1], ref[3], "normed")
    plain = bgq.block_norm(d["y"], pre_weight=d["pre_weight"], want_out=False)
    ref = reference(d["y"], None, post=False, post_weight=None, gate=None, residual_scale=1.0, pre=True,
                    pre_weight=d["pre_weight"], offset=0.0, eps=1e-6)
    check(plain, ref[1], ref[3], "plain norm")


@pytest.mark.gpu
@pytest.mark.parametrize("H", [256, 250])
def test_strided_rows_and_places_behind_them(H):
    T, wide = 11, H + 24
    d = make(T, wide, BF, F32, BF, "full", seed=4)
    y, res, gate = d["y"][:, 8:8 + H], d["residual"][:, 4:4 + H], d["gate"][:, 16:16 + H]
    pw, nw = d["post_weight"][:H].clone(), d["pre_weight"][:H].clone()
    big = torch.full((2, T, wide), 77.0, device="cuda")
    out, normed = big[0][:, 8:8 + H], big[1][:, 12:12 + H]
    bgq.block_norm(y, res, post_weight=pw, gate=gate, pre_weight=nw, out=out, normed=normed)
    ref = reference(y, res, post=True, post_weight=pw, gate=gate, residual_scale=1.0, pre=True, pre_weight=nw,
                    offset=0.0, eps=1e-6)
    check(out, ref[0], ref[2], "out")
    check(normed, ref[1], ref[3], "normed")
    big[0][:, 8:8 + H] = 77.0
    big[1][:, 12:12 + H] = 77.0
    assert bool((big == 77.0).all())  # nothing else was written
    # one row for all tokens
    one = d["y"][:1, :wide].expand(T, wide)
    assert torch.equal(bgq.block_norm(one, d["residual"]), bgq.block_norm(one.contiguous(), d["residual"]))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 2816), (37, 2816), (5000, 512), (3, 101)])
def test_in_place(T, H):
    d = make(T, H, BF, BF, BF, "channel", seed=2)
    kw = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    out, normed = bgq.block_norm(d["y"], d["residual"], **kw)
    y, res = d["y"].clone(), d["residual"].clone()
    bgq.block_norm(y, res, out=res, normed=y, **kw)
    assert torch.equal(res, out) and torch.equal(y, normed)


@pytest.mark.gpu
def test_zero_infinite_and_nan_rows():
    d = make(6, 320, BF, BF, BF, "channel", seed=3)
    d["y"][1] = 0
    d["y"][2, 5] = float("inf")
    d["y"][3, 7] = float("nan")
    d["residual"][4, 9] = float("nan")
    d["residual"][1] = 0
    kw = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    out, normed = bgq.block_norm(d["y"], d["residual"], **kw)
    ref = reference(d["y"], d["residual"], post=True, residual_scale=1.0, pre=True, offset=0.0, eps=1e-6, **kw)
    check(out, ref[0], ref[2], "out")
    check(normed, ref[1], ref[3], "normed")
    assert bool((out[1] == 0).all()) and bool((normed[1] == 0).all())


@pytest.mark.gpu
def test_no_rows():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    out, normed = bgq.block_norm(e, e, post_norm=True, pre_norm=True)
    assert out.shape == normed.shape == (0, 64)


@pytest.mark.gpu
def test_other_stream_and_graph():
    d = make(40, 2816, BF, BF, BF, "token", seed=5)
    kw = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    want = bgq.block_norm(d["y"], d["residual"], **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = bgq.block_norm(d["y"], d["residual"], stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, normed = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bgq.block_norm(d["y"], d["residual"], out=out, normed=normed, **kw)
    for rep in range(3):
        d["y"].copy_(torch.randn(40, 2816, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        eager = bgq.block_norm(d["y"], d["residual"], **kw)
        assert torch.equal(out, eager[0]) and torch.equal(normed, eager[1]), rep


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(y=torch.float16), dict(out=F32), dict(gate=(3, 3)), dict(post_weight=63), dict(pre_norm=False, normed=True),
    dict(want_out=False), dict(y_t=True)])
def test_binding_refusals(kw):
    y = torch.zeros(4, 64, dtype=kw.get("y", BF), device="cuda")
    res = torch.zeros(4, 64, dtype=BF, device="cuda")
    args = {}
    if "out" in kw:
        args["out"] = torch.zeros(4, 64, dtype=kw["out"], device="cuda")
    if "gate" in kw:
        args["gate"] = torch.zeros(*kw["gate"], device="cuda")
    if "post_weight" in kw:
        args["post_weight"] = torch.zeros(kw["post_weight"], dtype=BF, device="cuda")
    if "normed" in kw:
        args["normed"] = torch.zeros(4, 64, dtype=BF, device="cuda")
    if "want_out" in kw:
        args["want_out"] = False
    if "y_t" in kw:
        y = torch.zeros(64, 4, dtype=BF, device="cuda").T
    with pytest.raises(ValueError):
        bgq.block_norm(y, res, **args)
