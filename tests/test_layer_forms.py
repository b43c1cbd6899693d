"""The whole layer in every compiled form of the few-token matmuls -- group size, code
width and the chunks of 128 columns that a wave takes (2, 3 or 4) -- with slices that
end inside a chunk, and the arguments and formats of both forms of the layer."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq
import test_layer as base
import test_layer_schedule as schedule

# hidden and expert widths: the chunks of a wave in both matmuls; those that end in
# half a chunk are no multiples of 128
SIZES = [(256, 128, 2), (2048, 512, 2), (1984, 448, 2), (640, 384, 3), (1344, 320, 3), (2816, 704, 3),
         (4096, 3328, 4), (3264, 4032, 4)]


def chunks_of_a_wave(K):
    nch, log_split, split, _ = schedule.geometry(K, 64, 4)
    return max(2, -(-nch // split))


def cases():
    return [(H, I, gs) for H, I, _ in SIZES for gs in (32, 64, 128) if H % gs == 0 and I % gs == 0]


def test_sizes_reach_every_form():
    assert all(chunks_of_a_wave(H) == chunks_of_a_wave(I) == cpw for H, I, cpw in SIZES)
    for gs in (32, 64, 128):
        ways = {chunks_of_a_wave(H) for H, I, g in cases() if g == gs}
        assert ways == {2, 3, 4}
        assert gs == 128 or {chunks_of_a_wave(H) for H, I, g in cases() if g == gs and H % 128 == I % 128 == 64} == {2, 3, 4}


@pytest.mark.parametrize("H,I,gs", cases())
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,k,E", [(11, 2, 3), (1, 2, 3)])
def test_indices(H, I, gs, bits, T, k, E):
    """The units, tables and rows of these sizes, before any of them runs."""
    for down in (False, True):
        schedule.test_units_and_indices(T, k, E, H, I, gs, bits, down)


@pytest.mark.gpu
@pytest.mark.parametrize("H,I,gs", cases())
@pytest.mark.parametrize("bits", [4, 8])
def test_values(H, I, gs, bits):
    """11 tokens of 3 experts: tiles of 8 rows and of fewer."""
    rel, *_ = base.run_case(11, 3, H, I, 2, gs=gs, bits=bits, swiglu=gs == 64, seed=H + gs)
    assert rel <= 3 * base.R + 100 * base.U


@pytest.mark.gpu
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_one_token_with_biases_of_their_own(gs, bits):
    for H, I, cpw in SIZES:
        if H % gs == 0 and I % gs == 0:
            base.run_case(1, 4, H, I, 3, gs=gs, bits=bits, centred=False, seed=I + bits)


def tail_args(w):
    return dict(expert_scale=w["expert_scale"], post_weight=w["post"], pre_weight=w["pre"])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 24])
@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16])
def test_weights_stored_as_their_distance_from_one(T, wt):
    """1 + d is exact in fp32, so both ways give the same bits."""
    w = base.make(16, 512, 256, seed=20)
    d = {n: (torch.randint(-60, 60, (512,), device="cuda") / 128).to(wt) for n in ("norm", "post", "pre")}
    x, gate = base.tokens(w, T), w["r"](512)
    kw = lambda off: {n + "_weight": (d[n] if off else 1 + d[n].float()) for n in d}  # noqa: E731
    want = base.layer_of(w, 4, **kw(0))(x, residual=x, gate=gate)
    got = base.layer_of(w, 4, weight_offset=1.0, **kw(1))(x, residual=x, gate=gate)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("gs,bits,I", [(32, 4, 192), (128, 4, 256), (64, 8, 192), (32, 8, 192), (128, 8, 256)])
@pytest.mark.parametrize("swiglu,fp32_intermediate", [(False, False), (True, False), (False, True), (True, True)])
def test_many_tokens_of_every_format_equal_the_operators_in_turn(gs, bits, I, swiglu, fp32_intermediate):
    T, k = 45, 3
    w = base.make(12, 640, I, gs=gs, bits=bits, seed=21)
    x = base.tokens(w, T)
    layer = base.layer_of(w, k, norm_weight=w["norm"], swiglu=swiglu, fp32_intermediate=fp32_intermediate, **tail_args(w))
    out, normed = layer(x, residual=x)
    n = bgq.block_norm(x, pre_weight=w["norm"], want_out=False)
    _, ids, p = bgq.router_forward(x, w["router"], k, expert_scale=w["expert_scale"])
    y = bgq.expert_ffn_forward(n, ids, p, w["w_gateup"], w["s_gateup"], w["b_gateup"], w["w_down"], w["s_down"],
                               w["b_down"], fp32_out=True, swiglu=swiglu, fp32_intermediate=fp32_intermediate)
    want = bgq.block_norm(y, x, post_weight=w["post"], pre_weight=w["pre"])
    assert torch.equal(out, want[0]) and torch.equal(normed, want[1])


@pytest.mark.gpu
def test_few_tokens_keep_one_precision():
    """Up to 16 tokens h has 16 bits whatever the handle asks of larger batches."""
    w = base.make(12, 640, 192, seed=22)
    x = base.tokens(w, 9)
    a, b = (base.layer_of(w, 3, norm_weight=w["norm"], fp32_intermediate=f, **tail_args(w))(x, residual=x) for f in (False, True))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.gpu
def test_one_workspace_for_every_batch():
    w = base.make(16, 512, 256, seed=23)
    layer = base.layer_of(w, 4, norm_weight=w["norm"], **tail_args(w))
    ws = torch.empty(layer.workspace_bytes(17), dtype=torch.uint8, device="cuda")
    for T in (17, 16, 3, 1, 17):
        x = base.tokens(w, T)
        assert all(torch.equal(a, b) for a, b in zip(layer(x, residual=x, workspace=ws), layer(x, residual=x)))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 40])
@pytest.mark.parametrize("gs,bits", [(64, 4), (32, 4), (64, 8)])
def test_bad_tokens_stay_by_themselves(T, gs, bits):
    """A NaN or an infinity makes its own token NaN and no other; the others are those
    of the batch with harmless tokens in their places, up to the roundings that go by an
    expert's number of rows (2^-9 of n, of h and of the output, and those of the block
    scales' operands: as a whole 4 of them)."""
    w = base.make(12, 640, 192, gs=gs, bits=bits, seed=24)
    layer = base.layer_of(w, 3, norm_weight=w["norm"], **tail_args(w))
    good = base.tokens(w, T)
    x = good.clone()
    x[1, 3], x[2, 600], x[3] = float("nan"), float("inf"), 0
    ids = torch.empty(T, 3, dtype=torch.int32, device="cuda")
    out, normed = layer(x, ids=ids)
    want, want_normed = layer(good)
    assert bool(((ids >= 0) & (ids < 12)).all())
    for got, ref in ((out, want), (normed, want_normed)):
        assert bool(torch.isnan(got[1:3]).all()) and bool((got[3] == 0).all())
        rest = [0] + list(range(4, T))
        a, b = got[rest].double(), ref[rest].double()
        assert bool(torch.isfinite(a).all())
        assert float(torch.linalg.norm(a - b) / torch.linalg.norm(b)) <= 4 * 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("H", [333, 1001, 16383])
def test_norm_of_bad_rows_off_16_bytes(H):
    g = torch.Generator(device="cuda").manual_seed(H)
    y = torch.randn(6, H, generator=g, device="cuda").bfloat16()
    res = torch.randn(6, H, generator=g, device="cuda").bfloat16()
    want, want_normed = bgq.block_norm(y, res, post_norm=True, pre_norm=True)
    y2 = y.clone()
    y2[2, H - 1], y2[4, 0] = float("nan"), float("inf")
    out, normed = bgq.block_norm(y2, res, post_norm=True, pre_norm=True)
    keep = [0, 1, 3, 5]
    assert torch.equal(out[keep], want[keep]) and torch.equal(normed[keep], want_normed[keep])
    assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(normed[2]).all()) and bool(torch.isnan(normed[4]).all())
    # an infinity's mean of squares is infinite: the rest of its row is 0 before the residual
    assert torch.isnan(out[4, 0]) and torch.equal(out[4, 1:], res[4, 1:])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 40])
def test_two_graphs_of_two_layers_at_once(T):
    """Two handles, captured with what they allocate, replayed together on two streams."""
    ws = [base.make(16, 512, 256, seed=s) for s in (25, 26)]
    layers = [base.layer_of(w, 4, norm_weight=w["norm"], **tail_args(w)) for w in ws]
    xs = [base.tokens(w, T) for w in ws]
    for layer, x in zip(layers, xs):
        layer(x, residual=x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for layer, x in zip(layers, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(x, residual=x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(3):
        for w, x in zip(ws, xs):
            x.copy_(base.tokens(w, T))
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for layer, x, got in zip(layers, xs, outs):
            assert all(torch.equal(a, b) for a, b in zip(got, layer(x, residual=x))), rep


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 20])
def test_weights_past_32_bit_offsets(T):
    """6.7 GB of gate|up codes: most experts lie past 2^32 bytes."""
    E, H, I, k = 200, 4096, 4096, 4
    if T <= 16:
        _, w, layer, x = base.run_case(T, E, H, I, k, bits=8, seed=27)
    else:
        w = base.make(E, H, I, bits=8, seed=27)
        layer, x = base.layer_of(w, k, norm_weight=w["norm"]), base.tokens(w, T)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    out = layer(x, ids=ids, out=torch.empty(T, H, device="cuda"))
    far = ids.amax(1) * (2 * I * H) > 2**32
    assert bool(far.any())
    # the same token by a layer of its experts alone, in the order of their logits
    t = int(far.nonzero()[0])
    own = ids[t].long()
    small = dict(w, **{n: w[n][own].contiguous() for n in w if n[:2] in ("w_", "s_", "b_")}, router=w["router"][own].contiguous())
    got = base.layer_of(small, k, norm_weight=w["norm"], expert_scale=w["expert_scale"][own] if T <= 16 else None)(
        x[t:t + 1].contiguous(), out=torch.empty(1, H, device="cuda"))[0].double()
    want = out[t].double()
    # the order of the sums over experts, and n and h in bf16 in the larger batch
    assert float(torch.linalg.norm(got - want) / torch.linalg.norm(want)) <= (1e-5 if T <= 16 else 3 * 2.0 ** -9)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12])
def test_same_bits_beside_other_work(T):
    """Workgroups that start late, because other streams hold the GPU, leave their ranges
    to others: the bits stay."""
    w = base.make(32, 704, 320, seed=28)
    layer = base.layer_of(w, 6, norm_weight=w["norm"], **tail_args(w))
    x, other = base.tokens(w, T), base.tokens(w, T)
    want = layer(x, residual=x)
    a = torch.randn(2048, 2048, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(60):
        for s in streams:
            with torch.cuda.stream(s):
                _ = (a @ a).sum()
        if i % 3 == 0:
            layer(other, residual=other)
        got = layer(x, residual=x)
        assert all(torch.equal(u, v) for u, v in zip(got, want)), i
    torch.cuda.synchronize()
