"""The router's product in every tile of its launch rule, with several and uneven
column steps a wave, against 64 bits.

Products are exact, so a logit is off by its fp32 sums alone (u = 2^-24): an MFMA adds
32 products to its accumulator, a wave takes at most ceil(H / 32 / waves) steps of 32
columns, three MFMAs each for fp32 weights, then the waves' sums are added.  That is
L = 32 ceil(H / 32 / waves) parts + waves roundings, each within u of the terms'
magnitudes; the mean of squares is off by a like share, half of it in the root, and four
more roundings follow."""
import math

import pytest
import torch

import bit_gathered_quantized_amd as bgq

U = 2.0 ** -24


def tile_of(T, E):
    """(row blocks, expert blocks, waves) of 16, as the launch chooses them."""
    groups = lambda m, n: -(-T // (16 * m)) * -(-E // (16 * n))  # noqa: E731
    if groups(4, 4) > 256:
        return 4, 4, 4
    if groups(4, 4) > 128:
        return 4, 4, 8
    return (2, 2, 8) if groups(2, 2) >= 128 else (1, 1, 16)


def by_xcd(T, E):
    m, n, _ = tile_of(T, E)
    return -(-E // (16 * n)) > 4 and -(-T // (16 * m)) >= 8


# tokens, experts, H, the tile, token blocks grouped by XCD
CASES = [(1037, 1024, 1088, (4, 4, 4), True), (4001, 512, 2816, (4, 4, 4), True), (8321, 100, 1088, (4, 4, 4), False),
         (4201, 200, 4096, (4, 4, 4), False), (1025, 500, 2816, (4, 4, 8), True), (2049, 200, 1088, (4, 4, 8), False),
         (8190, 128, 2112, (4, 4, 8), False), (1000, 128, 1088, (2, 2, 8), False), (300, 400, 2816, (2, 2, 8), True),
         (100, 129, 1088, (1, 1, 16), False), (150, 90, 2880, (1, 1, 16), True), (9, 128, 16384, (1, 1, 16), False)]


@pytest.mark.parametrize("T,E,H,tile,xcd", CASES)
def test_cases_reach_their_tile(T, E, H, tile, xcd):
    assert tile_of(T, E) == tile and by_xcd(T, E) == xcd
    assert H // 32 > 2 * tile[2]  # more than two steps a wave


def wave_roundings(H, waves, parts):
    return 32 * math.ceil(H / 32 / waves) * parts + waves


@pytest.mark.gpu
@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H,tile,xcd", CASES)
def test_values(wt, T, E, H, tile, xcd):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(T, H) * (1 + r(H).abs())).bfloat16()
    w = (r(E, H) * (2.0 / math.sqrt(H))).to(wt)
    k, eps = min(E, 8), 1e-6
    logits, ids, _ = bgq.router_forward(x, w, k, eps=eps)
    xd, wd = x.double(), w.double()
    rstd = torch.rsqrt(xd.square().mean(-1, keepdim=True) + eps)
    ref, size = rstd * (xd @ wd.T), rstd * (xd.abs() @ wd.abs().T)
    L, Ls = wave_roundings(H, tile[2], 3 if wt is torch.float32 else 1), wave_roundings(H, tile[2], 1)
    err, bound = (logits.double() - ref).abs(), U * (L * size + (Ls / 2 + 4) * ref.abs()) + 1e-30
    rel = float(torch.linalg.norm(err) / torch.linalg.norm(size))
    print(f"worst error / bound {float((err / bound).max()):.3f}, overall {rel:.2e} of the terms", flush=True)
    assert bool((err <= bound).all())
    assert rel <= U * math.sqrt(L)  # signs as good as random
    assert torch.equal(ids.long(), logits.sort(dim=-1, descending=True, stable=True).indices[:, :k])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 2100])
def test_rows_past_32_bit_offsets(T):
    """Rows 2^22 (8 tokens: the widest there is) or 2^20 elements apart."""
    H, stride = 320, 1 << (22 if T == 8 else 20)
    rows = 600 if T == 8 else T
    big = torch.zeros(rows, stride, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    view = big[rows - T:, stride - H:]
    view.copy_(x)
    w = torch.randn(40, H, device="cuda").bfloat16()
    for a, b in zip(bgq.router_forward(view, w, 3), bgq.router_forward(x, w, 3)):
        assert torch.equal(a, b)
