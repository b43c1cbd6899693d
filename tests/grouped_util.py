"""Plain 64-bit forms of the products grouped by expert and of the microscaled values,
and the inputs of their tests."""
import torch

U = 2.0 ** -24
F64 = torch.float64
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def offsets_of(sizes, first=0, device="cuda"):
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device=device)


def decode(codes, scales):
    """64-bit values of codes [..., K / 2] under scale bytes [..., K / 32]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=F64, device=codes.device)
    c = codes.view(torch.uint8).long()
    v = torch.stack([grid[c & 15], grid[c >> 4]], -1).flatten(-2)
    s = scales.view(torch.uint8).to(F64)
    unit = torch.where(s == 255, torch.nan, torch.exp2(s - 127)).repeat_interleave(32, -1)
    return v * unit


def encode(v):
    """(codes, scale bytes) of 64-bit values [..., K], by the nearest of the grid's values."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    _, e = torch.frexp(torch.where(bad, 1.0, amax))
    s = torch.where(amax > 0, e.long() - 3, -127).clamp(-127, 127)
    a = (b.abs() * torch.exp2(-s.to(F64))).clamp(max=6.0)
    grid = torch.tensor(GRID, dtype=F64, device=v.device)
    gap = (a.unsqueeze(-1) - grid).abs()
    near = gap.amin(-1, keepdim=True)
    tie = gap == near  # one or two neighbours: of two the even code
    n = torch.arange(8, device=v.device)
    code = torch.where(tie & (n % 2 == 0), n, torch.where(tie, n + 8, 99)).amin(-1) % 8
    code = torch.where(bad, 0, code + 8 * torch.signbit(b).long()).flatten(-2)
    byte = torch.where(bad, 255, s + 127).squeeze(-1)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), byte.to(torch.uint8)


def random_mx(g, *shape, spread=3):
    """Random codes and scale bytes around 1."""
    K = shape[-1]
    codes = torch.randint(0, 256, shape[:-1] + (K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(127 - spread, 128 + spread, shape[:-1] + (K // 32,), generator=g, device="cuda").to(torch.uint8)
    return codes, scales


def product(x, w, offsets):
    """(values, sums of the terms' magnitudes) of rows x [A, K] and w [E, N, K] in 64 bits; rows of no
    expert are NaN."""
    out = torch.full((x.shape[0], w.shape[1]), torch.nan, dtype=F64, device=x.device)
    size = out.clone()
    ends = offsets.tolist()
    for e in range(w.shape[0]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            out[a:b] = x[a:b].to(F64) @ w[e].to(F64).t()
            size[a:b] = x[a:b].to(F64).abs() @ w[e].to(F64).abs().t()
    return out, size


def gradient(dy, x, offsets):
    """(dw, sums of the terms' magnitudes) in 64 bits."""
    ends = offsets.tolist()
    E = len(ends) - 1
    out = torch.zeros(E, dy.shape[1], x.shape[1], dtype=F64, device=x.device)
    size = out.clone()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if b > a:
            out[e] = dy[a:b].to(F64).t() @ x[a:b].to(F64)
            size[e] = dy[a:b].to(F64).abs().t() @ x[a:b].to(F64).abs()
    return out, size


def check(got, ref, size, terms, what=""):
    """Products are exact and each of at most terms + 8 additions (the terms, then joins of partial
    sums) is within u of the terms' magnitudes; the store rounds once (half a step).  With signs as
    good as random the overall error grows with the root of the additions."""
    half = torch.finfo(got.dtype).eps / 2
    err = (got.to(F64) - ref).abs()
    bound = U * (terms + 8) * size * (1 + half) + half * ref.abs() + 1e-38
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(f"{what} worst error / bound {worst:.3f}", flush=True)
    assert bool((err <= bound).all())
    if got.dtype is torch.float32 and err.numel():
        assert float(torch.linalg.norm(err)) <= U * (terms + 8) ** 0.5 * float(torch.linalg.norm(size))
