"""How the grouped products and the weights' gradient share out their work, replayed on the
CPU as the kernels do it: every row and column is computed once, nothing outside x, w and out is
touched whatever the offsets hold, and no buffer in LDS is overwritten while it is read."""
import math
import random

import pytest

UNIT, BN, GROUPS, GM = 32, 256, 256, 8


class Share:
    """The tiles of a call: strips of `bm` rows (with `tall` ones of more than half by blocks half as wide)."""

    def __init__(self, offsets, A, E, N, bm, tall):
        self.o, self.A, self.E, self.N, self.bm, self.tall = offsets, A, E, N, bm, tall
        self.per = -(-N // UNIT)
        rows = [self.rows(e)[1] - self.rows(e)[0] for e in range(E)]
        most = A // bm + min(A, E) if offsets is not None else -(-A // bm)
        strips = min(sum(-(-r // bm) for r in rows), most)
        high = min(sum(r // bm + (r % bm > bm // 2) for r in rows), strips) if tall else 0
        units = most * self.per
        self.groups = GROUPS if units >= GROUPS else -(-units // 8) * 8
        least = -(-self.per * UNIT // BN)
        jump = (self.per - least + 62) // 63
        best = None
        for lane in range(64):
            mine = min(least + lane * jump, self.per)
            t = min(2 * mine, self.per)
            tiles = (strips - high) * mine + high * t
            price = 0.0
            if tiles:
                low = min(bm / 2 if tall else bm, A / strips)
                total = (strips - high) * mine * (UNIT * math.ceil(self.per / mine - 1e-3) + 0.5 * low + 32)
                total += high * t * (UNIT * math.ceil(self.per / t - 1e-3) + 0.375 * bm + 32) if tall else 0
                price = math.ceil(tiles / self.groups - 1e-3) * total / tiles
            if best is None or price < best[0]:
                best = (price, min(least + lane * max(jump, 1), self.per))
        self.blocks = best[1]
        self.limit = most * self.of(tall)
        self.upto, before = [], 0
        for r in rows:
            full, rest = divmod(r, bm)
            mine = full * self.of(tall) + (self.of(tall and rest > bm // 2) if rest else 0)
            before = min(before + min(mine, self.limit), self.limit)
            self.upto.append(before)

    def of(self, tall):
        return min(2 * self.blocks, self.per) if tall else self.blocks

    def rows(self, e):
        if self.o is None:
            return 0, self.A
        lo = min(max(self.o[e], 0), self.A)
        return lo, min(max(self.o[e + 1], lo), self.A)

    def find(self, at):
        e = next(i for i, u in enumerate(self.upto) if u > at)
        local = at - (self.upto[e - 1] if e else 0)
        lo, hi = self.rows(e)
        count = -(-(hi - lo) // self.bm)
        rest = (hi - lo) % self.bm
        short = self.tall and 0 < rest <= self.bm // 2
        alike, high = count - short, self.of(self.tall)
        end = short and local >= alike * high
        mine = self.of(self.tall and not end)
        if end:
            strip, n = count - 1, local - alike * high
        else:
            group, r = divmod(local, GM * high)
            together = min(alike - group * GM, GM)
            n, s = divmod(r, together)
            strip = group * GM + s
        narrow, wide = divmod(self.per, mine)
        unit, units = n * narrow + min(n, wide), narrow + (n < wide)
        row = min(lo + strip * self.bm, hi)
        rows = min(self.bm, hi - row)
        cols = min(UNIT * units, self.N - UNIT * unit)
        assert not (self.tall and rows > self.bm // 2) or cols <= BN // 2
        assert cols <= BN
        return e, row, rows, UNIT * unit, cols

    def tiles(self):
        """Tile numbers in each workgroup's order."""
        count = self.upto[-1]
        share, per_xcd = -(-count // 8), self.groups // 8
        for group in range(self.groups):
            xcd, slot = group & 7, group >> 3
            yield range(xcd * share + slot, min((xcd + 1) * share, count), per_xcd)


CASES = [(16384, 128, 1408), (16381, 8, 2816), (64, 128, 1408), (8, 128, 2816), (333, 5, 264), (1, 1, 8), (5000, 1, 4096),
         (700, 1024, 40), (20, 3, 8192), (3000, 2, 72)]


@pytest.mark.parametrize("bm,tall", [(256, True), (256, False), (128, False), (32, False)])
@pytest.mark.parametrize("A,E,N", CASES)
def test_every_row_and_column_once(A, E, N, bm, tall):
    rng = random.Random(A + E + N + bm)
    for kind in range(3):
        if kind == 2:
            if E > 1:
                continue
            offsets = None
        else:
            cuts = sorted(rng.choices(range(A + 1), k=E + 1) if kind else [0, A] + rng.choices(range(A + 1), k=E - 1))
            offsets = cuts
        share = Share(offsets, A, E, N, bm, tall)
        units = {}
        seen = 0
        for tiles in share.tiles():
            for at in tiles:
                seen += 1
                e, row, rows, n0, cols = share.find(at)
                lo, hi = share.rows(e)
                assert lo <= row and rows >= 1 and row + rows <= hi and 0 <= n0 and cols >= 1 and n0 + cols <= N
                for s in range(row, row + rows, 16):
                    for c in range(n0, n0 + cols, UNIT):
                        assert (s, c) not in units
                        units[s, c] = e
        assert seen == share.upto[-1]
        want = 0
        for e in range(E):
            lo, hi = share.rows(e)
            want += sum(-(-min(bm, hi - r) // 16) for r in range(lo, hi, bm)) * share.per
        assert len(units) == want


@pytest.mark.parametrize("bm,tall", [(256, True), (256, False), (128, False), (32, False)])
def test_offsets_that_do_not_rise(bm, tall):
    rng = random.Random(bm)
    for _ in range(60):
        A, E, N = rng.randint(1, 3000), rng.randint(1, 40), 8 * rng.randint(1, 200)
        offsets = [rng.choice([rng.randint(-50, A + 50), -2**31, 2**31 - 1, 0, A]) for _ in range(E + 1)]
        share = Share(offsets, A, E, N, bm, tall)
        for tiles in share.tiles():
            for at in tiles:
                e, row, rows, n0, cols = share.find(at)
                assert 0 <= e < E and 0 <= row and rows >= 1 and row + rows <= A and 0 <= n0 and cols >= 1 and n0 + cols <= N


@pytest.mark.parametrize("D", [2, 3, 4])
def test_buffers_and_tiles_told(D):
    """Copies of the stage D - 1 ahead start after a step's barrier; a tile is told when the last stage of the one
    before it is issued, into one of 8 places, and read after the barrier of its first stage."""
    for stages in (1, 2, 3, 7):
        tiles = 23
        total = stages * tiles
        told = {}  # tile -> step after whose barrier it was written (-1: before the first)
        told[0] = -1
        for stage in range(total):
            issued = max(stage - (D - 1), -1)  # the step in which this stage is issued
            if (stage + 1) % stages == 0 and (stage + 1) // stages < tiles:
                told[(stage + 1) // stages] = issued
            # the buffer's last reader, stage - D, was done by the barrier of step stage - D + 1
            assert issued == -1 or stage - D + 1 <= issued
        for t in range(tiles):
            read = t * stages  # after this barrier
            assert told[t] < read
            later = t + 8
            assert later >= tiles or told[later] > read  # by then every wave has passed a later barrier


def dw_chunks(n, k, E):
    return -(-n // 3) if n * k * E >= 256 * 8 * 3 else n


@pytest.mark.parametrize("N,K,E", [(1408, 2816, 128), (264, 1000, 5), (8, 8, 1), (4096, 4096, 8), (136, 128, 4), (2816, 704, 64)])
def test_gradient_chunks_cover_every_tile(N, K, E):
    tn, tk = -(-N // 128), -(-K // 256)
    chunks = dw_chunks(tn, tk, E)
    count = chunks * tk * E
    share = -(-count // 8)
    groups = 256 if count >= 256 else -(-count // 8) * 8
    seen = set()
    for g in range(groups):
        for number in range((g & 7) * share + (g >> 3), min((g & 7) * share + share, count), groups >> 3):
            expert, rest = divmod(number, chunks * tk)
            kb, chunk = divmod(rest, chunks)
            for n in range(chunk * tn // chunks, (chunk + 1) * tn // chunks):
                assert (expert, kb, n) not in seen
                seen.add((expert, kb, n))
    assert len(seen) == tn * tk * E


def test_gradient_buffers():
    """x's three slots are filled in turn, a block of up to three stages once for its chunk; a slot is never filled
    while one of the two steps under way reads it, and holds what the step that reads it wants."""
    rng, D = random.Random(4), 3
    for _ in range(300):
        steps = []  # (x's slot, what it must hold, filled here?)
        slot = base = 0
        for block in range(rng.randint(1, 12)):
            stages = rng.choice([1, 1, 2, 2, 3, 3, 4, 5, 9])
            for n in range(rng.randint(1, 3)):
                fresh = n == 0 or stages > D
                if fresh:
                    base = slot
                for s in range(stages):
                    if fresh:
                        assert slot == (base + s) % D
                        slot = (slot + 1) % D
                    steps.append(((base + s) % D, (block, s), fresh))
        held = [None] * D
        for i in range(min(D - 1, len(steps))):  # before the first barrier
            if steps[i][2]:
                held[steps[i][0]] = steps[i][1]
        for i, (slot_read, want, _) in enumerate(steps):
            assert held[slot_read] == want  # barrier of step i: its copies are there
            ahead = i + D - 1
            if ahead < len(steps) and steps[ahead][2]:
                assert steps[ahead][0] not in [steps[j][0] for j in range(i, ahead)]
                held[steps[ahead][0]] = steps[ahead][1]
