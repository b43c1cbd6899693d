"""The few-token layer's second launch, replayed on the CPU: how its units of work
are cut over ranges, workgroups and waves, every index that follows from it, and
the order of its phases under workgroups that start late or not at all until
others have left."""
import random

import pytest

RANGES, WAVES, CHUNKS, THREADS, ROWS = 256, 8, 4, 512, 8
DEPTH, LAG = 4, 2


def geometry(K, gs, bits):
    nch = (K + 127) // 128
    log_split = 0 if nch <= 3 else 1 if nch <= 6 else 2 if nch <= 12 else 3
    return nch, log_split, 1 << log_split, WAVES >> log_split


def tiles_of(ids, E):
    """(tiles as lists of slots, slot -> tile) of the chosen experts ids[t][j]."""
    tiles, where, k = [], {}, len(ids[0])
    for e in range(E):
        rows = [t * k + j for t, row in enumerate(ids) for j, v in enumerate(row) if v == e]
        for i in range(0, len(rows), ROWS):
            for s in rows[i:i + ROWS]:
                where[s] = len(tiles)
            tiles.append((e, rows[i:i + ROWS]))
    return tiles, where


CASES = [(1, 8, 128, 2816, 704, 64, 4), (8, 8, 128, 2816, 704, 64, 4), (16, 8, 128, 2816, 768, 128, 8),
         (13, 2, 8, 256, 128, 32, 4), (16, 64, 64, 64, 64, 32, 8), (5, 1, 1, 4096, 4096, 32, 4),
         (16, 4, 4, 4096, 64, 64, 8), (3, 7, 1024, 192, 4032, 64, 4), (16, 64, 1024, 1088, 320, 64, 4),
         (2, 2, 3, 640, 2176, 128, 4)]


@pytest.mark.parametrize("T,k,E,H,I,gs,bits", CASES)
@pytest.mark.parametrize("down", [False, True])
def test_units_and_indices(T, k, E, H, I, gs, bits, down):
    rng = random.Random(T * 1000 + E)
    tiles, where = tiles_of([rng.sample(range(E), k) for _ in range(T)], E)
    A = T * k
    assert len(where) == A and len(tiles) <= A and all(1 <= len(r) <= ROWS for _, r in tiles)
    K = I if down else H
    G, upt = K // gs, (H // 32 if down else I // 16)
    nch, log_split, split, nu = geometry(K, gs, bits)
    N, groups = len(tiles) * upt, RANGES * nu

    def first(g):
        return N * g // groups

    # waves: their chunks partition the columns, at most CHUNKS each
    cover = []
    for ws in range(split):
        c0 = nch * ws >> log_split
        nc = (nch * (ws + 1) >> log_split) - c0
        assert nc <= CHUNKS
        cover += range(c0, c0 + nc)
    assert cover == list(range(nch))
    # a wave's table rows: lanes (block, row, piece) cover the slice from the piece in
    # which it begins, and the reads of 8 entries stay in the row
    pieces = 2 if 512 // gs <= 8 else 4
    rows = E * (H if down else 2 * I)
    for ws in range(split):
        c0 = nch * ws >> log_split
        nc = (nch * (ws + 1) >> log_split) - c0
        g0, ng = c0 * 128 // gs, min(nc * 128 // gs, G - c0 * 128 // gs)
        steps8 = (max(2, -(-nch // split)) * 128 // gs + 7) // 8
        for lr in range(16):
            sub = 2 * (lr * G + g0) & 15
            assert sub + 2 * ng <= 16 * pieces and sub + 16 * steps8 <= 16 * pieces and ng <= 8 * steps8
            for base in (0, rows - 16):  # the same piece for all units
                assert 2 * ((base + lr) * G + g0) & 15 == sub
    # units to tiles by a multiplication
    m = -(-2**31 // upt)
    for u in {0, upt - 1, upt, N - 1, max(N - upt, 0), max(N - upt - 1, 0), N // 2}:
        assert m < 2**32 and 2 * u * m >> 32 == u // upt
    done, seen = [0] * len(tiles), 0
    for r in range(RANGES):
        lo, hi = first(r * nu), first((r + 1) * nu)
        for i in range(nu):
            u0, u1 = first(r * nu + i), first(r * nu + i + 1)
            assert lo <= u0 <= u1 <= hi
            for u in range(u0, u1):
                seen += 1
                tile, c = divmod(u, upt)
                e = tiles[tile][0]
                for b in range(2):
                    row = e * H + 32 * c + 16 * b if down else e * 2 * I + 16 * c + (I if b else 0)
                    assert row + 16 <= E * (H if down else 2 * I)
        # what the range adds to its tiles' counters
        if lo < hi:
            assert (hi - 1) // upt - lo // upt < THREADS
            for tid in range(THREADS):
                t0 = lo // upt + tid
                if t0 * upt < hi:
                    done[t0] += min(hi, (t0 + 1) * upt) - max(lo, t0 * upt)
    assert seen == N and done == [upt] * len(tiles)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_shares_of_a_unit(split):
    """The waves of a unit, scheduled at random: every unit's outputs are made once,
    after all its shares and before their place is written again."""
    for units in range(24):
        for seed in range(4):
            rng = random.Random(seed)
            arrived, finished, outputs = [0] * DEPTH, [0] * DEPTH, []
            place = [[None] * split for _ in range(DEPTH)]

            def wave(ws):
                for it in range(units + LAG):
                    j = it - LAG
                    if j >= 0 and j % split == ws:
                        while arrived[j % DEPTH] < (j // DEPTH + 1) * split:
                            yield False
                        assert place[j % DEPTH] == [j] * split
                        yield True
                        assert place[j % DEPTH] == [j] * split
                        outputs.append(j)
                        finished[j % DEPTH] = j // DEPTH + 1
                    if it < units:
                        while finished[it % DEPTH] < it // DEPTH:
                            yield False
                        place[it % DEPTH][ws] = it
                        yield True
                        arrived[it % DEPTH] += 1

            live, idle = {w: wave(w) for w in range(split)}, 0
            while live:
                w = rng.choice(sorted(live))
                try:
                    idle = 0 if next(live[w]) else idle + 1
                except StopIteration:
                    del live[w]
                    idle = 0
                assert idle < 1000, "no wave gets on"
            assert sorted(outputs) == list(range(units))


def run_order(T, tiles, slots_tile, resident, rng, ranges=20):
    """Workgroups as generators, only `resident` of them started at a time and the
    scheduler picking one at random; returns the steps taken."""
    flags = {"gu": [0] * ranges, "dn": [0] * ranges}
    units = {"gu": 5, "dn": 7}
    done = {"gu": [0] * tiles, "dn": [0] * tiles}
    outputs = [0] * T

    def claim(name, r):
        won, flags[name][r] = not flags[name][r], 1
        return won

    def take(name):  # any untaken range
        while True:
            yield
            free = [i for i in range(ranges) if not flags[name][i]]
            if not free:
                return None
            yield
            if claim(name, free[0]):
                return free[0]

    def span(name, r):
        N = tiles * units[name]
        return range(N * r // ranges, N * (r + 1) // ranges)

    def group(b):
        own = {}
        for name in ("gu", "dn"):  # both of its own at once
            yield
            own[name] = claim(name, b)
        for name in ("gu", "dn"):
            r = b if own[name] else (yield from take(name))
            while r is not None:
                if name == "dn":  # one wait for all tiles of the range
                    for tile in {u // units["dn"] for u in span(name, r)}:
                        while done["gu"][tile] < units["gu"]:
                            yield "wait"
                for u in span(name, r):
                    yield
                for u in span(name, r):
                    done[name][u // units[name]] += 1
                r = yield from take(name)
        if b < T:  # workgroup t finishes token t
            for tile in slots_tile[b]:
                while done["dn"][tile] < units["dn"]:
                    yield "wait"
            outputs[b] += 1

    waiting, live, steps, idle = [group(b) for b in range(ranges)], [], 0, 0
    while waiting or live:
        while waiting and len(live) < resident:
            live.append(waiting.pop(0))
        g = rng.choice(live)
        try:
            idle = idle + 1 if next(g) == "wait" else 0
        except StopIteration:
            live.remove(g)
            idle = 0
        steps += 1
        assert idle < 20000, "nobody makes progress"
    assert outputs == [1] * T and done["gu"] == [units["gu"]] * tiles and done["dn"] == [units["dn"]] * tiles
    return steps


@pytest.mark.parametrize("resident", [1, 2, 5, 12])
@pytest.mark.parametrize("T,tiles", [(1, 3), (4, 9), (16, 40)])
def test_every_wait_ends_however_few_workgroups_run(resident, T, tiles):
    rng = random.Random(resident * 100 + T)
    slots = [[rng.randrange(tiles) for _ in range(3)] for _ in range(T)]
    for _ in range(5):
        run_order(T, tiles, slots, resident, rng)
