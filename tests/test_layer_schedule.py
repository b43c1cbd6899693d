"""The few-token layer's second launch, replayed on the CPU: how its units of work
are cut over ranges, workgroups and waves, every index that follows from it, and
the order of its phases under workgroups that start late or not at all until
others have left."""
import random

import pytest

RANGES, WAVES, CHUNKS, THREADS, ROWS = 256, 8, 4, 512, 8


def geometry(K, gs, bits):
    nch = (K + 127) // 128
    log_split = 0 if nch <= 4 else 1 if nch <= 8 else 2 if nch <= 16 else 3
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
    # tables: pieces of 16 bytes, two a thread, inside the buffer
    assert nu * 8 * G <= 2 * THREADS and nu * 64 * G <= 8 * 4096 // gs * 8
    assert (16 * G * 2) % 16 == 0
    # chain sums
    chain = 32 if gs == 32 else 64
    per_chunk = 128 // chain
    assert CHUNKS * per_chunk * 16 == 64 * per_chunk
    done, seen = [0] * len(tiles), 0
    for r in range(RANGES):
        lo, hi = first(r * nu), first((r + 1) * nu)
        steps = max(first(r * nu + i + 1) - first(r * nu + i) for i in range(nu))
        for i in range(nu):
            u0, u1 = first(r * nu + i), first(r * nu + i + 1)
            assert lo <= u0 <= u1 <= hi and u1 - u0 <= steps
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
    # outputs: threads over rows and columns
    out = 256 if down else 128
    for p in {0, 1, out - 1, nu * out - 1}:
        i, rr, c = p // out, p // (out // ROWS) % ROWS, p % (out // ROWS)
        assert i < nu and rr < ROWS and c < (32 if down else 16)


def run_order(T, tiles, slots_tile, resident, rng, ranges=12):
    """Workgroups as generators, only `resident` of them started at a time and the
    scheduler picking one at random; returns the steps taken."""
    flags = {"gu": [0] * ranges, "dn": [0] * ranges, "tok": [0] * T}
    units = {"gu": 5, "dn": 7}
    done = {"gu": [0] * tiles, "dn": [0] * tiles}
    outputs = [0] * T

    def take(name, own):
        n = len(flags[name])
        if own is not None:
            yield
            if not flags[name][own]:
                flags[name][own] = 1
                return own
        while True:
            yield
            free = [i for i in range(n) if not flags[name][i]]
            if not free:
                return None
            yield
            if not flags[name][free[0]]:
                flags[name][free[0]] = 1
                return free[0]

    def span(name, r):
        N = tiles * units[name]
        return range(N * r // ranges, N * (r + 1) // ranges)

    def group(b):
        for name in ("gu", "dn"):
            r = yield from take(name, b)
            while r is not None:
                for u in span(name, r):
                    if name == "dn":
                        while done["gu"][u // units["dn"]] < units["gu"]:
                            yield "wait"
                    yield
                for u in span(name, r):
                    done[name][u // units[name]] += 1
                r = yield from take(name, None)
        t = yield from take("tok", b % T)
        while t is not None:
            for tile in slots_tile[t]:
                while done["dn"][tile] < units["dn"]:
                    yield "wait"
            outputs[t] += 1
            t = yield from take("tok", None)

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
