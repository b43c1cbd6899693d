"""The cut of the few-token layer's matmuls (csrc/layer_cut.h), compiled for the host
and compared with the formulas that tests/test_layer_schedule.py replays, and the order
of its phases with the short way by which a workgroup ends a phase."""
import ctypes
import os
import random
import re
import subprocess

import pytest

import test_layer_schedule as schedule

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gathered_quantized_amd", "csrc")

SOURCE = r"""
#include "layer_cut.h"
using namespace moe::cut;
extern "C" {
int c_chunks(int K) { return chunks(K); }
int c_split_log(int n) { return split_log(n); }
int c_first_chunk(int n, int l, int w) { return first_chunk(n, l, w); }
int c_most_chunks(int n) { return most_chunks(n); }
int c_slice_columns(int K, int c, int n) { return slice_columns(K, c, n); }
int c_slice_group(int gs, int c) { return slice_group(gs, c); }
int c_slice_groups(int gs, int G, int c, int n) { return slice_groups(gs, G, c, n); }
int c_units_of_tile(int d, int H, int I) { return units_of_tile(d, H, I); }
int c_first_unit(int N, int s, int l) { return first_unit(N, s, l); }
uint32_t c_unit_magic(uint32_t u) { return unit_magic(u); }
int c_tile_of_unit(int u, uint32_t m) { return tile_of_unit(u, m); }
int c_expert_rows(int d, int H, int I) { return expert_rows(d, H, I); }
uint32_t c_unit_row(int d, int r, int e, int c) { return unit_row(d, r, e, c); }
int c_block_rows(int d, int I) { return block_rows(d, I); }
uint32_t c_table_load(int G, int g, int rows, int b, int r, int p) { return table_load(G, g, rows, b, r, p); }
int c_table_start(int G, int g, int r) { return table_start(G, g, r); }
int c_table_pieces(int gs) { return table_pieces(gs); }
int c_constant(int i) { const int v[] = {kWaves, kRanges, kTileRows, kChunk, kMaxChunks, kDepth, kLag}; return v[i]; }
// of the first 2^18 units, the first whose tile the multiplication gets wrong, or -1
int c_wrong_tile(uint32_t upt) {
    for (int u = 0; u < 1 << 18; ++u)
        if (tile_of_unit(u, unit_magic(upt)) != u / static_cast<int>(upt)) return u;
    return -1;
}
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    (d / "cut.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fPIC", "-shared", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-I", CSRC, str(d / "cut.cpp"), "-o", str(d / "cut.so")], check=True)
    lib = ctypes.CDLL(str(d / "cut.so"))
    for n in ("c_unit_magic", "c_unit_row", "c_table_load"):
        getattr(lib, n).restype = ctypes.c_uint32
    return lib


def test_constants(cut):
    names = ("WAVES", "RANGES", "ROWS", None, "CHUNKS", "DEPTH", "LAG")
    assert all(n is None or cut.c_constant(i) == getattr(schedule, n) for i, n in enumerate(names))
    assert cut.c_constant(3) == 128 and schedule.THREADS == 64 * schedule.WAVES
    # what the kernel's source still says for itself
    text = open(os.path.join(CSRC, "layer_few.hip")).read()
    assert re.search(r"kFewThreads = 64 \* kWaves;", text) and "static_assert(kRanges == kLayerRanges" in text
    assert re.search(r"constexpr int kLayerRanges = 256;", open(os.path.join(CSRC, "moe_internal.h")).read())


def test_units_to_tiles(cut):
    for upt in range(1, 257):
        assert cut.c_wrong_tile(upt) == -1, upt


@pytest.mark.parametrize("gs", [32, 64, 128])
def test_slices_of_every_width(cut, gs):
    for K in range(max(gs, 64), 4097, max(gs, 64)):
        nch, log_split, split, _ = schedule.geometry(K, gs, 4)
        assert cut.c_chunks(K) == nch and cut.c_split_log(nch) == log_split
        G, at, columns, groups = K // gs, 0, 0, 0
        for ws in range(split):
            c0 = cut.c_first_chunk(nch, log_split, ws)
            nc = cut.c_first_chunk(nch, log_split, ws + 1) - c0
            assert c0 == at == nch * ws >> log_split and 1 <= nc <= cut.c_most_chunks(nch) <= cut.c_constant(4)
            at += nc
            cols, g0, ng = cut.c_slice_columns(K, c0, nc), cut.c_slice_group(gs, c0), cut.c_slice_groups(gs, G, c0, nc)
            assert 128 * c0 == columns and gs * g0 == columns and cols == gs * ng
            columns, groups = columns + cols, groups + ng
            # table rows: loads on 16 bytes from the piece in which the slice begins,
            # reads inside what was loaded
            for r in range(16):
                start, pieces = cut.c_table_start(G, g0, r), cut.c_table_pieces(gs)
                assert start + 2 * ng <= 16 * pieces
                for b, rows in ((0, 0), (1, 16), (1, 704)):
                    want = 2 * G * (b * rows + r) + 2 * g0
                    got = cut.c_table_load(G, g0, rows, b, r, 0)
                    assert got + start == want and cut.c_table_load(G, g0, rows, b, r, 1) == got + 16
                    assert rows % 8 or got % 16 == 0
        assert at == nch and columns == K and groups == G


@pytest.mark.parametrize("T,k,E,H,I,gs,bits", schedule.CASES)
@pytest.mark.parametrize("down", [False, True])
def test_units_and_ranges(cut, T, k, E, H, I, gs, bits, down):
    rng = random.Random(T + E)
    tiles, _ = schedule.tiles_of([rng.sample(range(E), k) for _ in range(T)], E)
    upt = cut.c_units_of_tile(down, H, I)
    log_units = 3 - cut.c_split_log(cut.c_chunks(I if down else H))
    N, nu, ranges = len(tiles) * upt, 1 << log_units, cut.c_constant(1)
    assert upt == (H // 32 if down else I // 16) and N * ranges * nu < 2**30
    firsts = [cut.c_first_unit(N, s, log_units) for s in range(ranges * nu + 1)]
    assert firsts[0] == 0 and firsts[-1] == N and firsts == sorted(firsts)
    assert firsts == [N * s // (ranges * nu) for s in range(ranges * nu + 1)]
    # a range touches at most 5 tiles: it may begin and end inside one
    for r in range(ranges):
        lo, hi = firsts[r * nu], firsts[(r + 1) * nu]
        assert lo == hi or (hi - 1) // upt - lo // upt + 1 <= 5
    rows_e, magic = cut.c_expert_rows(down, H, I), cut.c_unit_magic(upt)
    rows = set()
    for e in {0, E - 1}:
        for c in range(upt):
            row, second = cut.c_unit_row(down, rows_e, e, c), cut.c_block_rows(down, I)
            assert row + second + 16 <= E * rows_e
            rows.update((e, row + b * second + i - e * rows_e) for b in range(2) for i in range(16))
    assert rows == {(e, r) for e in {0, E - 1} for r in range(rows_e)}  # every weight row once
    assert {cut.c_tile_of_unit(u, magic) for u in range(N)} == set(range(len(tiles)))


def test_a_range_can_touch_five_tiles(cut):
    """16 tokens by 64 experts in 1023 tiles: just under four tiles of units a range."""
    upt = cut.c_units_of_tile(True, 4096, 64)
    N = 1023 * upt
    most = max((cut.c_first_unit(N, 8 * (r + 1), 3) - 1) // upt - cut.c_first_unit(N, 8 * r, 3) // upt + 1 for r in range(256))
    assert most == 5


def run_order(T, tiles, slots_tile, resident, rng, ranges=20):
    """As in the schedule's replay, but a workgroup looks for another range only if it
    saw one untaken when it ended its last, as the kernel does."""
    flags = {"gu": [0] * ranges, "dn": [0] * ranges}
    units = {"gu": 5, "dn": 7}
    done = {"gu": [0] * tiles, "dn": [0] * tiles}
    outputs, looks = [0] * T, [0]

    def claim(name, r):
        won, flags[name][r] = not flags[name][r], 1
        return won

    def take(name):
        looks[0] += 1
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
        for name in ("gu", "dn"):
            yield
            own[name] = claim(name, b)
        for name in ("gu", "dn"):
            r = b if own[name] else (yield from take(name))
            while r is not None:
                if name == "dn":
                    for tile in {u // units["dn"] for u in span(name, r)}:
                        while done["gu"][tile] < units["gu"]:
                            yield "wait"
                for u in span(name, r):
                    yield
                left = not all(flags[name])  # read while the range's stores are under way
                yield
                for u in span(name, r):
                    done[name][u // units[name]] += 1
                r = (yield from take(name)) if left else None
        if b < T:
            for tile in slots_tile[b]:
                while done["dn"][tile] < units["dn"]:
                    yield "wait"
            outputs[b] += 1

    waiting, live, idle = [group(b) for b in range(ranges)], [], 0
    while waiting or live:
        while waiting and len(live) < resident:
            live.append(waiting.pop(0))
        g = rng.choice(live)
        try:
            idle = idle + 1 if next(g) == "wait" else 0
        except StopIteration:
            live.remove(g)
            idle = 0
        assert idle < 20000, "nobody makes progress"
    assert outputs == [1] * T and done["gu"] == [units["gu"]] * tiles and done["dn"] == [units["dn"]] * tiles
    return looks[0]


@pytest.mark.parametrize("resident", [1, 2, 5, 12, 20])
@pytest.mark.parametrize("T,tiles", [(1, 3), (4, 9), (16, 40)])
def test_every_wait_ends_with_the_short_way(resident, T, tiles):
    rng = random.Random(resident * 100 + T)
    slots = [[rng.randrange(tiles) for _ in range(3)] for _ in range(T)]
    looks = [run_order(T, tiles, slots, resident, rng) for _ in range(5)]
    assert resident > 1 or min(looks) > 0
