// How the layer for few tokens cuts its matmuls into units, ranges, waves and table
// rows, in plain integers: layer_few.hip uses it, and a test compiles it for the host.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>

#define MOE_CUT __host__ __device__ __forceinline__
#else
#define MOE_CUT inline
#endif

namespace moe {
namespace cut {

constexpr int kWaves = 8;          // of a workgroup
constexpr int kRangesLog = 8;      // ranges of units in each matmul: one workgroup a CU
constexpr int kRanges = 1 << kRangesLog;
constexpr int kTileRows = 8;       // rows of a tile
constexpr int kChunk = 128;        // columns of a chunk
constexpr int kMaxChunks = 4;      // of a wave's slice
constexpr int kDepth = 4;          // places for the shares of a unit's waves
constexpr int kLag = 2;            // units after which a unit's outputs are made

// 16-byte pieces of a wave's table row, for a slice of at most kMaxChunks chunks and from
// the piece on in which the slice begins.
constexpr int table_pieces(int gs) { return kMaxChunks * kChunk / gs <= 8 ? 2 : 4; }

// Chunks of a row of K columns.
MOE_CUT int chunks(int K) { return (K + kChunk - 1) / kChunk; }
// A row of nch chunks is cut over 1 << split_log waves, kMaxChunks chunks to a wave at most.
// Measured at rows of 6 and 22 chunks (widths 704, 768 and 2816), which get 3 chunks a
// wave, against 2; rows of 4, 7, 8 and 13 to 16 chunks get 2, where 4 on half the waves
// would fit too and has not been measured.
MOE_CUT int split_log(int nch) { return nch <= 3 ? 0 : nch <= 6 ? 1 : nch <= 12 ? 2 : 3; }
// The first chunk of wave ws of those waves (ws may be their number).
MOE_CUT int first_chunk(int nch, int log, int ws) { return nch * ws >> log; }
// Most chunks that one of them takes.
MOE_CUT int most_chunks(int nch) { return (nch + (1 << split_log(nch)) - 1) >> split_log(nch); }
// Columns of a slice of nc chunks from chunk ch0 on, and its first group and groups.
MOE_CUT int slice_columns(int K, int ch0, int nc) { return nc * kChunk < K - kChunk * ch0 ? nc * kChunk : K - kChunk * ch0; }
MOE_CUT int slice_group(int gs, int ch0) { return ch0 * kChunk / gs; }
MOE_CUT int slice_groups(int gs, int G, int ch0, int nc) {
    const int n = nc * kChunk / gs, left = G - slice_group(gs, ch0);
    return n < left ? n : left;
}

// A unit is 32 weight rows by all of K: down: 32 output columns; gate|up: 16 columns of
// h, both halves.
MOE_CUT int units_of_tile(bool down, int H, int I) { return down ? H / 32 : I / 16; }
// N units are cut into kRanges << log_units shares, a range's at work at a time in
// 1 << log_units of them: the first unit of a share (N share < 2^30).
MOE_CUT int first_unit(int N, int share, int log_units) { return N * share >> (kRangesLog + log_units); }

// u / upt for u < 2^18, upt <= 256, by m = ceil(2^31 / upt): u (m upt - 2^31) < 2^26, so
// the quotient errs by less than 1 / upt.
MOE_CUT uint32_t unit_magic(uint32_t upt) { return ((1u << 31) + upt - 1) / upt; }
MOE_CUT int tile_of_unit(int u, uint32_t magic) {
    return static_cast<int>(static_cast<uint64_t>(2u * static_cast<uint32_t>(u)) * magic >> 32);
}

// Weight rows of an expert; the first row of its unit col, and from the first to the
// second block of 16 rows of a unit.
MOE_CUT int expert_rows(bool down, int H, int I) { return down ? H : 2 * I; }
MOE_CUT uint32_t unit_row(bool down, int rows_e, int expert, int col) { return expert * rows_e + (down ? 32 : 16) * col; }
MOE_CUT int block_rows(bool down, int I) { return down ? 16 : I; }

// Tables of G entries a row: the byte, from the unit's first row on, at which a lane
// loads its first 16 bytes of row r of block b, the slice beginning with group g0 ...
MOE_CUT uint32_t table_load(int G, int g0, int rows, int b, int r, int piece) {
    return (2u * (r * G + g0) & ~15u) + 2u * G * rows * b + 16 * piece;
}
// ... and the byte of its row in LDS at which the slice begins.
MOE_CUT int table_start(int G, int g0, int r) { return 2 * (r * G + g0) & 15; }

}  // namespace cut
}  // namespace moe
