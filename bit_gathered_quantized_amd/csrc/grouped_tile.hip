// Grouped products of bf16 rows and bf16 weights in tiles of BM rows by BN columns.
#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

// A stage is 128 bytes (64 elements) of K.  Operands with K along their rows lie in LDS
// as rows of 128 bytes whose 16-byte pieces are XORed with the row's number, so that
// neither the copies nor the reads meet a bank twice; w [E, K, N] lies as 64 rows of BN
// columns in pieces of 32 bytes XORed the same way, and is turned by the reads.
template <int BM, int BN, int WM, int WN, bool kKN, bool kF32>
__global__ __launch_bounds__(64 * WM * WN) void moe_grouped_tile(GroupedArgs a, uint32_t most, uint32_t across) {
    constexpr int kWaves = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int kXJobs = BM / 8 / kWaves, kWJobs = BN / 8 / kWaves;
    static_assert(kXJobs * 8 * kWaves == BM && kWJobs * 8 * kWaves == BN && FN % 2 == 0, "tile");
    __shared__ __align__(16) unsigned char x0[BM * 128], x1[BM * 128], w0[BN * 128], w1[BN * 128];
    Tile t;
    if (!find_tile<BM, 8>(a.offsets, a.A, a.E, most, across, grid_index(), t)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int n0 = t.n * BN, cols = min(BN, a.N - n0);
    const uint32_t kbytes = 2u * a.K;

    // x: rows past the tile's last repeat it (their results are not stored)
    const unsigned char* const px = static_cast<const unsigned char*>(a.x) + t.row * a.x_stride;
    const Rsrc rx = make_rsrc(px, static_cast<uint32_t>((t.rows - 1) * a.x_stride) + kbytes);
    const uint32_t piece = 16u * ((lane & 7) ^ (lane >> 3));
    uint32_t xat[kXJobs], wat[kWJobs];
#pragma unroll
    for (int j = 0; j < kXJobs; ++j)
        xat[j] = static_cast<uint32_t>(min(8 * (j * kWaves + wave) + (lane >> 3), t.rows - 1)) * static_cast<uint32_t>(a.x_stride) + piece;
    const unsigned char* pw = static_cast<const unsigned char*>(a.w) + t.expert * a.w_expert;
    uint32_t wsize;
    int wrow[kWJobs];  // w [E, K, N]: the row of a stage
    if constexpr (kKN) {
        pw += 2 * n0;
        wsize = static_cast<uint32_t>(2 * cols);
#pragma unroll
        for (int j = 0; j < kWJobs; ++j) {
            constexpr int kPieces = BN / 8, kRowsJob = 64 / kPieces;
            wrow[j] = kRowsJob * (j * kWaves + wave) + lane / kPieces;
            const int p = lane % kPieces, col = 32 * ((p >> 1) ^ (wrow[j] & 7)) + 16 * (p & 1);
            wat[j] = col < 2 * cols ? static_cast<uint32_t>(wrow[j]) * static_cast<uint32_t>(a.w_stride) + col : kOutside;
        }
    } else {
        // LDS row 16 f + i holds column 32 (f / 2) + 8 (i / 4) + 4 (f % 2) + i % 4, so
        // that a lane ends up with 8 neighbouring columns of two products
        pw += n0 * a.w_stride;
        wsize = static_cast<uint32_t>((cols - 1) * a.w_stride) + kbytes;
#pragma unroll
        for (int j = 0; j < kWJobs; ++j) {
            const int r = 8 * (j * kWaves + wave) + (lane >> 3), f = r >> 4, i = r & 15;
            const int n = 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
            wat[j] = static_cast<uint32_t>(min(n, cols - 1)) * static_cast<uint32_t>(a.w_stride) + piece;
        }
    }
    const int stages = (a.K + 63) / 64;
    auto issue = [&](unsigned char* xs, unsigned char* ws, int s) {
        const uint32_t k = 128u * s;
        const bool inside = k + piece < kbytes;
#pragma unroll
        for (int j = 0; j < kXJobs; ++j)
            copy16(rx, xs + 1024 * (j * kWaves + wave), inside ? xat[j] : kOutside, k);
        if constexpr (kKN) {
            // the rows of a stage, at most 64: a resource of its own, as K rows may pass 32 bits
            const int rows = min(64, a.K - 64 * s);
            const Rsrc rw = make_rsrc(pw + 64 * s * a.w_stride, static_cast<uint32_t>((rows - 1) * a.w_stride) + wsize);
#pragma unroll
            for (int j = 0; j < kWJobs; ++j)
                copy16(rw, ws + 1024 * (j * kWaves + wave), wrow[j] < rows ? wat[j] : kOutside, 0);
        } else {
            const Rsrc rw = make_rsrc(pw, wsize);
#pragma unroll
            for (int j = 0; j < kWJobs; ++j)
                copy16(rw, ws + 1024 * (j * kWaves + wave), inside ? wat[j] : kOutside, k);
        }
    };
    f32x4 acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    int turned[kKN ? FN : 1];  // of columns 16 f of row 8 q + (lane & 15) / 4
    if constexpr (kKN) {
        const int r = 8 * q + (lr >> 2);
#pragma unroll
        for (int f = 0; f < FN; ++f) turned[f] = r * 2 * BN + 32 * ((wn * FN + f) ^ (r & 7)) + 8 * (lr & 3);
    }
    auto compute = [&](const unsigned char* xs, const unsigned char* ws) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = 128 * lr + 16 * ((4 * s + q) ^ (lr & 7));
            u32x4 wf[FN], xf[FM];
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if constexpr (kKN) {
                    // rows + 4: the XOR turns over bit 2, as that of f ^ 4 does
                    const u32x2 lo = read_turned(ws, turned[f] + 64 * s * BN);
                    const u32x2 hi = read_turned(ws, (turned[f] ^ 128) + 64 * s * BN + 8 * BN);
                    wf[f] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                } else {
                    wf[f] = read16(ws, at + 2048 * (wn * FN + f));
                }
            }
#pragma unroll
            for (int m = 0; m < FM; ++m) xf[m] = read16(xs, at + 2048 * (wm * FM + m));
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int m = 0; m < FM; ++m) acc[f][m] = mfma_bf16(wf[f], xf[m], acc[f][m]);
        }
    };
    issue(x0, w0, 0);
    copies_done<0>();
    for (int s = 0; s < stages; s += 2) {
        if (s + 1 < stages) issue(x1, w1, s + 1);
        compute(x0, w0);
        copies_done<0>();
        if (s + 1 >= stages) break;
        if (s + 2 < stages) issue(x0, w0, s + 2);
        compute(x1, w1);
        copies_done<0>();
    }
    // lane (lr, q) of a product holds columns 4 q .. 4 q + 3 of row lr
    constexpr int kOut = kF32 ? 4 : 2;
    unsigned char* const out = static_cast<unsigned char*>(a.out) + t.row * a.out_stride + static_cast<int64_t>(kOut) * n0;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
        const int row = 16 * (wm * FM + m) + lr;
        if (row >= t.rows) continue;
        unsigned char* const o = out + row * a.out_stride;
#pragma unroll
        for (int f = 0; f < FN; f += 2) {
            const f32x4 v = acc[f][m], u = acc[f + 1][m];
            const int c = 16 * (wn * FN + f);
            if constexpr (kKN) {
                const int col = c + 4 * q;
                if constexpr (kF32) {
                    if (col < cols) *reinterpret_cast<f32x4*>(o + 4 * col) = v;
                    if (col + 16 < cols) *reinterpret_cast<f32x4*>(o + 4 * col + 64) = u;
                } else {
                    if (col < cols) *reinterpret_cast<u32x2*>(o + 2 * col) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    if (col + 16 < cols)
                        *reinterpret_cast<u32x2*>(o + 2 * col + 32) = u32x2{pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
                }
            } else {
                const int col = c + 8 * q;
                if (col >= cols) continue;
                if constexpr (kF32) {
                    *reinterpret_cast<f32x4*>(o + 4 * col) = v;
                    *reinterpret_cast<f32x4*>(o + 4 * col + 16) = u;
                } else {
                    *reinterpret_cast<u32x4*>(o + 2 * col) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                  pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
                }
            }
        }
    }
}

template <int BM, int BN, int WM, int WN>
void launch(const GroupedArgs& a, hipStream_t s) {
    const uint32_t most = static_cast<uint32_t>(grid_tiles(a, BM)), across = (a.N + BN - 1) / BN;
    // a multiple of 8: the XCDs' shares are rounded up
    const dim3 grid = grid_of((static_cast<int64_t>(most) * across + 7) / 8 * 8), block(64 * WM * WN);
    if (a.w_kn) {
        if (a.out_f32)
            hipLaunchKernelGGL((moe_grouped_tile<BM, BN, WM, WN, true, true>), grid, block, 0, s, a, most, across);
        else
            hipLaunchKernelGGL((moe_grouped_tile<BM, BN, WM, WN, true, false>), grid, block, 0, s, a, most, across);
    } else {
        if (a.out_f32)
            hipLaunchKernelGGL((moe_grouped_tile<BM, BN, WM, WN, false, true>), grid, block, 0, s, a, most, across);
        else
            hipLaunchKernelGGL((moe_grouped_tile<BM, BN, WM, WN, false, false>), grid, block, 0, s, a, most, across);
    }
}

}  // namespace

hipError_t launch_grouped_bf16(const GroupedArgs& a, hipStream_t s) {
    launch<128, 128, 2, 2>(a, s);
    return hipGetLastError();
}

}  // namespace moe
