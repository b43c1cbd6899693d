// The gradient of the experts' weights:  dw[e, n, k] = sum over the rows r of expert e of
// dy[r, n] x[r, k].
//
// The sum runs along the rows, across both operands' memory: stages of 64 rows come to LDS
// as they lie and the reads turn them.  One workgroup a CU takes its tiles in turn; four of
// its waves only copy, D - 1 stages ahead, and eight multiply and store.  So nothing waits
// at a tile's end: a wave's memory operations end in order, and with copies and stores in one
// wave the next stage would wait for the last tile's stores.
//
// Bound by writing dw: 16384 rows of 128 experts by 1408 x 2816 take 286 us for 1.15 GB, of it
// 1.0 GB of dw.  The stores alone take 184 us, copies and products without stores 167 us; they
// overlap in part, since the copies' answers come late while the memory is busy with writes (with
// every expert reading the same rows, from L2, 249 us).
//
// Tiles are dealt by their number, an eighth of them to an XCD, and not by their rows: with few experts, or one that
// has most rows, the XCD with the longest experts ends last.  Rows even | as mild routing spreads them | as 1 / rank:
// the case above 248 | 286 | 551 us; 16381 rows of 8 experts by 2816 x 4096 363 | 466 | 893 us (an XCD an expert).
#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

// A workgroup takes chunks: neighbouring blocks of columns of dy against one block of x's.  Of an
// expert of up to D stages the block of x stays in LDS for the whole chunk.
struct DwTiles {
    uint32_t n, k;     // blocks of columns of dy and of x
    uint32_t chunks;   // of the n blocks
    uint32_t splits;   // runs of an expert's rows
    uint32_t count;    // of all chunks
};

template <int BN, int BK, int WN, int WK, int D, bool kF32>
__global__ __launch_bounds__(64 * (WN * WK + 4)) void moe_grouped_dw_tile(GroupedGradArgs a, DwTiles tiles) {
    constexpr int kWaves = WN * WK, kLoaders = 4, FN = BN / WN / 16, FK = BK / WK / 16, kStage = 64;
    constexpr int kYJobs = BN / 8 / kLoaders, kXJobs = BK / 8 / kLoaders, kJobs = kYJobs + kXJobs;
    static_assert(kYJobs * 8 * kLoaders == BN && kXJobs * 8 * kLoaders == BK && FK % 2 == 0, "tile");
    __shared__ __align__(16) unsigned char ybuf[D][BN * 128], xbuf[D][BK * 128];
    __shared__ __align__(16) unsigned char turn[kWaves][16 * 128];  // results on their way out
    // Tiles are dealt out within each XCD's run of neighbours (workgroups go to the XCDs in
    // turn): those at work at a time read the same rows.
    const uint32_t share = (tiles.count + 7) / 8, first = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    const uint32_t end = min((blockIdx.x & 7) * share + share, tiles.count), step_by = gridDim.x >> 3;
    if (first >= end) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    struct Chunk {
        int expert, split, n, n_end, k0, row, rows;  // blocks [n, n_end) of dy; rows [row, row + rows) of dy and x
        int stages;
    };
    auto find = [&](uint32_t number) {
        const uint32_t whole = number / tiles.splits, of_expert = tiles.chunks * tiles.k;
        Chunk t;
        t.split = __builtin_amdgcn_readfirstlane(static_cast<int>(number - whole * tiles.splits));
        t.expert = __builtin_amdgcn_readfirstlane(static_cast<int>(whole / of_expert));
        const uint32_t rest = whole - t.expert * of_expert, kb = rest / tiles.chunks, chunk = rest - kb * tiles.chunks;
        t.k0 = __builtin_amdgcn_readfirstlane(static_cast<int>(kb * BK));
        t.n = __builtin_amdgcn_readfirstlane(static_cast<int>(chunk * tiles.n / tiles.chunks));
        t.n_end = __builtin_amdgcn_readfirstlane(static_cast<int>((chunk + 1) * tiles.n / tiles.chunks));
        int lo = 0, hi = a.A;
        if (a.offsets) {  // through the scalar cache: a vector load would wait for the copies before it
            const auto* const o = (const __attribute__((address_space(4))) int32_t*)a.offsets;
            lo = min(max(o[t.expert], 0), a.A);
            hi = min(max(o[t.expert + 1], lo), a.A);
        }
        if (tiles.splits > 1) {  // whole stages
            const int64_t all = (hi - lo + kStage - 1) / kStage;
            const int from = lo + kStage * static_cast<int>(all * t.split / static_cast<int>(tiles.splits));
            hi = min(hi, lo + kStage * static_cast<int>(all * (t.split + 1) / static_cast<int>(tiles.splits)));
            lo = min(from, hi);
        }
        t.row = __builtin_amdgcn_readfirstlane(lo);
        t.rows = __builtin_amdgcn_readfirstlane(hi - lo);
        t.stages = max((t.rows + kStage - 1) / kStage, 1);  // without rows one of zeros
        return t;
    };

    // A stage is a step: the copiers wait for its copies, then all waves meet, then the
    // copiers start the stage D - 1 steps ahead, in the buffer of the last step.
    if (wave >= kWaves) {
        const int w = wave - kWaves;
        uint32_t ahead = first, steps = 0;  // steps: those whose copies are under way
        Chunk t = find(ahead);
        int stage = 0, buffer = 0, x_slot = 0;
        bool new_x = true, last_x = true;  // whether the stage at hand, and the last issued, copy x
        uint32_t yat[kYJobs], xat[kXJobs];
        int yrow[kYJobs], xrow[kXJobs];
        auto aim = [&] {
            const int ycols = min(BN, a.N - BN * t.n), xcols = min(BK, a.K - t.k0);
#pragma unroll
            for (int j = 0; j < kYJobs; ++j) {
                constexpr int kPieces = BN / 8;
                yrow[j] = 64 / kPieces * (j * kLoaders + w) + lane / kPieces;
                const int p = lane % kPieces, col = 32 * ((p >> 1) ^ turn_key(yrow[j])) + 16 * (p & 1);
                yat[j] = col < 2 * ycols ? static_cast<uint32_t>(yrow[j]) * static_cast<uint32_t>(a.dy_stride) + col : kOutside;
            }
#pragma unroll
            for (int j = 0; j < kXJobs; ++j) {
                constexpr int kPieces = BK / 8;
                xrow[j] = 64 / kPieces * (j * kLoaders + w) + lane / kPieces;
                const int p = lane % kPieces, col = 32 * ((p >> 1) ^ turn_key(xrow[j])) + 16 * (p & 1);
                xat[j] = col < 2 * xcols ? static_cast<uint32_t>(xrow[j]) * static_cast<uint32_t>(a.x_stride) + col : kOutside;
            }
        };
        auto issue = [&] {
            // rows past the expert's last read zeros
            const int from = t.row + kStage * stage, rows = min(kStage, t.rows - kStage * stage);
            const int ycols = min(BN, a.N - BN * t.n);
            const Rsrc ry = make_rsrc(static_cast<const unsigned char*>(a.dy) + from * a.dy_stride + 2 * static_cast<int64_t>(BN * t.n),
                                      static_cast<uint32_t>(max(rows - 1, 0) * a.dy_stride) + 2 * ycols);
#pragma unroll
            for (int j = 0; j < kYJobs; ++j)
                copy16(ry, ybuf[buffer] + 1024 * (j * kLoaders + w), yrow[j] < rows ? yat[j] : kOutside, 0);
            if (new_x) {
                const int xcols = min(BK, a.K - t.k0);
                const Rsrc rx = make_rsrc(static_cast<const unsigned char*>(a.x) + from * a.x_stride + 2 * static_cast<int64_t>(t.k0),
                                          static_cast<uint32_t>(max(rows - 1, 0) * a.x_stride) + 2 * xcols);
#pragma unroll
                for (int j = 0; j < kXJobs; ++j)
                    copy16(rx, xbuf[x_slot] + 1024 * (j * kLoaders + w), xrow[j] < rows ? xat[j] : kOutside, 0);
                x_slot = x_slot + 1 == D ? 0 : x_slot + 1;
            }
            last_x = new_x;
            buffer = buffer + 1 == D ? 0 : buffer + 1;
            ++steps;
            if (++stage == t.stages) {
                stage = 0;
                if (++t.n < t.n_end) {
                    new_x = t.stages > D;
                    aim();
                } else {
                    ahead += step_by;
                    new_x = true;
                    if (ahead < end) {
                        t = find(ahead);
                        aim();
                    }
                }
            }
        };
        aim();
        for (int i = 0; i < D - 1 && ahead < end; ++i) issue();
        for (uint32_t at = 0; at < steps; ++at) {
            // all but the last stage's
            if (ahead >= end)
                wait_copies<0>();
            else if (last_x)
                wait_copies<(D - 2) * kJobs>();
            else
                wait_copies<(D - 2) * kYJobs>();
            step_barrier();
            if (ahead < end) issue();
        }
        return;
    }

    const int lr = lane & 15, q = lane >> 4, wk = wave / WN, wn = wave % WN;
    f32x4 acc[FN][FK];
    const int r = 8 * q + (lr >> 2);
    int yturn[FN], xturn[FK];
#pragma unroll
    for (int n = 0; n < FN; ++n) yturn[n] = r * 2 * BN + 32 * ((wn * FN + n) ^ turn_key(r)) + 8 * (lr & 3);
#pragma unroll
    for (int k = 0; k < FK; ++k) xturn[k] = r * 2 * BK + 32 * ((wk * FK + k) ^ turn_key(r)) + 8 * (lr & 3);
    int buffer = 0, x_base = 0;  // the slot of x's first stage
    uint32_t here = first;
    for (Chunk t = find(here);;) {
        const int n0 = BN * t.n, ycols = min(BN, a.N - n0), xcols = min(BK, a.K - t.k0);
        // whether this wave's part of the tile holds anything
        const bool active = 16 * wn * FN < ycols && 16 * wk * FK < xcols;
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int k = 0; k < FK; ++k) acc[n][k] = f32x4{0.f, 0.f, 0.f, 0.f};
        int x_now = x_base;
        for (int stage = 0; stage < t.stages; ++stage) {
            step_barrier();
            const unsigned char *const ys = ybuf[buffer], *const xs = xbuf[x_now];
            buffer = buffer + 1 == D ? 0 : buffer + 1;
            x_now = x_now + 1 == D ? 0 : x_now + 1;
            if (!active) continue;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 yf[FN], xf[FK];
#pragma unroll
                for (int n = 0; n < FN; ++n) {
                    const u32x2 lo = read_turned(ys, yturn[n] + 64 * s * BN), hi = read_turned(ys, yturn[n] + 64 * s * BN + 8 * BN);
                    yf[n] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
#pragma unroll
                for (int k = 0; k < FK; ++k) {
                    const u32x2 lo = read_turned(xs, xturn[k] + 64 * s * BK), hi = read_turned(xs, xturn[k] + 64 * s * BK + 8 * BK);
                    xf[k] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
#pragma unroll
                for (int n = 0; n < FN; ++n)
#pragma unroll
                    for (int k = 0; k < FK; ++k) acc[n][k] = mfma_bf16(xf[k], yf[n], acc[n][k]);
            }
        }
        // A product's lanes hold 16 rows of n; memory wants rows of 128 bytes.  So 16 rows of
        // 128 bytes at a time go through LDS, pieces of 16 bytes XORed with the row (a wave's
        // own: no barrier).  Storing the products as they lie, 64 bytes of 16 rows an
        // instruction, measured 380 | 343 us at 16384 rows of 128 experts by 1408 x 2816.
        constexpr int kOut = kF32 ? 4 : 2, kBlock = 128 / (16 * kOut);  // products in 128 bytes
        unsigned char* const out = static_cast<unsigned char*>(a.dw) +
                                   kOut * (((static_cast<int64_t>(t.split) * a.E + t.expert) * a.N + n0) * a.K + t.k0);
        const uint32_t pitch = static_cast<uint32_t>(kOut * a.K);
        const Rsrc ro = make_rsrc(out, (ycols - 1) * pitch + kOut * xcols);
        unsigned char* const mine = turn[wave];
#pragma unroll
        for (int n = 0; n < FN; ++n) {
#pragma unroll
            for (int k = 0; k < FK; k += kBlock) {
#pragma unroll
                for (int i = 0; i < kBlock; i += kF32 ? 1 : 2) {
                    u32x4 v;
                    int piece;
                    if constexpr (kF32) {
                        v = __builtin_bit_cast(u32x4, acc[n][k + i]);
                        piece = 4 * i + q;
                    } else {
                        v = eight_bf16(acc[n][k + i], acc[n][k + i + 1]);
                        piece = 2 * (i + (q & 1)) + (q >> 1);
                    }
                    *reinterpret_cast<u32x4*>(mine + 128 * lr + 16 * (piece ^ (lr & 7))) = v;
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = 8 * half + (lane >> 3), p = lane & 7;
                    const u32x4 v = read16(mine, 128 * r + 16 * (p ^ (r & 7)));
                    const int row = 16 * (wn * FN + n) + r, col = 16 * (wk * FK + k) + p * (16 / kOut);
                    store16(ro, v, row < ycols && col < xcols ? static_cast<uint32_t>(row) * pitch + kOut * col : kOutside);
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        // the next tile reads the same x where it stayed, else the slots that come next
        const bool same = ++t.n < t.n_end;
        if (!same || t.stages > D) x_base = x_now;
        if (same) continue;
        here += step_by;
        if (here >= end) break;
        t = find(here);
    }
}

// Sums of the splits, in their order; four values a thread.
template <bool kF32>
__global__ __launch_bounds__(256) void moe_grouped_dw_join(const float* parts, int64_t size, int splits, void* out) {
    const int64_t i = 4 * (static_cast<int64_t>(grid_index()) * 256 + threadIdx.x);
    if (i >= size) return;  // a multiple of 64
    f32x4 v = *reinterpret_cast<const f32x4*>(parts + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(parts + s * size + i);
    if constexpr (kF32)
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = v;
    else
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

constexpr int kTileN = 128, kTileK = 256;

// Into how many runs the rows of an expert are cut: where the tiles alone do not give
// every CU one and there are rows enough for four stages a run.
int splits_of(int32_t A, int32_t E, int32_t N, int32_t K) {
    const int64_t tiles = static_cast<int64_t>(E) * ((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
    const int64_t most = static_cast<int64_t>(A) / E / 256, want = 256 / tiles;
    return static_cast<int>(want < 2 || most < 2 ? 1 : want < most ? want : most);
}

}  // namespace

size_t grouped_dw_workspace(int32_t A, int32_t E, int32_t N, int32_t K) {
    const int splits = splits_of(A, E, N, K);
    return splits > 1 ? static_cast<size_t>(splits) * E * N * K * sizeof(float) : 0;
}

hipError_t launch_grouped_dw(const GroupedGradArgs& a, hipStream_t s) {
    DwTiles t;
    t.n = (a.N + kTileN - 1) / kTileN;
    t.k = (a.K + kTileK - 1) / kTileK;
    t.splits = splits_of(a.A, a.E, a.N, a.K);
    // Chunks of up to three blocks where every CU gets eight, else single ones.  1 | 2 | 3 | 4 blocks, us: 16384 rows of 128
    // experts by 1408 x 2816 348 | 295 | 288 | 316 (6: 298), by 2048 x 2048 369 | 321 | 288 | 325, by 2816 x 1408 333 |
    // 315 | 296 | 320; of 64 by 2816 x 4096 635 | 621 | 588 | 586; of 256 by 1024 x 2048 304 | 259 | 221 | 243; 4096 rows of
    // 128 by 1408 x 2816 207 | 212 | 215 | 196.
    t.chunks = static_cast<int64_t>(t.n) * t.k * a.E >= 256 * 8 * 3 ? (t.n + 2) / 3 : t.n;
    t.count = t.chunks * t.k * a.E * t.splits;
    const dim3 grid(t.count < 256 ? (t.count + 7) / 8 * 8 : 256), block(64 * 12);
    GroupedGradArgs to = a;
    if (t.splits > 1) to.dw = a.ws;
    if (t.splits > 1 || a.out_f32)
        hipLaunchKernelGGL((moe_grouped_dw_tile<kTileN, kTileK, 2, 4, 3, true>), grid, block, 0, s, to, t);
    else
        hipLaunchKernelGGL((moe_grouped_dw_tile<kTileN, kTileK, 2, 4, 3, false>), grid, block, 0, s, to, t);
    if (t.splits > 1) {
        const int64_t size = static_cast<int64_t>(a.E) * a.N * a.K;
        const dim3 join = grid_of((size / 4 + 255) / 256);
        if (a.out_f32)
            hipLaunchKernelGGL((moe_grouped_dw_join<true>), join, dim3(256), 0, s, a.ws, size, static_cast<int>(t.splits), a.dw);
        else
            hipLaunchKernelGGL((moe_grouped_dw_join<false>), join, dim3(256), 0, s, a.ws, size, static_cast<int>(t.splits), a.dw);
    }
    return hipGetLastError();
}

}  // namespace moe
