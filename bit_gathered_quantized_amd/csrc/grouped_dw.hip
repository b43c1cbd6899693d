// The gradient of the experts' weights:  dw[e, n, k] = sum over the rows r of expert e of
// dy[r, n] x[r, k].
//
// The sum runs along the rows, across both operands' memory: tiles of 64 rows come to LDS
// as they lie and the reads turn them.
#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

// Pieces of 32 bytes of row r (mod 64) are XORed with r, for the turning reads: four rows
// at a time.
template <int BN, int BK, int WN, int WK, bool kF32>
__global__ __launch_bounds__(64 * WN * WK) void moe_grouped_dw_tile(GroupedGradArgs a, uint32_t tiles_n, uint32_t tiles_k,
                                                                   uint32_t splits) {
    constexpr int kWaves = WN * WK, FN = BN / WN / 16, FK = BK / WK / 16;
    constexpr int kYJobs = BN / 8 / kWaves, kXJobs = BK / 8 / kWaves;
    static_assert(kYJobs * 8 * kWaves == BN && kXJobs * 8 * kWaves == BK, "tile");
    __shared__ __align__(16) unsigned char y0[BN * 128], y1[BN * 128], x0[BK * 128], x1[BK * 128];
    const uint32_t index = grid_index();
    // a run of neighbouring tiles for each XCD: those of an expert read the same rows
    const uint32_t tiles = tiles_n * tiles_k * a.E * splits, share = (tiles + 7) / 8;
    const uint32_t number = (index & 7) * share + (index >> 3);
    if ((index >> 3) >= share || number >= tiles) return;
    const uint32_t of_expert = tiles_n * tiles_k, whole = number / splits, split = number - whole * splits;
    const int expert = whole / of_expert;
    const uint32_t rest = whole - expert * of_expert;
    const int k0 = (rest / tiles_n) * BK, n0 = (rest % tiles_n) * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4, wk = wave / WN, wn = wave % WN;
    int begin = 0, end = a.A;
    if (a.offsets) expert_rows(a.offsets, expert, a.E, a.A, begin, end);
    const int stages_all = (end - begin + 63) / 64;
    const int s0 = static_cast<int>(static_cast<int64_t>(stages_all) * split / splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(stages_all) * (split + 1) / splits);
    const int ycols = min(BN, a.N - n0), xcols = min(BK, a.K - k0);

    uint32_t yat[kYJobs], xat[kXJobs];
    int yrow[kYJobs], xrow[kXJobs];
#pragma unroll
    for (int j = 0; j < kYJobs; ++j) {
        constexpr int kPieces = BN / 8;
        yrow[j] = 64 / kPieces * (j * kWaves + wave) + lane / kPieces;
        const int p = lane % kPieces, col = 32 * ((p >> 1) ^ (yrow[j] & 7)) + 16 * (p & 1);
        yat[j] = col < 2 * ycols ? static_cast<uint32_t>(yrow[j]) * static_cast<uint32_t>(a.dy_stride) + col : kOutside;
    }
#pragma unroll
    for (int j = 0; j < kXJobs; ++j) {
        constexpr int kPieces = BK / 8;
        xrow[j] = 64 / kPieces * (j * kWaves + wave) + lane / kPieces;
        const int p = lane % kPieces, col = 32 * ((p >> 1) ^ (xrow[j] & 7)) + 16 * (p & 1);
        xat[j] = col < 2 * xcols ? static_cast<uint32_t>(xrow[j]) * static_cast<uint32_t>(a.x_stride) + col : kOutside;
    }
    auto issue = [&](unsigned char* ys, unsigned char* xs, int s) {
        const int first = begin + 64 * s, rows = min(64, end - first);
        const Rsrc ry = make_rsrc(static_cast<const unsigned char*>(a.dy) + first * a.dy_stride + 2 * static_cast<int64_t>(n0),
                                  static_cast<uint32_t>((rows - 1) * a.dy_stride) + 2 * ycols);
        const Rsrc rx = make_rsrc(static_cast<const unsigned char*>(a.x) + first * a.x_stride + 2 * static_cast<int64_t>(k0),
                                  static_cast<uint32_t>((rows - 1) * a.x_stride) + 2 * xcols);
        // rows past the expert's last read zeros
#pragma unroll
        for (int j = 0; j < kYJobs; ++j) copy16(ry, ys + 1024 * (j * kWaves + wave), yrow[j] < rows ? yat[j] : kOutside, 0);
#pragma unroll
        for (int j = 0; j < kXJobs; ++j) copy16(rx, xs + 1024 * (j * kWaves + wave), xrow[j] < rows ? xat[j] : kOutside, 0);
    };
    f32x4 acc[FN][FK];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int k = 0; k < FK; ++k) acc[n][k] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int r = 8 * q + (lr >> 2);
    int yturn[FN], xturn[FK];
#pragma unroll
    for (int n = 0; n < FN; ++n) yturn[n] = r * 2 * BN + 32 * ((wn * FN + n) ^ (r & 7)) + 8 * (lr & 3);
#pragma unroll
    for (int k = 0; k < FK; ++k) xturn[k] = r * 2 * BK + 32 * ((wk * FK + k) ^ (r & 7)) + 8 * (lr & 3);
    auto compute = [&](const unsigned char* ys, const unsigned char* xs) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 yf[FN], xf[FK];
            // rows + 4: the XOR turns over bit 2, as that of the piece's number with 4 does
#pragma unroll
            for (int n = 0; n < FN; ++n) {
                const u32x2 lo = read_turned(ys, yturn[n] + 64 * s * BN), hi = read_turned(ys, (yturn[n] ^ 128) + 64 * s * BN + 8 * BN);
                yf[n] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int k = 0; k < FK; ++k) {
                const u32x2 lo = read_turned(xs, xturn[k] + 64 * s * BK), hi = read_turned(xs, (xturn[k] ^ 128) + 64 * s * BK + 8 * BK);
                xf[k] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int k = 0; k < FK; ++k) acc[n][k] = mfma_bf16(xf[k], yf[n], acc[n][k]);
        }
    };
    if (s0 < s1) {
        issue(y0, x0, s0);
        copies_done<0>();
        for (int s = s0; s < s1; s += 2) {
            if (s + 1 < s1) issue(y1, x1, s + 1);
            compute(y0, x0);
            copies_done<0>();
            if (s + 1 >= s1) break;
            if (s + 2 < s1) issue(y0, x0, s + 2);
            compute(y1, x1);
            copies_done<0>();
        }
    }
    // lane (lr, q) of a product holds columns 4 q .. 4 q + 3 of k and row lr of n
    constexpr int kOut = kF32 ? 4 : 2;
    unsigned char* const out = static_cast<unsigned char*>(a.dw) +
                               kOut * (((static_cast<int64_t>(split) * a.E + expert) * a.N + n0) * a.K + k0);
#pragma unroll
    for (int n = 0; n < FN; ++n) {
        const int row = 16 * (wn * FN + n) + lr;
        if (row >= ycols) continue;
#pragma unroll
        for (int k = 0; k < FK; ++k) {
            const int col = 16 * (wk * FK + k) + 4 * q;
            if (col >= xcols) continue;
            const f32x4 v = acc[n][k];
            unsigned char* const o = out + kOut * (static_cast<int64_t>(row) * a.K + col);
            if constexpr (kF32)
                *reinterpret_cast<f32x4*>(o) = v;
            else
                *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
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

constexpr int kTile = 128;

// Into how many runs the rows of an expert are cut: where the tiles alone do not give
// every CU two workgroups and there are rows enough for four stages a run.
int splits_of(int32_t A, int32_t E, int32_t N, int32_t K) {
    const int64_t tiles = static_cast<int64_t>(E) * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
    const int64_t most = static_cast<int64_t>(A) / E / 256, want = (512 + tiles - 1) / tiles;
    return static_cast<int>(tiles >= 256 || most < 2 ? 1 : want < most ? want : most);
}

}  // namespace

size_t grouped_dw_workspace(int32_t A, int32_t E, int32_t N, int32_t K) {
    const int splits = splits_of(A, E, N, K);
    return splits > 1 ? static_cast<size_t>(splits) * E * N * K * sizeof(float) : 0;
}

hipError_t launch_grouped_dw(const GroupedGradArgs& a, hipStream_t s) {
    const uint32_t tn = (a.N + kTile - 1) / kTile, tk = (a.K + kTile - 1) / kTile;
    const int splits = splits_of(a.A, a.E, a.N, a.K);
    const int64_t tiles = static_cast<int64_t>(tn) * tk * a.E * splits;
    const dim3 grid = grid_of((tiles + 7) / 8 * 8), block(256);  // a multiple of 8: the XCDs' shares are rounded up
    GroupedGradArgs to = a;
    if (splits > 1) to.dw = a.ws;
    if (splits > 1 || a.out_f32)
        hipLaunchKernelGGL((moe_grouped_dw_tile<kTile, kTile, 2, 2, true>), grid, block, 0, s, to, tn, tk, splits);
    else
        hipLaunchKernelGGL((moe_grouped_dw_tile<kTile, kTile, 2, 2, false>), grid, block, 0, s, to, tn, tk, splits);
    if (splits > 1) {
        const int64_t size = static_cast<int64_t>(a.E) * a.N * a.K;
        const dim3 join = grid_of((size / 4 + 255) / 256);
        if (a.out_f32)
            hipLaunchKernelGGL((moe_grouped_dw_join<true>), join, block, 0, s, a.ws, size, splits, a.dw);
        else
            hipLaunchKernelGGL((moe_grouped_dw_join<false>), join, block, 0, s, a.ws, size, splits, a.dw);
    }
    return hipGetLastError();
}

}  // namespace moe
