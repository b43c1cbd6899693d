// Grouped products on microscaled weights, with microscaled or bf16 rows, in tiles of BM
// rows by BN columns.
#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

// LDS row r of w holds this column of the tile, so that a lane ends up with 8
// neighbouring columns of two products.
__device__ __forceinline__ int column_of(int r) {
    const int f = r >> 4, i = r & 15;
    return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
}

// Bytes [at, at + 16) of a row of `size` scale bytes that starts at p; zeros past its
// end (`at` is uniform).
__device__ __forceinline__ u32x4 scales16(const uint8_t* p, int at, int size) {
    u32x4 v = {0, 0, 0, 0};
    if (at + 16 <= size) {
        __builtin_memcpy(&v, p + at, 16);  // any alignment
    } else {
        for (int i = 0; at + i < size; ++i) {
            const uint32_t b = static_cast<uint32_t>(p[at + i]) << (8 * (i & 3));
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] |= (i >> 2) == w ? b : 0;
        }
    }
    return v;
}

// The results of a wave: lane (lr, q) of a product holds columns 8 q + 4 (f % 2) .. + 3 of
// row lr.
template <int FM, int FN, bool kF32>
__device__ __forceinline__ void store_rows(const GroupedArgs& a, const Tile& t, const f32x4 (&acc)[FN][FM], int n0, int cols,
                                           int m_at, int n_at, int lr, int q) {
    constexpr int kOut = kF32 ? 4 : 2;
    unsigned char* const out = static_cast<unsigned char*>(a.out) + t.row * a.out_stride + static_cast<int64_t>(kOut) * n0;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
        const int row = m_at + 16 * m + lr;
        if (row >= t.rows) continue;
        unsigned char* const o = out + row * a.out_stride;
#pragma unroll
        for (int f = 0; f < FN; f += 2) {
            const f32x4 v = acc[f][m], u = acc[f + 1][m];
            const int col = n_at + 16 * f + 8 * q;
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

// Both sides microscaled.  A stage is 128 bytes of codes (256 values) of a row; pieces of
// 16 bytes, one block of 32 each, are XORed with the row's number.  Scales of two stages
// lie beside them, 16 bytes a row, ordered so that lane quarter q reads its four (blocks
// 2 q and 2 q + 1 of both stages) as one word.
template <int BM, int BN, int WM, int WN, bool kF32>
__global__ __launch_bounds__(64 * WM * WN) void moe_grouped_mx_tile(GroupedArgs a, uint32_t most, uint32_t across) {
    constexpr int kWaves = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int kXJobs = BM / 8 / kWaves, kWJobs = BN / 8 / kWaves, kSJobs = (BM + BN) / (64 * kWaves);
    static_assert(kXJobs * 8 * kWaves == BM && kWJobs * 8 * kWaves == BN && FN % 2 == 0, "tile");
    static_assert(kSJobs * 64 * kWaves == BM + BN && BM % 64 == 0, "scales");
    __shared__ __align__(16) unsigned char x0[BM * 128], x1[BM * 128], w0[BN * 128], w1[BN * 128];
    __shared__ __align__(16) unsigned char scale[2][(BM + BN) * 16];
    Tile t;
    if (!find_tile<BM, 8>(a.offsets, a.A, a.E, most, across, grid_index(), t)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int n0 = t.n * BN, cols = min(BN, a.N - n0);
    const int kbytes = a.K / 2, blocks = a.K / 32;

    const unsigned char* const px = static_cast<const unsigned char*>(a.x) + static_cast<int64_t>(t.row) * kbytes;
    const unsigned char* const pw = static_cast<const unsigned char*>(a.w) + (static_cast<int64_t>(t.expert) * a.N + n0) * kbytes;
    const Rsrc rx = make_rsrc(px, static_cast<uint32_t>(t.rows) * kbytes), rw = make_rsrc(pw, static_cast<uint32_t>(cols) * kbytes);
    const uint32_t piece = 16u * ((lane & 7) ^ (lane >> 3));
    uint32_t xat[kXJobs], wat[kWJobs];
#pragma unroll
    for (int j = 0; j < kXJobs; ++j)
        xat[j] = static_cast<uint32_t>(min(8 * (j * kWaves + wave) + (lane >> 3), t.rows - 1) * kbytes) + piece;
#pragma unroll
    for (int j = 0; j < kWJobs; ++j)
        wat[j] = static_cast<uint32_t>(min(column_of(8 * (j * kWaves + wave) + (lane >> 3)), cols - 1) * kbytes) + piece;
    const uint8_t* ps[kSJobs];  // this thread's rows of scales
#pragma unroll
    for (int j = 0; j < kSJobs; ++j) {
        const int r = 64 * (j * kWaves + wave) + lane;
        ps[j] = r < BM ? a.xs + static_cast<int64_t>(t.row + min(r, t.rows - 1)) * blocks
                       : a.ws + (static_cast<int64_t>(t.expert) * a.N + n0 + min(column_of(r - BM), cols - 1)) * blocks;
    }
    const int stages = (a.K + 255) / 256;
    auto issue = [&](unsigned char* xs, unsigned char* ws, int s) {
        const uint32_t k = 128u * s;
        const bool inside = k + piece < static_cast<uint32_t>(kbytes);
#pragma unroll
        for (int j = 0; j < kXJobs; ++j)
            copy16(rx, xs + 1024 * (j * kWaves + wave), inside ? xat[j] : kOutside, k);
#pragma unroll
        for (int j = 0; j < kWJobs; ++j)
            copy16(rw, ws + 1024 * (j * kWaves + wave), inside ? wat[j] : kOutside, k);
    };
    u32x4 next[kSJobs];
    auto load_scales = [&](int pair) {
#pragma unroll
        for (int j = 0; j < kSJobs; ++j) next[j] = scales16(ps[j], 16 * pair, blocks);
    };
    auto put_scales = [&](int pair) {
#pragma unroll
        for (int j = 0; j < kSJobs; ++j) {
            const u32x4 v = next[j];
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = i & 1 ? (v[i >> 1] >> 16) | (v[2 + (i >> 1)] & 0xFFFF0000u)
                             : (v[i >> 1] & 0xFFFFu) | (v[2 + (i >> 1)] << 16);
            *reinterpret_cast<u32x4*>(&scale[pair & 1][16 * (64 * (j * kWaves + wave) + lane)]) = o;
        }
    };
    f32x4 acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint32_t sx[FM], sw[FN];
    auto get_scales = [&](int pair) {
        const unsigned char* const p = scale[pair & 1] + 16 * lr + 4 * q;
#pragma unroll
        for (int m = 0; m < FM; ++m) sx[m] = *reinterpret_cast<const uint32_t*>(p + 256 * (wm * FM + m));
#pragma unroll
        for (int f = 0; f < FN; ++f) sw[f] = *reinterpret_cast<const uint32_t*>(p + 16 * BM + 256 * (wn * FN + f));
    };
    auto compute = [&](const unsigned char* xs, const unsigned char* ws, auto odd) {
        constexpr int kOdd = decltype(odd)::value;
        auto step = [&](auto which) {
            constexpr int S = decltype(which)::value;
            const int at = 128 * lr + 16 * ((2 * q + S) ^ (lr & 7));
            u32x4 wf[FN], xf[FM];
#pragma unroll
            for (int f = 0; f < FN; ++f) wf[f] = read16(ws, at + 2048 * (wn * FN + f));
#pragma unroll
            for (int m = 0; m < FM; ++m) xf[m] = read16(xs, at + 2048 * (wm * FM + m));
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int m = 0; m < FM; ++m)
                    acc[f][m] = mfma_mx<2 * kOdd + S, 2 * kOdd + S>(wf[f], xf[m], acc[f][m], sw[f], sx[m]);
        };
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
    };
    issue(x0, w0, 0);
    load_scales(0);
    put_scales(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the scales are in LDS
    copies_done<0>();
    for (int s = 0; s < stages; s += 2) {
        const int pair = s >> 1;
        const bool more = s + 2 < stages;
        if (more) load_scales(pair + 1);
        if (s + 1 < stages) issue(x1, w1, s + 1);
        get_scales(pair);
        compute(x0, w0, std::integral_constant<int, 0>());
        copies_done<0>();
        if (s + 1 >= stages) break;
        if (more) issue(x0, w0, s + 2);
        compute(x1, w1, std::integral_constant<int, 1>());
        if (more) put_scales(pair + 1);
        __builtin_amdgcn_s_waitcnt(0xC07F);
        copies_done<0>();
    }
    store_rows<FM, FN, kF32>(a, t, acc, n0, cols, 16 * wm * FM, 16 * wn * FN, lr, q);
}

// bf16 rows.  A stage is 128 values of K: 256 bytes of a row of x, 64 of w.  A lane
// quarter q holds block q of the stage: its 16 bytes of codes become four operands, word
// i of the codes against x's values 32 q + 8 i .. + 7.  A code under its scale is exact in
// bf16.
template <int BM, int BN, int WM, int WN, bool kF32>
__global__ __launch_bounds__(64 * WM * WN) void moe_grouped_bf16_mx_tile(GroupedArgs a, uint32_t most, uint32_t across) {
    constexpr int kWaves = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int kXJobs = BM / 4 / kWaves, kWJobs = BN / 16 / kWaves, kThreads = 64 * kWaves;
    static_assert(kXJobs * 4 * kWaves == BM && kWJobs * 16 * kWaves == BN && FN % 2 == 0 && kWaves % 4 == 0, "tile");
    static_assert(BN <= kThreads, "scales");
    __shared__ __align__(16) unsigned char x0[BM * 256], x1[BM * 256], w0[BN * 64], w1[BN * 64];
    __shared__ __align__(16) unsigned char scale[2][BN * 16];
    Tile t;
    if (!find_tile<BM, 8>(a.offsets, a.A, a.E, most, across, grid_index(), t)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int n0 = t.n * BN, cols = min(BN, a.N - n0);
    const int wbytes = a.K / 2, blocks = a.K / 32;
    const uint32_t xbytes = 2u * a.K;

    const unsigned char* const px = static_cast<const unsigned char*>(a.x) + t.row * a.x_stride;
    const unsigned char* const pw = static_cast<const unsigned char*>(a.w) + (static_cast<int64_t>(t.expert) * a.N + n0) * wbytes;
    const Rsrc rx = make_rsrc(px, static_cast<uint32_t>((t.rows - 1) * a.x_stride) + xbytes);
    const Rsrc rw = make_rsrc(pw, static_cast<uint32_t>(cols) * wbytes);
    const uint32_t xpiece = 16u * (lr ^ ((4 * wave + q) & 15)), wpiece = 16u * ((lane & 3) ^ (lane >> 3 & 3));
    uint32_t xat[kXJobs], wat[kWJobs];
#pragma unroll
    for (int j = 0; j < kXJobs; ++j)
        xat[j] = static_cast<uint32_t>(min(4 * (j * kWaves + wave) + q, t.rows - 1)) * static_cast<uint32_t>(a.x_stride) + xpiece;
#pragma unroll
    for (int j = 0; j < kWJobs; ++j)
        wat[j] = static_cast<uint32_t>(min(column_of(16 * (j * kWaves + wave) + (lane >> 2)), cols - 1) * wbytes) + wpiece;
    const uint8_t* const ps = a.ws + (static_cast<int64_t>(t.expert) * a.N + n0 + min(column_of(threadIdx.x), cols - 1)) * blocks;
    const int stages = (a.K + 127) / 128;
    auto issue = [&](unsigned char* xs, unsigned char* ws, int s) {
        const bool xin = 256u * s + xpiece < xbytes, win = 64u * s + wpiece < static_cast<uint32_t>(wbytes);
#pragma unroll
        for (int j = 0; j < kXJobs; ++j)
            copy16(rx, xs + 1024 * (j * kWaves + wave), xin ? xat[j] : kOutside, 256u * s);
#pragma unroll
        for (int j = 0; j < kWJobs; ++j)
            copy16(rw, ws + 1024 * (j * kWaves + wave), win ? wat[j] : kOutside, 64u * s);
    };
    u32x4 next;
    auto put_scales = [&](int four) {  // word q of a row: block q of each of four stages
        if (BN < kThreads && threadIdx.x >= BN) return;
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i] |= (next[j] >> (8 * i) & 0xFFu) << (8 * j);
        }
        *reinterpret_cast<u32x4*>(&scale[four & 1][16 * threadIdx.x]) = o;
    };
    f32x4 acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const unsigned char* xs, const unsigned char* ws, int s) {
        const unsigned char* const sc = scale[s >> 2 & 1] + 16 * lr + 4 * q + (s & 3);
        u32x4 xf[4][FM];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < FM; ++m) xf[i][m] = read16(xs, 256 * (16 * (wm * FM + m) + lr) + 16 * ((4 * q + i) ^ lr));
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const u32x4 c = read16(ws, 64 * (16 * (wn * FN + f) + lr) + 16 * (q ^ (lr >> 1 & 3)));
            const float unit = mx_scale(sc[256 * (wn * FN + f)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 w = mx_as_bf16(c[i], unit);
#pragma unroll
                for (int m = 0; m < FM; ++m) acc[f][m] = mfma_bf16(w, xf[i][m], acc[f][m]);
            }
        }
    };
    issue(x0, w0, 0);
    next = scales16(ps, 0, blocks);
    put_scales(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the scales are in LDS
    copies_done<0>();
    for (int s = 0; s < stages; s += 2) {
        // scales of four stages are loaded in the first two before them and put in the second
        if (s % 4 == 0) next = scales16(ps, 4 * s + 16, blocks);
        if (s + 1 < stages) issue(x1, w1, s + 1);
        compute(x0, w0, s);
        copies_done<0>();
        if (s + 1 >= stages) break;
        if (s + 2 < stages) issue(x0, w0, s + 2);
        compute(x1, w1, s + 1);
        if (s % 4 == 2) put_scales((s >> 2) + 1);
        __builtin_amdgcn_s_waitcnt(0xC07F);
        copies_done<0>();
    }
    store_rows<FM, FN, kF32>(a, t, acc, n0, cols, 16 * wm * FM, 16 * wn * FN, lr, q);
}

template <int BM, int BN>
dim3 tiles(const GroupedArgs& a, uint32_t& most, uint32_t& across) {
    most = static_cast<uint32_t>(grid_tiles(a, BM));
    across = (a.N + BN - 1) / BN;
    return grid_of((static_cast<int64_t>(most) * across + 7) / 8 * 8);  // a multiple of 8: the XCDs' shares are rounded up
}

}  // namespace

hipError_t launch_grouped_mx(const GroupedArgs& a, hipStream_t s) {
    uint32_t most, across;
    const dim3 grid = tiles<128, 128>(a, most, across);
    if (a.out_f32)
        hipLaunchKernelGGL((moe_grouped_mx_tile<128, 128, 2, 2, true>), grid, dim3(256), 0, s, a, most, across);
    else
        hipLaunchKernelGGL((moe_grouped_mx_tile<128, 128, 2, 2, false>), grid, dim3(256), 0, s, a, most, across);
    return hipGetLastError();
}

hipError_t launch_grouped_bf16_mx(const GroupedArgs& a, hipStream_t s) {
    uint32_t most, across;
    const dim3 grid = tiles<64, 128>(a, most, across);
    if (a.out_f32)
        hipLaunchKernelGGL((moe_grouped_bf16_mx_tile<64, 128, 1, 4, true>), grid, dim3(256), 0, s, a, most, across);
    else
        hipLaunchKernelGGL((moe_grouped_bf16_mx_tile<64, 128, 1, 4, false>), grid, dim3(256), 0, s, a, most, across);
    return hipGetLastError();
}

}  // namespace moe
