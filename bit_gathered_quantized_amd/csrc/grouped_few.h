// Grouped products for few rows an expert: bound by reading the weights, and for the
// smallest calls by the latency of doing so.
//
// A workgroup takes 16 rows of an expert by 16 NT columns.  Its eight waves cut K and join
// their sums through LDS in wave order; each streams its part of the weights straight into
// registers, kAhead steps at a time with the next ones on their way, so that all of a short product is
// under way at once.  A step is 64 bytes of a row of w, a lane quarter q holding 16 of them: 32
// of K in bf16, 128 (a block a quarter) of codes.
#pragma once

#include "grouped_product.h"

namespace moe {
namespace {

// Workgroup `index` takes block index % blocks of the columns of strip index / blocks, of all
// strips of up to 16 rows in the order of the experts; false past the last.  All values
// are uniform.
__device__ __forceinline__ bool few_strip(const GroupedArgs& a, uint32_t want, int& expert, int& row, int& rows) {
    const int lane = threadIdx.x & 63;
    if (!a.offsets) {
        expert = 0;
        row = 16 * want;
        rows = min(16, a.A - row);
        return rows > 0;
    }
    uint32_t before = 0;
    for (int base = 0; base < a.E; base += 256) {  // four loads in flight
        int lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) expert_rows(a.offsets, base + 64 * i + lane, a.E, a.A, lo[i], hi[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int mine = (hi[i] - lo[i] + 15) / 16;
            const uint32_t upto = before + static_cast<uint32_t>(wave_scan(min(mine, 1 << 24)));
            const uint64_t hit = __builtin_amdgcn_ballot_w64(upto > want);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                expert = base + 64 * i + l;
                const int number = static_cast<int>(want) - (__builtin_amdgcn_readlane(static_cast<int>(upto), l) - __builtin_amdgcn_readlane(mine, l));
                const int end = __builtin_amdgcn_readlane(hi[i], l);
                row = min(__builtin_amdgcn_readlane(lo[i], l) + 16 * number, end);
                rows = min(16, end - row);
                return rows > 0;
            }
            before = min(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), 63)), 1u << 24);
        }
    }
    return false;
}

template <Form F, int NT, bool kF32>
__global__ __launch_bounds__(512) void moe_grouped_few(GroupedArgs a, uint32_t blocks) {
    constexpr bool kMxX = F == Form::kMx, kMxW = F != Form::kRows;
    constexpr int kWaves = 8, kWide = 16 * NT, kAhead = NT == 4 || F == Form::kBf16Mx ? 2 : 4;
    constexpr int kX = F == Form::kBf16Mx ? 4 : 1;  // 16-byte pieces of x a step and lane
    __shared__ float part[kWaves][NT][256];
    const uint32_t index = grid_index(), strip = index / blocks;
    int expert, row0, rows;
    if (!few_strip(a, strip, expert, row0, rows)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int n0 = static_cast<int>(index - strip * blocks) * kWide, cols = min(kWide, a.N - n0);
    const uint32_t xbytes = kMxX ? a.K / 2 : 2u * a.K, wbytes = kMxW ? a.K / 2 : 2u * a.K, scale_row = a.K / 32;
    const int64_t xs = kMxX ? static_cast<int64_t>(xbytes) : a.x_stride, ws = kMxW ? static_cast<int64_t>(wbytes) : a.w_stride;
    const int64_t w_row = static_cast<int64_t>(expert) * a.N + n0;
    const Rsrc rx = make_rsrc(static_cast<const unsigned char*>(a.x) + row0 * xs, static_cast<uint32_t>((rows - 1) * xs) + xbytes);
    const Rsrc rw = make_rsrc(kMxW ? static_cast<const unsigned char*>(a.w) + w_row * ws
                                   : static_cast<const unsigned char*>(a.w) + expert * a.w_expert + n0 * ws,
                              static_cast<uint32_t>((cols - 1) * ws) + wbytes);
    const Rsrc rxs = make_rsrc(kMxX ? a.xs + static_cast<int64_t>(row0) * scale_row : nullptr, kMxX ? rows * scale_row : 0);
    const Rsrc rws = make_rsrc(kMxW ? a.ws + w_row * scale_row : nullptr, kMxW ? cols * scale_row : 0);
    const uint32_t xat = lr < rows ? static_cast<uint32_t>(lr) * static_cast<uint32_t>(xs) : kOutside;
    uint32_t wat[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int c = 16 * t + lr;
        wat[t] = c < cols ? static_cast<uint32_t>(c) * static_cast<uint32_t>(ws) : kOutside;
    }

    struct Step {
        u32x4 x[kX], w[NT];
        uint32_t sx, sw[NT];
    };
    auto load16 = [](Rsrc r, uint32_t at) { return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0)); };
    auto load1 = [](Rsrc r, uint32_t at) { return static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b8(r, at, 0, 0)); };
    const int steps = (wbytes + 63) / 64, s0 = steps * wave / kWaves, s1 = steps * (wave + 1) / kWaves;
    // what lies past the row, the columns, the end of K or this wave's part reads zeros
    auto load = [&](Step& p, int s) {
        const uint32_t k = 64u * s + 16u * q;  // of a row of w
        const bool in = s < s1 && k < wbytes;
        const uint32_t scale = 4u * s + q;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const bool there = in && wat[t] != kOutside;
            p.w[t] = load16(rw, there ? wat[t] + k : kOutside);
            if constexpr (kMxW) p.sw[t] = load1(rws, there ? (16 * t + lr) * scale_row + scale : kOutside);
        }
        const bool there = in && xat != kOutside;
#pragma unroll
        for (int i = 0; i < kX; ++i) p.x[i] = load16(rx, there ? xat + kX * k + 16 * i : kOutside);
        if constexpr (kMxX) p.sx = load1(rxs, there ? lr * scale_row + scale : kOutside);
    };
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Step& p) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (F == Form::kRows) {
                acc[t] = mfma_bf16(p.w[t], p.x[0], acc[t]);
            } else if constexpr (kMxX) {
                acc[t] = mfma_mx<0, 0>(p.w[t], p.x[0], acc[t], p.sw[t], p.sx);
            } else {
                const float unit = mx_scale(p.sw[t]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t] = mfma_bf16(mx_as_bf16(p.w[t][i], unit), p.x[i], acc[t]);
            }
        }
    };
    Step now[kAhead], next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(now[i], s0 + i);
    for (int s = s0; s < s1; s += 2 * kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(next[i], s + kAhead + i);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) multiply(now[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(now[i], s + 2 * kAhead + i);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) multiply(next[i]);
    }
    // lane (lr, q) holds columns 4 q .. 4 q + 3 of row lr
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(&part[wave][t][16 * lr + 4 * q]) = acc[t];
    __syncthreads();
    // a thread two neighbouring columns of a row
    for (int i = threadIdx.x; i < 8 * kWide; i += 512) {
        const int r = i / (kWide / 2), c = 2 * (i % (kWide / 2));
        if (r >= rows || c >= cols) continue;
        float v = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float* const p = &part[w][c >> 4][16 * r + (c & 15)];
            v += p[0];
            u += p[1];
        }
        unsigned char* const o = static_cast<unsigned char*>(a.out) + (row0 + r) * a.out_stride;
        if constexpr (kF32)
            *reinterpret_cast<float2*>(o + 4 * static_cast<int64_t>(n0 + c)) = float2{v, u};
        else
            *reinterpret_cast<uint32_t*>(o + 2 * static_cast<int64_t>(n0 + c)) = pack_bf16x2(v, u);
    }
}

template <Form F, int NT>
void launch_few_tile(const GroupedArgs& a, int64_t most, hipStream_t s) {
    const uint32_t blocks = (a.N + 16 * NT - 1) / (16 * NT);
    const dim3 grid = grid_of(most * blocks);
    if (a.out_f32)
        hipLaunchKernelGGL((moe_grouped_few<F, NT, true>), grid, dim3(512), 0, s, a, blocks);
    else
        hipLaunchKernelGGL((moe_grouped_few<F, NT, false>), grid, dim3(512), 0, s, a, blocks);
}

template <Form F>
void launch_few(const GroupedArgs& a, hipStream_t s) {
    // Narrow tiles until there are two for every CU.  16 | 64 columns, K 4096 by N 4096, bf16: 1 row
    // 9.4 | 19 us, 32 rows (512 narrow tiles) 19 | 22 us, 64 rows 34 | 22 us.
    const int64_t most = most_strips(a, 16);
    if (most * ((a.N + 15) / 16) > 512)
        launch_few_tile<F, 4>(a, most, s);
    else
        launch_few_tile<F, 1>(a, most, s);
}

}  // namespace
}  // namespace moe
