// The router's product:  logits[t, e] = rstd_t * sum_c x[t, c] w[e, c],
// rstd_t = 1 / sqrt(mean_c x[t, c]^2 + eps)  (1 without MOE_R_NORM).
//
// A weight of the norm, or a scale of the router, is a factor of w's columns, so
// it belongs in w once; then x enters the product as the bf16 it is, and rstd,
// one number a row, multiplies the finished sum.  Products are exact, sums fp32.
//
// Few tokens (T <= 8): one workgroup an expert, its four waves cut the columns.
// Bound by launch and load latency; the waves read w's row once and x from L2
// (8 tokens, 128 experts, H 2816, fp32: 7.7 us with top-k).
//
// More tokens: 16, 32 or 64 tokens by as many experts a workgroup on
// v_mfma_f32_16x16x32_bf16, its waves cutting the columns and joined through LDS
// in wave order.  An fp32 w goes in as three bf16 parts, hi + mid + lo = w to the
// last bit (8 + 8 + 8 significant bits), three MFMAs instead of one; a row's sum
// of squares is the diagonal of x x^T, one MFMA more, from operands already in
// registers.  Bound by cache reads: a tile reads its x and w rows once, so
// larger tiles read less and smaller ones fill the GPU (rule below).  2048 tokens
// and 128 experts: 14 us with bf16 weights, 17 us with fp32.
#include "router_few.h"

namespace moe {
namespace {

using router::load16;
using router::make_rsrc;
using router::Rsrc;

template <int TM, bool kWF32>
__global__ __launch_bounds__(256) void moe_router_product_few(RouterArgs a) {
    __shared__ float part[2][4][16];
    router::few_tokens<TM, kWF32>(a, blockIdx.x, part);
}

// ------------------------------------------------------------- MFMA tiles
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// Eight fp32 values as bf16 hi + mid + lo, exactly.
__device__ __forceinline__ void split3(u32x4 a, u32x4 b, u32x4 (&p)[3]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[s][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            if (s < 2) {
                v[2 * i] -= __uint_as_float(p[s][i] << 16);
                v[2 * i + 1] -= __uint_as_float(p[s][i] & 0xFFFF0000u);
            }
        }
    }
}

// MT row blocks of 16 tokens, NT of 16 experts, WAVES cuts of the columns.  A wave has
// the operands of one step of 32 columns in flight: the other waves fill the time, and
// more steps measured slower (16 x 16 with fp32 weights at 512 tokens, 1 | 2 steps 10.6
// | 11.3 us; 32 x 32 at 2048, 1 | 2 | 3 steps 16.9 | 18.1 | 19.5 us; not measured for
// 64 x 64, whose loads outlast a wave's own MFMAs of a step).
template <int MT, int NT, int WAVES, bool kWF32>
__global__ __launch_bounds__(64 * WAVES) void moe_router_product_tile(RouterArgs a) {
    constexpr int kRows = 16 * MT, kExperts = 16 * NT, kW = kWF32 ? 4 : 2, kRaw = kWF32 ? 2 : 1, kParts = kWF32 ? 3 : 1;
    // wave-private turning buffers in the loop, then the waves' sums
    union Smem {
        u32x4 turn[WAVES][MT + NT * kRaw][64];
        struct {
            float part[WAVES][kRows][kExperts], sq[WAVES][kRows];
        };
    };
    __shared__ Smem sm;
    auto& part = sm.part;
    auto& sq = sm.sq;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int H = a.H, E = a.E;
    // Workgroups go to the XCDs in turn.  A grid of (8, expert blocks, ...) gives all
    // expert blocks of a token block to one XCD, one after the other, so that its x
    // comes from memory once, not once per block; else z is 0.
    const uint32_t first = (blockIdx.x + 8 * blockIdx.z) * kRows;
    if (first >= static_cast<uint32_t>(a.T)) return;  // the whole workgroup
    const int t0 = first, e0 = blockIdx.y * kExperts;
    const int rows = min(kRows, a.T - t0), experts = min(kExperts, E - e0);
    // rows past the batch and experts past E read zeros
    const uint32_t xrow = 2u * static_cast<uint32_t>(a.x_stride), wrow = static_cast<uint32_t>(H) * kW;
    const void* const px = a.x + t0 * a.x_stride;
    const void* const pw = static_cast<const char*>(a.weight) + static_cast<size_t>(e0) * wrow;
    const uint32_t nx = (rows - 1) * xrow + 2u * H, nw = experts * wrow;

    f32x4 acc[MT][NT], gram[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        gram[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = gram[m];
    }
    const int steps = H / 32, s0 = steps * wave / WAVES, s1 = steps * (wave + 1) / WAVES;
    // Loads are coalesced: 4 (fp32 weights: 8) lanes in a row read its 64 (128)
    // bytes of a step.  The operand wants lane (lr, q) to hold columns 8 q .. 8 q + 7
    // of row lr, so each 1 KB goes through LDS, 16-byte pieces XOR-swizzled so that
    // neither side meets a bank twice.  Loading the operand layout directly costs a
    // cache lookup a lane instead of one a row.
    const int r4 = lane >> 2, p4 = lane & 3, r8 = lane >> 3, p8 = lane & 7;
    const uint32_t xat = r4 * xrow + 16u * p4;
    const uint32_t wat = kWF32 ? r8 * wrow + 16u * p8 : r4 * wrow + 16u * p4;
    const int put4 = 4 * r4 + (p4 ^ (r4 >> 2 & 3)), get4 = 4 * lr + (q ^ (lr >> 2 & 3));
    u32x4 x[MT], raw[NT][kRaw];
    // past the wave's share nothing is read
    auto load = [&](int s) {
        const Rsrc rx = make_rsrc(px, s < s1 ? nx : 0), rw = make_rsrc(pw, s < s1 ? nw : 0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < kRaw; ++h)
                raw[n][h] = load16(rw, wat + (16u * n + 8u * h) * wrow + 32u * kW * s);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load16(rx, xat + 16u * m * xrow + 64u * s);
    };
    auto compute = [&] {
        u32x4 (&buf)[MT + NT * kRaw][64] = sm.turn[wave];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (kWF32) {  // rows of 8 pieces over two buffers, row r8 + 8 h
#pragma unroll
                for (int h = 0; h < 2; ++h) buf[MT + 2 * n + h][8 * r8 + (p8 ^ ((r8 + 8 * h) >> 1 & 7))] = raw[n][h];
            } else {
                buf[MT + n][put4] = raw[n][0];
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) buf[m][put4] = x[m];
        __builtin_amdgcn_wave_barrier();
        u32x4 w[NT][kParts], xo[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) xo[m] = buf[m][get4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (kWF32) {
                const u32x4* row = &buf[MT + 2 * n + (lr >> 3)][8 * (lr & 7)];
                split3(row[(2 * q) ^ (lr >> 1 & 7)], row[(2 * q + 1) ^ (lr >> 1 & 7)], w[n]);
            } else {
                w[n][0] = buf[MT + n][get4];
            }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] = mfma16(xo[m], w[n][p], acc[m][n]);
#pragma unroll
        for (int m = 0; m < MT; ++m) gram[m] = mfma16(xo[m], xo[m], gram[m]);
    };
    load(s0);
    for (int s = s0; s < s1; ++s) {
        compute();
        load(s + 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();  // the turning buffers become the sums
    // lane (lr, q) holds rows 4 q + v and column lr of each 16 x 16 product
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int r = 16 * m + 4 * q + v;
#pragma unroll
            for (int n = 0; n < NT; ++n) part[wave][r][16 * n + lr] = acc[m][n][v];
            if (lr == 4 * q + v) sq[wave][r] = gram[m][v];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kExperts; i += 64 * WAVES) {
        const int r = i / kExperts, e = i % kExperts;
        float v = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            v += part[w][r][e];
            s += sq[w][r];
        }
        if (r < rows && e < experts)
            a.logits[static_cast<size_t>(t0 + r) * E + e0 + e] = a.norm ? v / sqrtf(s / H + a.eps) : v;
    }
}

template <int TM>
void few(const RouterArgs& a, hipStream_t s) {
    if (a.weight_f32)
        hipLaunchKernelGGL((moe_router_product_few<TM, true>), dim3(a.E), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((moe_router_product_few<TM, false>), dim3(a.E), dim3(256), 0, s, a);
}
template <int MT, int NT, int WAVES>
void tile(const RouterArgs& a, hipStream_t s) {
    const uint32_t down = (static_cast<uint32_t>(a.T) + 16 * MT - 1) / (16 * MT), across = (a.E + 16 * NT - 1) / (16 * NT);
    // By XCD where x would be read often and every XCD has its share.  By XCD | not:
    // 4001 tokens and 512 experts (8 blocks across) 56 | 72 us; 4 or 2 across 18.0 |
    // 17.9 and 28.3 | 27.7 us; 16 tokens and 128 experts 12 | 10 us.
    const bool by_xcd = across > 4 && down >= 8 && down <= 8 * 65535;
    const dim3 grid(by_xcd ? 8 : down, across, by_xcd ? (down + 7) / 8 : 1), block(64 * WAVES);
    if (a.weight_f32)
        hipLaunchKernelGGL((moe_router_product_tile<MT, NT, WAVES, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((moe_router_product_tile<MT, NT, WAVES, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_router_product(const RouterArgs& a, hipStream_t s) {
    const int64_t T = a.T, E = a.E;
    // workgroups of the tile of m row blocks by n blocks of experts
    auto groups = [&](int m, int n) { return (T + 16 * m - 1) / (16 * m) * ((E + 16 * n - 1) / (16 * n)); };
    if (T <= 1)
        few<1>(a, s);
    else if (T <= 2)
        few<2>(a, s);
    else if (T <= 4)
        few<4>(a, s);
    else if (T <= 8)
        few<8>(a, s);
    // the largest tile that still gives every other CU a workgroup.  Measured with top-k,
    // 64 x 64 | 32 x 32 | 16 x 16, 128 experts: 8192 tokens 35 | 46 | 105 us, 5120
    // 29.4 | 34 us, 4096 29.9 | 27 us, 2048 22 | 14 | 26 us, 512 18 | 11.3 | 9.8 us
    // (fp32 weights 28 | 16 | 13 us), 64 (fp32) 24 | 15 | 10 us.  With more than one
    // 64 x 64 workgroup a CU two of four waves at a time, so that one starts or ends
    // while the other multiplies, not one of eight (4001 tokens and 512 experts 53 | 58
    // us; 8192 and 128, one to a CU, 42 | 35 us)
    else if (groups(4, 4) > 256)
        tile<4, 4, 4>(a, s);
    else if (groups(4, 4) > 128)
        tile<4, 4, 8>(a, s);
    else if (groups(2, 2) >= 128)
        tile<2, 2, 8>(a, s);
    else
        tile<1, 1, 16>(a, s);
    return hipGetLastError();
}

}  // namespace moe
