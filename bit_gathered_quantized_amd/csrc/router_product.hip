// The router's product:  logits[t, e] = rstd_t * sum_c x[t, c] w[e, c],
// rstd_t = 1 / sqrt(mean_c x[t, c]^2 + eps)  (1 without MOE_R_NORM).
//
// A weight of the norm, or a scale of the router, is a factor of w's columns, so
// it belongs in w once; then x enters the product as the bf16 it is, and rstd,
// one number a row, multiplies the finished sum.  Products are exact, sums fp32.
//
// Few tokens (T <= 16): one workgroup an expert, its four waves cut the columns.
// Bound by launch and load latency; the waves read w's row once and x from L2.
//
// More tokens: 16 or 64 tokens by 32 experts a workgroup on
// v_mfma_f32_16x16x32_bf16, eight waves cutting the columns and joined through
// LDS in wave order.  An fp32 w goes in as three bf16 parts, hi + mid + lo = w to
// the last bit (8 + 8 + 8 significant bits), three MFMAs instead of one; a row's
// sum of squares is the diagonal of x x^T, one MFMA more, from operands already
// in registers.
#include "moe_internal.h"

namespace moe {
namespace {

typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t n) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(n), 0x00020000);
}
// 16 bytes at byte offset `at`, zeros past the resource's end.
__device__ __forceinline__ u32x4 load16(Rsrc r, uint32_t at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ float bf16_at(u32x4 v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
}

// ------------------------------------------------------------- few tokens
// v[i] summed over the wave's lanes for every i < N (a power of two); lane l
// returns the sum of i = l / (64 / N).  Each exchange halves what a lane carries.
template <int N>
__device__ __forceinline__ float wave_sums(float (&v)[N], int lane) {
    int off = 32;
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = up ? v[n + i] : v[i], other = up ? v[i] : v[n + i];
            v[i] = mine + __shfl_xor(other, off);
        }
    }
    float s = v[0];
    for (; off > 0; off /= 2) s += __shfl_xor(s, off);
    return s;
}

template <int TM, bool kWF32>
__global__ __launch_bounds__(256) void moe_router_product_few(RouterArgs a) {
    __shared__ float part[2][4][TM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e = blockIdx.x, H = a.H, T = a.T;
    constexpr int kW = kWF32 ? 4 : 2;
    const Rsrc rw = make_rsrc(static_cast<const char*>(a.weight) + static_cast<size_t>(e) * H * kW, H * kW);
    float dot[TM], sq[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) dot[t] = sq[t] = 0.f;
    for (int c = 8 * threadIdx.x; c < H; c += 8 * 256) {  // H is a multiple of 64
        float w[8];
        if constexpr (kWF32) {
            const u32x4 lo = load16(rw, 4 * c), hi = load16(rw, 4 * c + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __uint_as_float(lo[i]);
                w[4 + i] = __uint_as_float(hi[i]);
            }
        } else {
            const u32x4 v = load16(rw, 2 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = bf16_at(v, i);
        }
        u32x4 x[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t)
            x[t] = *reinterpret_cast<const u32x4*>(a.x + min(t, T - 1) * a.x_stride + c);
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = bf16_at(x[t], i);
                dot[t] = fmaf(v, w[i], dot[t]);
                sq[t] = fmaf(v, v, sq[t]);
            }
    }
    const float d = wave_sums<TM>(dot, lane), q = wave_sums<TM>(sq, lane);
    if (lane % (64 / TM) == 0) {
        part[0][wave][lane / (64 / TM)] = d;
        part[1][wave][lane / (64 / TM)] = q;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < T) {
        const int t = threadIdx.x;
        float v = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            v += part[0][w][t];
            s += part[1][w][t];
        }
        a.logits[static_cast<size_t>(t) * a.E + e] = a.norm ? v / sqrtf(s / H + a.eps) : v;
    }
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

constexpr int kTileWaves = 8, kTileExperts = 32;

template <int MT, bool kWF32>
__global__ __launch_bounds__(64 * kTileWaves) void moe_router_product_tile(RouterArgs a) {
    constexpr int kRows = 16 * MT, kW = kWF32 ? 4 : 2, kParts = kWF32 ? 3 : 1;
    __shared__ float part[kTileWaves][kRows][kTileExperts];
    __shared__ float sq[kTileWaves][kRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int H = a.H, E = a.E;
    const int t0 = blockIdx.x * kRows, e0 = blockIdx.y * kTileExperts;
    const int rows = min(kRows, a.T - t0), experts = min(kTileExperts, E - e0);
    // rows past the batch and experts past E read zeros
    const uint32_t xrow = 2u * static_cast<uint32_t>(a.x_stride), wrow = static_cast<uint32_t>(H) * kW;
    const Rsrc rx = make_rsrc(a.x + t0 * a.x_stride, (rows - 1) * xrow + 2u * H);
    const Rsrc rw = make_rsrc(static_cast<const char*>(a.weight) + static_cast<size_t>(e0) * wrow, experts * wrow);

    f32x4 acc[MT][2], gram[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = gram[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = H / 32, s0 = steps * wave / kTileWaves, s1 = steps * (wave + 1) / kTileWaves;
    uint32_t xat[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xat[m] = (16 * m + lr) * xrow + 16u * q;
    const uint32_t wat = lr * wrow + 8u * kW * q;
#pragma unroll 2
    for (int s = s0; s < s1; ++s) {
        u32x4 x[MT], w[2][kParts];
        u32x4 raw[2][kWF32 ? 2 : 1];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < (kWF32 ? 2 : 1); ++h)
                raw[n][h] = load16(rw, wat + 16u * n * wrow + 32u * kW * s + 16u * h);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load16(rx, xat[m] + 64u * s);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if constexpr (kWF32)
                split3(raw[n][0], raw[n][1], w[n]);
            else
                w[n][0] = raw[n][0];
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) acc[m][n] = mfma16(x[m], w[n][p], acc[m][n]);
#pragma unroll
        for (int m = 0; m < MT; ++m) gram[m] = mfma16(x[m], x[m], gram[m]);
    }
    // lane (lr, q) holds rows 4 q + v and column lr of each 16 x 16 product
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int r = 16 * m + 4 * q + v;
            part[wave][r][lr] = acc[m][0][v];
            part[wave][r][16 + lr] = acc[m][1][v];
            if (lr == 4 * q + v) sq[wave][r] = gram[m][v];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kTileExperts; i += 64 * kTileWaves) {
        const int r = i / kTileExperts, e = i % kTileExperts;
        float v = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) {
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
template <int MT>
void tile(const RouterArgs& a, hipStream_t s) {
    const dim3 grid((a.T + 16 * MT - 1) / (16 * MT), (a.E + kTileExperts - 1) / kTileExperts);
    if (a.weight_f32)
        hipLaunchKernelGGL((moe_router_product_tile<MT, true>), grid, dim3(64 * kTileWaves), 0, s, a);
    else
        hipLaunchKernelGGL((moe_router_product_tile<MT, false>), grid, dim3(64 * kTileWaves), 0, s, a);
}

}  // namespace

hipError_t launch_router_product(const RouterArgs& a, hipStream_t s) {
    if (a.T <= 1)
        few<1>(a, s);
    else if (a.T <= 2)
        few<2>(a, s);
    else if (a.T <= 4)
        few<4>(a, s);
    else if (a.T <= 8)
        few<8>(a, s);
    else if (a.T <= 16)
        few<16>(a, s);
    else if (static_cast<int64_t>(a.T) * a.E < 64 * 128 * 32)
        tile<1>(a, s);
    else
        tile<4>(a, s);
    return hipGetLastError();
}

}  // namespace moe
