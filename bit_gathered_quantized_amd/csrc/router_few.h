// The router's product for few tokens: one expert's logits by a workgroup of
// four waves that cut the columns.  Shared by the router's own launch and by the
// layer's first.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

namespace router {

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

// Logits of expert e for a.T <= TM tokens, by 256 threads.
template <int TM, bool kWF32>
__device__ __forceinline__ void few_tokens(const RouterArgs& a, int e, float (&part)[2][4][16]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int H = a.H, T = a.T;
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

}  // namespace router
}  // namespace
}  // namespace moe
