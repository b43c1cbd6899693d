// The norms around a block of one row, in registers: shared by the block norm's
// kernel and the layer's last step.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

namespace norm {

// A buffer resource over one row of a tensor (p the same in every lane of a
// wave).  Loads past its end, or from a tensor that is absent (p == nullptr),
// read nothing and return zeros, stores there are dropped: no branch stands
// between the loads of a row, so they are all in flight together.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc row_rsrc(const void* p, int64_t row_bytes, int64_t row, int H, int size) {
    const char* q = static_cast<const char*>(p) + (p ? row * row_bytes : 0);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(q), 0, p ? H * size : 0, 0x00020000);
}

// VEC values as loaded: fp32 in lo and hi, bf16 in lo alone.
template <int VEC>
struct Raw {
    u32x4 lo, hi;
};
template <>
struct Raw<1> {
    uint32_t u;
};
// `h` is `r` for an fp32 tensor and an empty resource for a bf16 one.
template <int VEC>
__device__ __forceinline__ Raw<VEC> load_raw(Rsrc r, Rsrc h, int c, bool f32) {
    Raw<VEC> v;
    if constexpr (VEC == 1) {
        const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(h, 4 * c, 0, 0);
        v.u = f32 ? w : static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * c, 0, 0)) << 16;
    } else {
        const int at = f32 ? 4 * c : 2 * c;
        v.lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        v.hi = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(h, at + 16, 0, 0));
    }
    return v;
}
// The same for a type known when compiling.
template <int VEC, bool kF32>
__device__ __forceinline__ Raw<VEC> load_raw(Rsrc r, int c) {
    Raw<VEC> v;
    if constexpr (VEC == 1) {
        if constexpr (kF32)
            v.u = __builtin_amdgcn_raw_buffer_load_b32(r, 4 * c, 0, 0);
        else
            v.u = static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * c, 0, 0)) << 16;
    } else {
        v.lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (kF32 ? 4 : 2) * c, 0, 0));
        if constexpr (kF32)
            v.hi = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * c + 16, 0, 0));
    }
    return v;
}
template <int VEC>
__device__ __forceinline__ float value(const Raw<VEC>& r, int i, bool f32) {
    if constexpr (VEC == 1) {
        return __uint_as_float(r.u);
    } else {
        const uint32_t w = i < 4 ? r.lo[i & 3] : r.hi[i & 3], p = r.lo[i >> 1];
        return __uint_as_float(f32 ? w : (i & 1 ? p & 0xFFFF0000u : p << 16));
    }
}
template <int VEC>
__device__ __forceinline__ void store_values(Rsrc r, int c, const float (&v)[VEC], bool f32) {
    if constexpr (VEC == 1) {
        if (f32)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, 4 * c, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v[0]), r, 2 * c, 0, 0);
    } else if (f32) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), r, 4 * c, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}), r, 4 * c + 16, 0,
                                               0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])},
                                               r, 2 * c, 0, 0);
    }
}

// Sum of v over the WAVES waves that share a row, the same value in every
// thread: lanes by exchange, waves through LDS in wave order.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* lds) {
    // lanes i ^ 1, i ^ 2, then mirrors of 8 and 16 once quads agree, without LDS
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += lds[w];
    }
    return v;
}

// The row of one token from its loads to its stores, but for the block's output,
// which the caller brings as z (zeros past H).  WAVES waves own the row, NV * VEC
// values a thread: value v of piece i is column c0 + 64 WAVES VEC i + v.  kS: the
// type of residual and out, 1 fp32, 0 bf16, -1 a.stream_f32 says.
template <int WAVES, int NV, int VEC, int kS>
struct Row {
    static constexpr int kStep = 64 * WAVES * VEC;
    // 16 values a thread in 16-wave workgroups: 128 registers, so the gate and
    // the last weights are loaded once the others are done with
    static constexpr bool kLate = VEC == 1 && NV >= 16;
    Raw<VEC> rr[NV], rp[NV], rn[NV], rg[NV];
    float g0;
    bool sf32, wf32, gf32, channel;
    Rsrc sg, hg, sn, hn;

    __device__ __forceinline__ void load_gate(int c0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rg[i] = load_raw<VEC>(sg, hg, c0 + i * kStep, gf32);
    }
    __device__ __forceinline__ void load_pre(int c0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rn[i] = load_raw<VEC>(sn, hn, c0 + i * kStep, wf32);
    }
    __device__ __forceinline__ void load(const NormArgs& a, int64_t t, int c0) {
        const int H = a.H;
        sf32 = kS < 0 ? a.stream_f32 : kS == 1;
        wf32 = a.weight_f32;
        gf32 = a.gate_f32;
        channel = a.gate != nullptr && a.gate_stride_h != 0;
        const int ssize = sf32 ? 4 : 2, wsize = wf32 ? 4 : 2, gsize = gf32 ? 4 : 2;
        const Rsrc none = row_rsrc(nullptr, 0, 0, 0, 0);
        const Rsrc sr = row_rsrc(a.residual, a.residual_stride * ssize, t, H, ssize), hr = sf32 ? sr : none;
        const Rsrc sp = row_rsrc(a.post_weight, 0, 0, H, wsize), hp = wf32 ? sp : none;
        sn = row_rsrc(a.pre_weight, 0, 0, H, wsize);
        hn = wf32 ? sn : none;
        sg = row_rsrc(channel ? a.gate : nullptr, a.gate_stride_t * gsize, t, H, gsize);
        hg = gf32 ? sg : none;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (kS < 0)
                rr[i] = load_raw<VEC>(sr, hr, c0 + i * kStep, sf32);
            else
                rr[i] = load_raw<VEC, kS == 1>(sr, c0 + i * kStep);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) rp[i] = load_raw<VEC>(sp, hp, c0 + i * kStep, wf32);
        if constexpr (!kLate) {
            load_gate(c0);
            load_pre(c0);
        }
        g0 = a.gate_scale;
        if (a.gate && !channel)
            g0 *= gf32 ? static_cast<const float*>(a.gate)[t * a.gate_stride_t]
                       : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t * a.gate_stride_t]);
    }
    __device__ __forceinline__ void finish(const NormArgs& a, int64_t t, int c0, float (&z)[NV][VEC],
                                           float (&lds)[2][16]) {
        const int H = a.H;
        if (a.post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < VEC; ++v) ss = fmaf(z[i][v], z[i][v], ss);
            const float rstd = 1.f / sqrtf(row_sum<WAVES>(ss, lds[0]) / H + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    z[i][v] *= rstd * (a.post_weight ? a.weight_offset + value(rp[i], v, wf32) : 1.f);
        }
        if constexpr (kLate) load_gate(c0);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = c0 + i * kStep < H;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                z[i][v] *= channel ? g0 * value(rg[i], v, gf32) : g0;
                if (a.residual) z[i][v] = fmaf(a.residual_scale, value(rr[i], v, sf32), z[i][v]);
                // past H the zeros may have met an infinite factor: left out
                ss = in ? fmaf(z[i][v], z[i][v], ss) : ss;
            }
        }
        if constexpr (kLate) load_pre(c0);
        const int ssize = sf32 ? 4 : 2;
        const Rsrc so = row_rsrc(a.out, a.out_stride * ssize, t, H, ssize);
#pragma unroll
        for (int i = 0; i < NV; ++i) store_values(so, c0 + i * kStep, z[i], sf32);
        if (a.normed) {
            const int nsize = a.normed_f32 ? 4 : 2;
            const Rsrc sm = row_rsrc(a.normed, a.normed_stride * nsize, t, H, nsize);
            const float rstd = 1.f / sqrtf(row_sum<WAVES>(ss, lds[1]) / H + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    z[i][v] *= rstd * (a.pre_weight ? a.weight_offset + value(rn[i], v, wf32) : 1.f);
                store_values(sm, c0 + i * kStep, z[i], a.normed_f32);
            }
        }
    }
};

}  // namespace norm
}  // namespace
}  // namespace moe
