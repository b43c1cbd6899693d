// Norms around a block, fused with the block's gate and the residual scale:
//
//   z      = gate_scale * gate * (rms(y) * (offset + post_weight)   or   y)
//   out    = residual_scale * residual + z
//   normed = rms(out) * (offset + pre_weight)         rms(v) = v / sqrt(mean(v^2) + eps)
//
// One pass: a row of y and residual is read once into registers, both means of
// squares are formed there, and out and normed are written once.  Sums, norms
// and the sum with the residual are fp32; out and normed are each rounded once,
// and normed is formed from the unrounded fp32 out.
//
// Bound by HBM for many rows (16384 rows of 4096 bf16 with all parts: 95 us,
// 5.7 TB/s), by launch and load latency for few (one row of 2816: 4 us).  A row
// belongs to one wave (four rows a workgroup: sums by cross-lane moves alone, no
// barrier) or to a workgroup of 4 or 16 waves (one LDS exchange per sum).  Every
// element is loaded and stored by the same thread, and all loads of a row come
// before its first store, so out and normed may lie on y or residual.
//
// Every load of a row is issued before the first use: y, residual, weights and
// gate are independent, so a row pays one memory latency.
#include "moe_internal.h"

namespace moe {
namespace {

// A workgroup: four rows of one wave each, or one row of 4 or 16 waves.
template <int WAVES>
constexpr int kNormThreads = WAVES == 1 ? 256 : 64 * WAVES;

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
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += lds[w];
    }
    return v;
}

// kYF32, kSF32: y, and residual and out, are fp32.  kSlots: y is the fp32
// [T * k, H] output of the down matmul, already weighted; row t is the sum of
// its k slots in slot order (slots whose expert id is out of range were never
// written and are skipped).
template <int WAVES, int NV, int VEC, bool kYF32, bool kSF32, bool kSlots>
__global__ __launch_bounds__(kNormThreads<WAVES>) void moe_block_norm_kernel(NormArgs a) {
    constexpr int kRows = kNormThreads<WAVES> / 64 / WAVES, kStep = 64 * WAVES * VEC;
    __shared__ float lds[2][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + (WAVES == 1 ? wave : 0);
    if (t >= a.T) return;  // whole waves of one row: no barrier is left waiting
    const int c0 = VEC * (WAVES == 1 ? threadIdx.x & 63 : threadIdx.x);
    const int H = a.H;
    const bool wf32 = a.weight_f32, gf32 = a.gate_f32, channel = a.gate != nullptr && a.gate_stride_h != 0;
    constexpr int kYSize = kYF32 ? 4 : 2, kSSize = kSF32 ? 4 : 2;
    const int wsize = wf32 ? 4 : 2, gsize = gf32 ? 4 : 2;
    const Rsrc none = row_rsrc(nullptr, 0, 0, 0, 0);
    const Rsrc sy = row_rsrc(kSlots ? nullptr : a.y, a.y_stride * kYSize, t, H, kYSize);
    const Rsrc sr = row_rsrc(a.residual, a.residual_stride * kSSize, t, H, kSSize);
    const Rsrc sp = row_rsrc(a.post_weight, 0, 0, H, wsize), sn = row_rsrc(a.pre_weight, 0, 0, H, wsize);
    const Rsrc sg = row_rsrc(channel ? a.gate : nullptr, a.gate_stride_t * gsize, t, H, gsize);
    const Rsrc hp = wf32 ? sp : none, hn = wf32 ? sn : none, hg = gf32 ? sg : none;

    // 16 values a thread in 16-wave workgroups: 128 registers, so the gate and
    // the last weights are loaded once the others are done with
    constexpr bool kLate = VEC == 1 && NV >= 16;
    Raw<VEC> ry[NV], rr[NV], rp[NV], rn[NV], rg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * kStep;
        if constexpr (!kSlots) ry[i] = load_raw<VEC, kYF32>(sy, c);
        rr[i] = load_raw<VEC, kSF32>(sr, c);
        rp[i] = load_raw<VEC>(sp, hp, c, wf32);
        if constexpr (!kLate) rg[i] = load_raw<VEC>(sg, hg, c, gf32);
        if constexpr (!kLate) rn[i] = load_raw<VEC>(sn, hn, c, wf32);
    }
    float g0 = a.gate_scale;
    if (a.gate && !channel)
        g0 *= gf32 ? static_cast<const float*>(a.gate)[t * a.gate_stride_t]
                   : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t * a.gate_stride_t]);
    float z[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) z[i][v] = kSlots ? 0.f : value(ry[i], v, kYF32);
    if constexpr (kSlots) {
        // two slots at a time: their loads are in flight together
        for (int j0 = 0; j0 < a.k; j0 += 2) {
            Raw<VEC> r[2][NV];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t s = t * a.k + min(j0 + u, a.k - 1);
                const int32_t id = a.ids[s];
                const bool ok = j0 + u < a.k && id >= 0 && id < a.E;
                const Rsrc rs = row_rsrc(ok ? a.y : nullptr, 4 * static_cast<int64_t>(H), s, H, 4);
#pragma unroll
                for (int i = 0; i < NV; ++i) r[u][i] = load_raw<VEC, true>(rs, c0 + i * kStep);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) z[i][v] += value(r[u][i], v, true);
        }
    }

    if (a.post) {
        float ss = 0.f;  // values past H are zeros
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
    if constexpr (kLate) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rg[i] = load_raw<VEC>(sg, hg, c0 + i * kStep, gf32);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = c0 + i * kStep < H;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            z[i][v] *= channel ? g0 * value(rg[i], v, gf32) : g0;
            if (a.residual) z[i][v] = fmaf(a.residual_scale, value(rr[i], v, kSF32), z[i][v]);
            // past H the zeros may have met an infinite factor: left out
            ss = in ? fmaf(z[i][v], z[i][v], ss) : ss;
        }
    }
    if constexpr (kLate) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rn[i] = load_raw<VEC>(sn, hn, c0 + i * kStep, wf32);
    }
    const Rsrc so = row_rsrc(a.out, a.out_stride * kSSize, t, H, kSSize);
#pragma unroll
    for (int i = 0; i < NV; ++i) store_values(so, c0 + i * kStep, z[i], kSF32);
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

template <int WAVES, int NV, int VEC, bool kYF32, bool kSF32, bool kSlots = false>
hipError_t launch_one(const NormArgs& a, hipStream_t s) {
    constexpr int kRows = kNormThreads<WAVES> / 64 / WAVES;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) + kRows - 1) / kRows));
    hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, kYF32, kSF32, kSlots>), grid, dim3(kNormThreads<WAVES>), 0,
                       s, a);
    return hipGetLastError();
}
template <int WAVES, int NV, int VEC>
hipError_t launch_sized(const NormArgs& a, hipStream_t s) {
    if (a.y_f32)
        return a.stream_f32 ? launch_one<WAVES, NV, VEC, true, true>(a, s) : launch_one<WAVES, NV, VEC, true, false>(a, s);
    return a.stream_f32 ? launch_one<WAVES, NV, VEC, false, true>(a, s) : launch_one<WAVES, NV, VEC, false, false>(a, s);
}
template <int NV>
hipError_t launch_slots(const NormArgs& a, hipStream_t s) {
    return a.stream_f32 ? launch_one<4, NV, 8, true, true, true>(a, s) : launch_one<4, NV, 8, true, false, true>(a, s);
}

// Whether every row of a tensor starts on 16 bytes.
bool rows_aligned(const void* p, int64_t stride, bool f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (f32 ? 4 : 2) % 16 == 0;
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    const bool vec = a.H % 8 == 0 && rows_aligned(a.y, a.y_stride, a.y_f32) &&
                     rows_aligned(a.residual, a.residual_stride, a.stream_f32) &&
                     rows_aligned(a.out, a.out_stride, a.stream_f32) &&
                     rows_aligned(a.normed, a.normed_stride, a.normed_f32) && rows_aligned(a.post_weight, 0, false) &&
                     rows_aligned(a.pre_weight, 0, false) &&
                     (a.gate_stride_h == 0 || rows_aligned(a.gate, a.gate_stride_t, a.gate_f32));
    if (a.ids) {  // slots of the down matmul: H <= 4096
        if (!vec || a.H > 4096) return hipErrorInvalidValue;
        return a.H <= 2048 ? launch_slots<1>(a, s) : launch_slots<2>(a, s);
    }
    if (!vec) {
        if (a.H <= 1024) return launch_sized<4, 4, 1>(a, s);
        return a.H <= 4096 ? launch_sized<16, 4, 1>(a, s) : launch_sized<16, 16, 1>(a, s);
    }
    // One wave a row (no barrier) where a wave's two 16-byte pieces hold it and
    // there are rows enough for four waves a CU; else four waves, up to four
    // pieces each; else sixteen.  Measured, one against four waves: 16384 rows of
    // 256 12.8 | 32.8 us, of 1024 29.6 | 41.8 us, but 8192 of 2048 31.8 | 30.9 us and
    // 512 of 2048 5.8 | 4.4 us; four against sixteen: 4096 rows of 8192 54 | 82 us.
    if (a.T >= 1024 && a.H <= 512) return launch_sized<1, 1, 8>(a, s);
    if (a.T >= 1024 && a.H <= 1024) return launch_sized<1, 2, 8>(a, s);
    if (a.H <= 2048) return launch_sized<4, 1, 8>(a, s);
    if (a.H <= 4096) return launch_sized<4, 2, 8>(a, s);
    return a.H <= 8192 ? launch_sized<4, 4, 8>(a, s) : launch_sized<16, 2, 8>(a, s);
}

}  // namespace moe
