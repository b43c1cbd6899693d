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
// Bound by HBM for many rows, by launch and load latency for few.  A row
// belongs to one wave (four rows a workgroup: sums by cross-lane moves alone, no
// barrier) or to a workgroup of four waves (one LDS exchange per sum); rows
// wider than a wave's registers hold, and batches too small to fill the GPU with
// one wave a row, take the workgroup.  Every element is loaded and stored by the
// same thread, and all loads of a row come before its first store, so out and
// normed may lie on y or residual.
//
// Every load of a row is issued before the first use: y, residual, weights and
// gate are independent, so a row pays one memory latency.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;

// VEC values of a tensor of type `f32` (else bf16), as loaded.
template <int VEC>
struct Raw {
    uint32_t u[VEC];
};
template <int VEC>
__device__ __forceinline__ void load_raw(Raw<VEC>& r, const void* p, int64_t at, bool f32) {
    if constexpr (VEC == 1) {
        r.u[0] = f32 ? static_cast<const uint32_t*>(p)[at] : static_cast<const uint16_t*>(p)[at];
    } else {
        static_assert(VEC == 8, "vector width");
        if (f32) {
            const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint32_t*>(p) + at);
            const u32x4 a = q[0], b = q[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.u[i] = a[i];
                r.u[4 + i] = b[i];
            }
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.u[i] = a[i];
        }
    }
}
template <int VEC>
__device__ __forceinline__ float value(const Raw<VEC>& r, int i, bool f32) {
    if (f32) return __uint_as_float(r.u[i]);
    if constexpr (VEC == 1) return __uint_as_float(r.u[0] << 16);
    return __uint_as_float(i & 1 ? r.u[i >> 1] & 0xFFFF0000u : r.u[i >> 1] << 16);
}
template <int VEC>
__device__ __forceinline__ void store_values(void* p, int64_t at, const float (&v)[VEC], bool f32) {
    if constexpr (VEC == 1) {
        if (f32)
            static_cast<float*>(p)[at] = v[0];
        else
            static_cast<uint16_t*>(p)[at] = f32_to_bf16(v[0]);
    } else {
        if (f32) {
            f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
            q[0] = f32x4{v[0], v[1], v[2], v[3]};
            q[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at) =
                u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        }
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
__global__ __launch_bounds__(kNormThreads) void moe_block_norm_kernel(NormArgs a) {
    constexpr int kRows = kNormThreads / 64 / WAVES, kStep = 64 * WAVES * VEC;
    __shared__ float lds[2][4];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0);
    if (t >= a.T) return;  // whole waves of one row: no barrier is left waiting
    const int c0 = VEC * (WAVES == 1 ? threadIdx.x & 63 : threadIdx.x);
    const int H = a.H;
    const bool wf32 = a.weight_f32, gf32 = a.gate_f32;

    Raw<VEC> ry[NV], rr[NV], rp[NV], rn[NV], rg[NV];
    float z[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * kStep;
        if (c >= H) continue;
        if constexpr (!kSlots) load_raw(ry[i], a.y, t * a.y_stride + c, kYF32);
        if (a.residual) load_raw(rr[i], a.residual, t * a.residual_stride + c, kSF32);
        if (a.post_weight) load_raw(rp[i], a.post_weight, c, wf32);
        if (a.gate && a.gate_stride_h) load_raw(rg[i], a.gate, t * a.gate_stride_t + c, gf32);
        if (a.pre_weight) load_raw(rn[i], a.pre_weight, c, wf32);
    }
    float g0 = a.gate_scale;
    if (a.gate && !a.gate_stride_h) {
        Raw<1> r;
        load_raw(r, a.gate, t * a.gate_stride_t, gf32);
        g0 *= value(r, 0, gf32);
    }
    if constexpr (kSlots) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[i][v] = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int64_t s = t * a.k + j;
            const int32_t id = a.ids[s];
            if (id < 0 || id >= a.E) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * kStep;
                if (c >= H) continue;
                Raw<VEC> r;
                load_raw(r, a.y, s * H + c, true);
#pragma unroll
                for (int v = 0; v < VEC; ++v) z[i][v] += value(r, v, true);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[i][v] = c0 + i * kStep < H ? value(ry[i], v, kYF32) : 0.f;
    }

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
            for (int v = 0; v < VEC; ++v) {
                z[i][v] *= rstd;
                if (a.post_weight && c0 + i * kStep < H) z[i][v] *= a.weight_offset + value(rp[i], v, wf32);
            }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * kStep;
        if (c >= H) continue;  // z stays 0 there
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float g = g0;
            if (a.gate && a.gate_stride_h) g *= value(rg[i], v, gf32);
            z[i][v] *= g;
            if (a.residual) z[i][v] = fmaf(a.residual_scale, value(rr[i], v, kSF32), z[i][v]);
            ss = fmaf(z[i][v], z[i][v], ss);
        }
    }
    if (a.out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * kStep;
            if (c < H) store_values(a.out, t * a.out_stride + c, z[i], kSF32);
        }
    }
    if (a.normed) {
        const float rstd = 1.f / sqrtf(row_sum<WAVES>(ss, lds[1]) / H + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * kStep;
            if (c >= H) continue;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                z[i][v] *= rstd;
                if (a.pre_weight) z[i][v] *= a.weight_offset + value(rn[i], v, wf32);
            }
            store_values(a.normed, t * a.normed_stride + c, z[i], a.normed_f32);
        }
    }
}

template <int WAVES, int NV, int VEC>
hipError_t launch_sized(const NormArgs& a, hipStream_t s) {
    constexpr int kRows = kNormThreads / 64 / WAVES;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) + kRows - 1) / kRows));
    const dim3 block(kNormThreads);
    if (a.ids) {
        if (a.stream_f32)
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, true, true, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, true, false, true>), grid, block, 0, s, a);
    } else if (a.y_f32) {
        if (a.stream_f32)
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, true, true, false>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, true, false, false>), grid, block, 0, s, a);
    } else {
        if (a.stream_f32)
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, false, true, false>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((moe_block_norm_kernel<WAVES, NV, VEC, false, false, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
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
    if (!vec) {
        if (a.H <= 1024) return launch_sized<4, 4, 1>(a, s);
        if (a.H <= 4096) return launch_sized<4, 16, 1>(a, s);
        return launch_sized<4, 64, 1>(a, s);
    }
    // one wave a row where that fills the GPU (four waves a SIMD and more)
    if (a.T >= 4096 && a.H <= 2048) return launch_sized<1, 4, 8>(a, s);
    if (a.H <= 2048) return launch_sized<4, 1, 8>(a, s);
    if (a.H <= 4096) return launch_sized<4, 2, 8>(a, s);
    if (a.H <= 8192) return launch_sized<4, 4, 8>(a, s);
    return launch_sized<4, 8, 8>(a, s);
}

}  // namespace moe
