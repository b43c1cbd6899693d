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
#include "block_norm.h"

namespace moe {
namespace {

// A workgroup: four rows of one wave each, or one row of 4 or 16 waves.
template <int WAVES>
constexpr int kNormThreads = WAVES == 1 ? 256 : 64 * WAVES;

// kYF32, kSF32: y, and residual and out, are fp32.  kSlots: y is the fp32
// [T * k, H] output of the down matmul, already weighted; row t is the sum of
// its k slots in slot order (slots whose expert id is out of range were never
// written and are skipped).
template <int WAVES, int NV, int VEC, bool kYF32, bool kSF32, bool kSlots>
__global__ __launch_bounds__(kNormThreads<WAVES>) void moe_block_norm_kernel(NormArgs a) {
    using namespace norm;
    constexpr int kRows = kNormThreads<WAVES> / 64 / WAVES, kStep = 64 * WAVES * VEC;
    __shared__ float lds[2][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = static_cast<int64_t>(grid_index()) * kRows + (WAVES == 1 ? wave : 0);
    if (t >= a.T) return;  // whole waves of one row: no barrier is left waiting
    const int c0 = VEC * (WAVES == 1 ? threadIdx.x & 63 : threadIdx.x);
    Raw<VEC> ry[NV];
    if constexpr (!kSlots) {
        const Rsrc sy = row_rsrc(a.y, a.y_stride * (kYF32 ? 4 : 2), t, a.H, kYF32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < NV; ++i) ry[i] = load_raw<VEC, kYF32>(sy, c0 + i * kStep);
    }
    Row<WAVES, NV, VEC, kSF32> row;
    row.load(a, t, c0);
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
                const Rsrc rs = row_rsrc(ok ? a.y : nullptr, 4 * static_cast<int64_t>(a.H), s, a.H, 4);
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
    row.finish(a, t, c0, z, lds);
}

template <int WAVES, int NV, int VEC, bool kYF32, bool kSF32, bool kSlots = false>
hipError_t launch_one(const NormArgs& a, hipStream_t s) {
    constexpr int kRows = kNormThreads<WAVES> / 64 / WAVES;
    const dim3 grid = grid_of((static_cast<int64_t>(a.T) + kRows - 1) / kRows);
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
