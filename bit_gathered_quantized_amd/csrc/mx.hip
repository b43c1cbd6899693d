// Microscaled 4-bit values: blocks of 32 along a row under a scale 2^s, codes e2m1.
//
//   s = floor(log2(max |v|)) - 2  at least -127,  code = v / 2^s to nearest, ties to even
//
// The exponent field of max |v| is floor(log2) + 127 (0 where s is -127 anyway, 255 for
// NaN and infinity), so the scale byte is that field minus 2.  The division by 2^s, the
// rounding and the cut at 6 are the conversion instruction's.  Four neighbouring lanes
// hold a block, 8 values each.  Bound by memory: one pass, 16-byte accesses on the
// values (16384 rows of 2 x 704 bf16 values with a GELU: 52 MB in 10 us, 5.2 TB/s; 2048 x 2816:
// 15 MB in 4.7 us, of which launch and latency take over half).
#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

constexpr int kThreads = 256;

// The largest of four neighbouring lanes.
__device__ __forceinline__ uint32_t max_of_four(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true)));  // lanes 1 0 3 2
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true)));  // lanes 2 3 0 1
}

template <bool kF32>
__device__ __forceinline__ void load8(const unsigned char* p, float (&v)[8]) {
    if constexpr (kF32) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
}

// Eighths of blocks ("units") in row order, one a thread; units < 2^31, a row's number is
// the high half of unit * magic, shifted.
struct Units {
    uint32_t count, per_row, magic, shift;
};

template <bool kF32, int GLU>
__global__ __launch_bounds__(kThreads) void moe_mx_quantize_kernel(MxArgs a, Units u) {
    const uint32_t unit = grid_index() * kThreads + threadIdx.x;
    if (unit >= u.count) return;  // whole blocks: the count is a multiple of 4
    constexpr int kSize = kF32 ? 4 : 2;
    const uint32_t row = __umulhi(unit, u.magic) >> u.shift, at = unit - row * u.per_row;
    const unsigned char* const p = static_cast<const unsigned char*>(a.values) + row * a.stride + 8 * kSize * static_cast<int64_t>(at);
    float v[8];
    load8<kF32>(p, v);
    if constexpr (GLU != 0) {
        float w[8];
        load8<kF32>(p + kSize * static_cast<int64_t>(a.K), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (GLU == 1 ? gelu_tanh(v[i]) : silu(v[i])) * w[i];
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t field = max_of_four(top) >> 23;
    const uint32_t byte = field == 255 ? 255u : field < 2 ? 0u : field - 2;
    const float scale = mx_scale(field == 255 ? 127u : byte);
    uint32_t codes = 0;
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[0], v[1], scale, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2], v[3], scale, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4], v[5], scale, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6], v[7], scale, 3);
    *reinterpret_cast<uint32_t*>(a.codes + 4 * static_cast<size_t>(unit)) = field == 255 ? 0u : codes;
    if ((unit & 3) == 0) a.scales[unit >> 2] = static_cast<uint8_t>(byte);
}

template <bool kF32>
__global__ __launch_bounds__(kThreads) void moe_mx_dequantize_kernel(MxArgs a, Units u) {
    const uint32_t unit = grid_index() * kThreads + threadIdx.x;
    if (unit >= u.count) return;
    const uint32_t row = __umulhi(unit, u.magic) >> u.shift, at = unit - row * u.per_row;
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(a.codes + 4 * static_cast<size_t>(unit));
    const u32x4 v = mx_as_bf16(codes, mx_scale(a.scales[unit >> 2]));
    unsigned char* const p = static_cast<unsigned char*>(a.values) + row * a.stride + (kF32 ? 32 : 16) * static_cast<int64_t>(at);
    if constexpr (kF32) {
        u32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            lo[2 * i] = v[i] << 16;
            lo[2 * i + 1] = v[i] & 0xFFFF0000u;
            hi[2 * i] = v[2 + i] << 16;
            hi[2 * i + 1] = v[2 + i] & 0xFFFF0000u;
        }
        *reinterpret_cast<u32x4*>(p) = lo;
        *reinterpret_cast<u32x4*>(p + 16) = hi;
    } else {
        *reinterpret_cast<u32x4*>(p) = v;
    }
}

// units < 2^31 and per_row >= 4: with 2^(l - 1) < per_row <= 2^l and magic =
// floor(2^(31 + l) / per_row) + 1 the quotient is exact.
Units units_of(const MxArgs& a) {
    Units u;
    u.per_row = static_cast<uint32_t>(a.K / 8);
    u.count = static_cast<uint32_t>(a.R * u.per_row);
    int l = 0;
    while ((1u << l) < u.per_row) ++l;
    u.magic = static_cast<uint32_t>((uint64_t{1} << (31 + l)) / u.per_row + 1);
    u.shift = static_cast<uint32_t>(l - 1);
    return u;
}

}  // namespace

hipError_t launch_mx_quantize(const MxArgs& a, hipStream_t s) {
    const Units u = units_of(a);
    const dim3 grid = grid_of((static_cast<int64_t>(u.count) + kThreads - 1) / kThreads), block(kThreads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, a, u); };
    if (a.glu == 0)
        a.f32 ? go(moe_mx_quantize_kernel<true, 0>) : go(moe_mx_quantize_kernel<false, 0>);
    else if (a.glu == 1)
        a.f32 ? go(moe_mx_quantize_kernel<true, 1>) : go(moe_mx_quantize_kernel<false, 1>);
    else
        a.f32 ? go(moe_mx_quantize_kernel<true, 2>) : go(moe_mx_quantize_kernel<false, 2>);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxArgs& a, hipStream_t s) {
    const Units u = units_of(a);
    const dim3 grid = grid_of((static_cast<int64_t>(u.count) + kThreads - 1) / kThreads), block(kThreads);
    if (a.f32)
        hipLaunchKernelGGL((moe_mx_dequantize_kernel<true>), grid, block, 0, s, a, u);
    else
        hipLaunchKernelGGL((moe_mx_dequantize_kernel<false>), grid, block, 0, s, a, u);
    return hipGetLastError();
}

}  // namespace moe
