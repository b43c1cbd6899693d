// Device pieces shared by the products grouped by expert.
#pragma once

#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

namespace grouped {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) unsigned char LdsByte;

__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t n) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(n), 0x00020000);
}
// Past every resource below (their sizes stay under it): reads zeros.
constexpr uint32_t kOutside = 0xFFFFFFF0u;

// 16 bytes a lane from r at `at` + `step` (uniform) to lds + 16 * lane, lds uniform.
__device__ __forceinline__ void copy16(Rsrc r, unsigned char* lds, uint32_t at, uint32_t step) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsByte*)lds, 16, at, step, 0, 0);
}
// The wave's copies but the last n are in LDS; then those of all waves, and every
// wave is done with what it read before.
template <int N>
__device__ __forceinline__ void copies_done() {
    static_assert(N < 64, "vmcnt");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);  // the other counters are not waited for
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ u32x4 read16(const unsigned char* lds, int at) {
    return *reinterpret_cast<const u32x4*>(lds + at);
}
// Four rows of 16 columns (2-byte elements): lane 4 r + c of each 16 points at columns
// 4 c .. 4 c + 3 of row r and gets column l of the four rows, l its number in the 16.
__device__ __forceinline__ u32x2 read_turned(const unsigned char* lds, int at) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)((LdsByte*)const_cast<unsigned char*>(lds) + at));
    return __builtin_bit_cast(u32x2, v);
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}
// 128 products of 4-bit values a lane quarter's 32 at a time; sa and sb hold the scale
// byte of the lane's 32 values at byte SA, SB.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, SA, sa, SB, sb);
}

// 2^(b - 127) of a scale byte, NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    const uint32_t v = b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23;
    return __uint_as_float(v);
}
// The 8 codes of a word under their scale, as bf16 (exact).
__device__ __forceinline__ u32x4 mx_as_bf16(uint32_t codes, float unit) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 3))};
}

// ------------------------------------------------------- tiles of the experts
// Rows [lo, hi) of expert e, none for e >= E; offsets outside [0, A] are cut off, so
// whatever the array holds no row outside x and out is touched.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int E, int A, int& lo, int& hi) {
    const int at = min(e, E - 1);
    const int first = offsets[at], last = offsets[at + 1];  // read by all lanes: no branch
    lo = min(max(first, 0), A);
    hi = min(max(e < E ? last : 0, lo), A);
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}

struct Tile {
    int expert, row, rows;  // rows [row, row + rows) of x, 1 <= rows
    int m, tiles_m;         // number of this block of rows in its expert, and of how many
    int n;                  // block of columns
};

// Workgroup `index` takes one tile of BM rows by one of `across` blocks of columns.  The
// grid covers the most tiles that A rows over E experts can make (`most` blocks of rows);
// their true number is known here alone, and offsets that make more leave the rest out.
// Workgroups go to the XCDs in turn, so each XCD gets a run of neighbouring tiles: those
// of an expert share its weights in one L2.  In an expert, GM blocks of rows at a time
// run through all columns.  All values are uniform; most * across < 2^31.
template <int BM, int GM>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int A, int E, uint32_t most, uint32_t across,
                                          uint32_t index, Tile& t) {
    const int lane = threadIdx.x & 63;
    constexpr int kLoads = 4;  // experts a lane holds at a time
    auto place = [&](uint32_t local, int expert, int begin, int end) {
        t.expert = expert;
        t.tiles_m = (end - begin + BM - 1) / BM;
        const uint32_t block = local / (GM * across), rest = local - block * (GM * across);
        const uint32_t high = min(static_cast<uint32_t>(t.tiles_m) - block * GM, static_cast<uint32_t>(GM));
        t.m = block * GM + rest % high;
        t.n = rest / high;
        t.row = begin + t.m * BM;
        t.rows = min(BM, end - t.row);
    };
    uint32_t total = 0;
    for (int base = 0; offsets && base < E; base += 64 * kLoads) {
        int v = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int lo, hi;
            expert_rows(offsets, base + 64 * i + lane, E, A, lo, hi);
            v += (hi - lo + BM - 1) / BM;
        }
        total = min(total + static_cast<uint32_t>(__builtin_amdgcn_readlane(wave_scan(v), 63)), most);
    }
    if (!offsets) total = most;
    const uint32_t tiles = total * across, share = (tiles + 7) / 8;
    const uint32_t at = (index & 7) * share + (index >> 3);
    if ((index >> 3) >= share || at >= tiles) return false;
    if (!offsets) {
        place(at, 0, 0, A);
        return true;
    }
    const uint32_t want = at / across;
    uint32_t before = 0;
    for (int base = 0; base < E; base += 64 * kLoads) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int lo, hi;
            expert_rows(offsets, base + 64 * i + lane, E, A, lo, hi);
            const int mine = (hi - lo + BM - 1) / BM;
            const uint32_t upto = before + static_cast<uint32_t>(wave_scan(mine));
            const uint64_t hit = __builtin_amdgcn_ballot_w64(upto > want);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                const uint32_t first = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto) - mine, l));
                place(at - first * across, base + 64 * i + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(hi, l));
                return true;
            }
            before = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), 63));
        }
    }
    return false;
}

// The most row blocks of bm rows that A rows over E experts make.
inline int64_t grid_tiles(const GroupedArgs& a, int64_t bm) {
    return a.offsets ? a.A / bm + (a.A < a.E ? a.A : a.E) : (a.A + bm - 1) / bm;
}

}  // namespace grouped
}  // namespace
}  // namespace moe
