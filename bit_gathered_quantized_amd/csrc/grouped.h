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
// kOnce: read once by the whole GPU (non-temporal).
template <bool kOnce = false>
__device__ __forceinline__ void copy16(Rsrc r, unsigned char* lds, uint32_t at, uint32_t step) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsByte*)lds, 16, at, step, 0, kOnce ? 2 : 0);
}
// Of a wave that only copies: all but its last N copies are in LDS.
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N < 64, "vmcnt");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}
// Barrier of all waves; each has waited for its own writes to LDS and copies before.
__device__ __forceinline__ void step_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ u32x4 read16(const unsigned char* lds, int at) {
    return *reinterpret_cast<const u32x4*>(lds + at);
}
__device__ __forceinline__ void store16(Rsrc r, u32x4 v, uint32_t at) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 0);
}
// Four rows of 16 columns (2-byte elements): lane 4 r + c of each 16 points at columns
// 4 c .. 4 c + 3 of row r and gets column l of the four rows, l its number in the 16.
__device__ __forceinline__ u32x2 read_turned(const unsigned char* lds, int at) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)((LdsByte*)const_cast<unsigned char*>(lds) + at));
    return __builtin_bit_cast(u32x2, v);
}

// For those reads rows of 2-byte elements lie in pieces of 32 bytes XORed with this: a half
// wave reads 32 bytes of rows 0 .. 3 and 8 .. 11 (or 4 on) at a time, each from banks of its own.
__device__ __forceinline__ int turn_key(int row) { return (row & 3) | (row >> 1 & 4); }

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

// Two products f, f + 1 as lanes hold them (lane (lr, q): columns 4 q .. 4 q + 3 of row lr)
// turned into 8 neighbouring columns a lane: those from 8 (q / 2) on of product f + q % 2.
__device__ __forceinline__ void neighbours(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// The same, rounded to bf16.
__device__ __forceinline__ u32x4 eight_bf16(f32x4 v, f32x4 u) {
    uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]), c = pack_bf16x2(u[0], u[1]), d = pack_bf16x2(u[2], u[3]);
    neighbours(a, c);
    neighbours(b, d);
    return u32x4{a, b, c, d};
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

// The smallest of the wave's values.
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
    auto with = [&](auto dpp, auto rows) {
        const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(-1, static_cast<int>(v), decltype(dpp)::value, decltype(rows)::value, 0xF, false));
        v = min(v, o);
    };
    using std::integral_constant;
    with(integral_constant<int, 0x111>(), integral_constant<int, 0xF>());  // row_shr:1
    with(integral_constant<int, 0x112>(), integral_constant<int, 0xF>());
    with(integral_constant<int, 0x114>(), integral_constant<int, 0xF>());
    with(integral_constant<int, 0x118>(), integral_constant<int, 0xF>());
    with(integral_constant<int, 0x142>(), integral_constant<int, 0xA>());  // row_bcast:15
    with(integral_constant<int, 0x143>(), integral_constant<int, 0xC>());  // row_bcast:31
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

constexpr int kUnit = 32;  // columns
struct Tile {
    int expert, row, rows;  // rows [row, row + rows) of x
    int n0, cols;           // columns [n0, n0 + cols)
    bool tall;              // the strip has more than half its rows
};

// What a workgroup computes, tile by tile.  A strip is up to BM rows of an expert; a tile is a
// strip by a block of its columns: at most BN, or BN / 2 in a tall strip (kTall; rows over
// BM / 2).  The number of strips is known on the device alone; `most` are the most that A rows over E
// experts can make, and offsets that make more leave the rest out.
//
// Tiles are dealt to the workgroups in turn.  Workgroups go to the XCDs in turn, and each XCD
// has a run of neighbouring tiles: those at work at a time share weights and rows in its L2.
// (An equal run of all columns for every workgroup ends the rounds evenly, but then nothing is
// shared in time: 16384 rows of 128 experts by 1408 x 2816, 268 | 377 us.)  A strip is cut into
// as many blocks of columns, of nearly equal width, as make the rounds cheapest.
template <int BM, int BN, bool kTall>
struct Share {
    static constexpr float kXPart = 0.5f, kFixed = 32.f;
    static constexpr int GM = 8;   // strips that run through all columns together
    const int32_t* offsets;
    const uint32_t* upto;          // LDS: tiles of experts 0 .. e
    int A, E, N;
    uint32_t per_strip;            // units
    uint32_t blocks;               // blocks of a strip (tall ones: twice as many, at most one a unit)
    uint32_t begin, end, step;

    __device__ __forceinline__ uint32_t blocks_of(bool tall) const { return tall ? min(2 * blocks, per_strip) : blocks; }

    // By all waves; ends with a barrier.
    __device__ __forceinline__ void init(const GroupedArgs& a, uint32_t* lds, uint32_t most) {
        offsets = a.offsets;
        upto = lds;
        A = a.A;
        E = a.E;
        N = a.N;
        per_strip = (N + kUnit - 1) / kUnit;
        const uint32_t groups = gridDim.x, of_xcd = groups >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
        const int lane = threadIdx.x & 63;
        auto rows_of = [&](int e) {
            int lo = 0, hi = e < E ? A : 0;
            if (offsets) expert_rows(offsets, e, E, A, lo, hi);
            return hi - lo;
        };
        auto sum = [&](int v) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(wave_scan(v), 63)); };
        // Every wave counts the strips: four loads in flight.
        uint32_t strips = 0, tall = 0;
        int rows[4];
        for (int base = 0; base < E; base += 256) {
            int n = 0, high = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) rows[i] = rows_of(base + 64 * i + lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                n += (rows[i] + BM - 1) / BM;
                high += rows[i] / BM + (rows[i] % BM > BM / 2);
            }
            strips += sum(n);
            if constexpr (kTall) tall += sum(high);
        }
        strips = min(strips, most);
        tall = min(tall, strips);
        // Every lane prices one number of blocks: rounds of tiles times a tile's mean price,
        // the rows it reads a stage, of w and of x (those mostly from L2: half), and a fixed part.
        const uint32_t least = (per_strip * kUnit + BN - 1) / BN, jump = (per_strip - least + 62) / 63;
        const uint32_t mine = min(least + lane * jump, per_strip);
        const float low = static_cast<float>(strips - tall), rows_low = min(static_cast<float>(kTall ? BM / 2 : BM), static_cast<float>(A) / strips);
        auto wide = [&](uint32_t n) { return kUnit * ceilf(static_cast<float>(per_strip) / n - 1e-3f); };
        const uint32_t mine_tall = min(2 * mine, per_strip);
        const float tiles = low * mine + static_cast<float>(tall) * mine_tall;
        const float all = low * mine * (wide(mine) + kXPart * rows_low + kFixed) +
                          (kTall ? static_cast<float>(tall) * mine_tall * (wide(mine_tall) + kXPart * 0.75f * BM + kFixed) : 0.f);
        float price = ceilf(tiles / groups - 1e-3f) * all / tiles;
        // the cheapest, of equal ones the fewest: a positive float's bits are in its order, and
        // the last six hold the lane
        blocks = min(least + (wave_min((__float_as_uint(price) & ~63u) | lane) & 63u) * max(jump, 1u), per_strip);
        const uint32_t limit = most * blocks_of(kTall);
        if (threadIdx.x < 64) {
            uint32_t before = 0;
            for (int base = 0; base < E; base += 256) {
                if (E > 256) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) rows[i] = rows_of(base + 64 * i + lane);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = base + 64 * i + lane, full = rows[i] / BM, rest = rows[i] % BM;
                    const int mine = full * blocks_of(kTall) + (rest ? blocks_of(kTall && rest > BM / 2) : 0);
                    // (limit < 2^24: no sum of a wave's passes 32 bits, whatever the offsets)
                    const uint32_t s = min(before + static_cast<uint32_t>(wave_scan(min(mine, static_cast<int>(limit)))), limit);
                    if (e < E) lds[e] = s;
                    before = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(s), 63));
                }
            }
        }
        __syncthreads();
        const uint32_t count = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(lds[E - 1])));
        const uint32_t share = (count + 7) / 8;
        begin = xcd * share + slot;
        end = min((xcd + 1) * share, count);
        step = of_xcd;
    }
    __device__ __forceinline__ uint32_t next(uint32_t at) const { return at + step; }
    // Tile `at` < end; all values are uniform.
    __device__ __forceinline__ Tile find(uint32_t at) const {
        const int lane = threadIdx.x & 63;
        int e = 0;
        for (int base = 0; base < E; base += 64) {
            const uint64_t hit = __builtin_amdgcn_ballot_w64(base + lane < E && upto[min(base + lane, E - 1)] > at);
            if (hit) {
                e = base + __builtin_ctzll(hit);
                break;
            }
        }
        const uint32_t local = at - (e ? __builtin_amdgcn_readfirstlane(static_cast<int>(upto[e - 1])) : 0);
        int lo = 0, hi = A;
        if (offsets) {  // through the scalar cache: a vector load would wait for the copies before it
            const auto* const o = (const __attribute__((address_space(4))) int32_t*)offsets;
            lo = min(max(o[e], 0), A);
            hi = min(max(o[e + 1], lo), A);
        }
        // strips of one height first: of a tall strip all, of the others the last
        const uint32_t all = static_cast<uint32_t>(hi - lo + BM - 1) / BM;
        const bool short_end = kTall && (hi - lo) % BM != 0 && (hi - lo) % BM <= BM / 2;
        const uint32_t alike = all - short_end, high = blocks_of(kTall);
        const bool at_end = short_end && local >= alike * high;
        const uint32_t mine = blocks_of(kTall && !at_end);
        uint32_t strip, n;
        if (at_end) {
            strip = all - 1;
            n = local - alike * high;
        } else {
            const uint32_t group = local / (GM * high), rest = local - group * (GM * high);
            const uint32_t together = min(alike - group * GM, static_cast<uint32_t>(GM));
            n = rest / together;
            strip = group * GM + rest - n * together;
        }
        const uint32_t narrow = per_strip / mine, wide = per_strip - narrow * mine;
        const uint32_t unit = n * narrow + min(n, wide), units = narrow + (n < wide);
        Tile t;
        t.expert = e;
        t.row = __builtin_amdgcn_readfirstlane(min(lo + static_cast<int>(strip) * BM, hi));
        t.rows = min(BM, hi - t.row);
        t.n0 = __builtin_amdgcn_readfirstlane(static_cast<int>(kUnit * unit));
        t.cols = min(__builtin_amdgcn_readfirstlane(static_cast<int>(kUnit * units)), N - t.n0);
        t.tall = kTall && t.rows > BM / 2;
        return t;
    }
};

// The most strips of bm rows that A rows over E experts make.
inline int64_t most_strips(const GroupedArgs& a, int64_t bm) {
    return a.offsets ? a.A / bm + (a.A < a.E ? a.A : a.E) : (a.A + bm - 1) / bm;
}

}  // namespace grouped
}  // namespace
}  // namespace moe
