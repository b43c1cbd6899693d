// Grouped products: tiles of 128 rows by 256 columns, or 256 by 128 in strips of more than
// 128 rows, so that an expert of up to 256 rows reads its weights once.
//
// One workgroup a CU takes the tiles of its share in turn.  Four of its waves only copy,
// D - 1 stages ahead, through D buffers in LDS; eight multiply and store.  A stage is a step:
// the copiers wait for its copies, all waves meet, the copiers start the stage D - 1 steps
// ahead in the buffer of the last step, and the others multiply.  So neither a tile's end nor the
// search for the next tile holds up the copies.
//
//   kRows    bf16 x, bf16 w [E, N, K]:  a stage is 64 of K
//   kCols    bf16 x, bf16 w [E, K, N]:  the same, w turned by the reads
//   kMx      both microscaled:          256 of K
//   kBf16Mx  bf16 x, microscaled w:     128 of K; no strips of 256 rows
//
// For many rows an expert there are tiles of 256 x 256 (kLow = 256), a wave's part 64 by 128, with two
// buffers: a third less to copy and a quarter less to read from LDS for a product.
//
// For few rows an expert strips have kLow = 32 rows, so that the room of the rows goes to one more
// buffer, or to stages of 256 of K (kBf16Mx).
//
// What bounds it: with many experts reading w (4096 rows of 128 experts by 2816 x 1408, w turned,
// 180 us for 1.05 GB) and, from 32 rows an expert on, the way from L2 to LDS, since each block of columns
// brings the strip's rows again (16384 rows of 128 experts by 1408 x 2816: 255 us for 1.15 GB of
// memory and 1.9 GB of copies; both sides microscaled 88 us); with few experts the rate at which LDS
// feeds the products (16381 rows of 8 experts by 2816 x 4096: 337 us, 1120 TFLOP/s; microscaled 119 us,
// 3180 TFLOP/s; a stage's reads and copies take as many cycles of LDS as its products on the matrix units).
//
// A buffer holds rows of 128 bytes of K, those of x first, in pieces of 16 bytes XORed
// with the row's number so that neither the copies nor the reads meet a bank twice (kCols: w
// as 64 rows of the tile's columns in pieces of 32 bytes; kBf16Mx: rows of 256 bytes of x
// and 64 of w, or of 512 and 128).
#pragma once

#include "grouped.h"

namespace moe {
namespace {

using namespace grouped;

enum class Form { kRows, kCols, kMx, kBf16Mx };

// LDS row r of w holds this column of the tile, so that a lane ends up with 8
// neighbouring columns of two products.
__device__ __forceinline__ int column_of(int r) {
    const int f = r >> 4, i = r & 15;
    return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
}

// SB bytes (4 or 8) of a row of `size` scale bytes from `at` on, at < size, zeros past its end: as
// they lie (take_scales) and in place (place_scales).  At the row's end the last SB bytes are read,
// to be moved down.  at and size are uniform; rows start on any byte.  kShort: size < SB.
template <int SB, bool kShort>
__device__ __forceinline__ u32x2 take_scales(const uint8_t* p, int at, int size) {
    u32x2 v = {0, 0};
    if constexpr (kShort) {
        for (int i = 0; at + i < size; ++i) {
            const uint32_t b = static_cast<uint32_t>(p[at + i]) << (8 * (i & 3));
            v[0] |= i < 4 ? b : 0;
            v[1] |= i < 4 ? 0 : b;
        }
    } else {
        __builtin_memcpy(&v, p + min(at, size - SB), SB);
    }
    return v;
}
template <int SB, bool kShort>
__device__ __forceinline__ u32x2 place_scales(u32x2 v, int at, int size) {
    if constexpr (kShort) return v;
    const int down = 8 * (at - min(at, size - SB));
    return SB == 8 ? __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, v) >> down) : u32x2{v[0] >> down, 0};
}

// A wave's results: rows m_at .. and columns n_at .. of a tile, acc[f][m] the product of
// columns 16 f .. and rows 16 m ...
template <int FM, int FN, bool kTurn, bool kF32>
__device__ __forceinline__ void store_tile(const GroupedArgs& a, const Tile& t, const f32x4 (&acc)[FN][FM], int m_at, int n_at,
                                           int lr, int q) {
    constexpr int kOut = kF32 ? 4 : 2;
    // Of tiles of 256 x 256 the compiler would keep the addresses through the products, in scratch memory (116 to 240
    // bytes a lane against 36 to 56; for fp32 up to ten reads and writes of it in every stage, now one at most).  16381 rows of 8 experts by 2816 x
    // 4096, kept | made here: bf16 out 334 | 332 us, w turned 329 | 327, both microscaled 121 | 119; fp32 out 363 |
    // 354, 450 | 355, 191 | 141.
    if constexpr (FN == 8) asm("" : "+v"(lr), "+v"(q));
    const Rsrc r = make_rsrc(static_cast<unsigned char*>(a.out) + t.row * a.out_stride + static_cast<int64_t>(kOut) * t.n0,
                             static_cast<uint32_t>(max(t.rows - 1, 0) * a.out_stride) + kOut * t.cols);
#pragma unroll
    for (int m = 0; m < FM; ++m) {
        const int row = m_at + 16 * m + lr;
        const uint32_t at = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.out_stride);
#pragma unroll
        for (int f = 0; f < FN; f += 2) {
            const f32x4 v = acc[f][m], u = acc[f + 1][m];
            const int c = n_at + 16 * f;
            auto place = [&](int col) { return row < t.rows && col < t.cols ? at + kOut * col : kOutside; };
            // lane (lr, q) holds columns 4 q .. + 3 of row lr of either product; of w [E, N, K]
            // they are neighbours, 8 q .. and 8 q + 4 ..
            if constexpr (kF32) {
                const int col = kTurn ? c + 4 * q : c + 8 * q;
                store16(r, __builtin_bit_cast(u32x4, v), place(col));
                store16(r, __builtin_bit_cast(u32x4, u), place(col + (kTurn ? 16 : 4)));
            } else if constexpr (kTurn) {
                store16(r, eight_bf16(v, u), place(c + 16 * (q & 1) + 8 * (q >> 1)));
            } else {
                store16(r, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])},
                        place(c + 8 * q));
            }
        }
    }
}

constexpr int kCopiers = 4, kMultipliers = 8;

// kOnce: w is read once (non-temporal loads).  kShort: K shorter than a stage.
template <Form F, int kLow, bool kOnce, bool kF32, bool kShort>
__global__ __launch_bounds__(64 * (kCopiers + kMultipliers)) void moe_grouped_product(GroupedArgs a, uint32_t most) {
    constexpr bool kMxX = F == Form::kMx, kMixed = F == Form::kBf16Mx, kMxW = kMxX || kMixed, kTurn = F == Form::kCols;
    constexpr bool kLong = kMixed && kLow < 128, kTall = kLow == 128 && !kMixed, kBig = kLow == 256;
    constexpr int kWide = 256;                                     // columns of the tile of a short strip
    constexpr int BM = kTall ? 2 * kLow : kLow, BN = kWide, D = kBig ? 2 : kLow == 128 || kMixed ? 3 : 4;
    constexpr int kStage = kMxX || kLong ? 256 : kMixed ? 128 : 64;  // of K
    constexpr int kXRow = kMxX ? 128 : 2 * kStage, kWRow = kMxW ? kStage / 2 : 2 * kStage;  // bytes of a row
    constexpr int kBuffer = kLow * kXRow + kWide * kWRow, kJobs = kBuffer / 1024 / kCopiers;
    constexpr int kXJobs = kLow * kXRow / 1024 / kCopiers, kXTall = kTall ? 2 * kXJobs : kXJobs;  // of them x's, in a tall strip
    constexpr int kSB = kStage / 32, kSRows = !kMxW ? 0 : kMxX ? kLow + kWide : kWide;  // scale bytes of a row and stage
    constexpr int kSJobs = (kSRows + 64 * kCopiers - 1) / (64 * kCopiers), kSBuffer = kMxW ? kSRows * kSB : 16;
    constexpr int FM = kLow == 32 ? 2 : 4, FN = kBig ? 8 : kLow == 128 ? 4 : 2, kColumns = 16 * FN;  // a wave's part: up to 64 rows by kColumns
    static_assert(kXJobs * kCopiers * 1024 == kLow * kXRow && kJobs * kCopiers * 1024 == kBuffer, "copies");
    static_assert(!kTall || (kXRow == 128 && kWRow == 128 && kWide == 2 * kLow), "a buffer holds either tile");
    __shared__ __align__(16) unsigned char buffers[D][kBuffer];
    __shared__ __align__(16) unsigned char scales[D][kSBuffer];
    __shared__ uint32_t upto[MOE_MAX_EXPERTS];
    // the next tiles, from the copiers to the others: row, rows, n0, cols, flags (1 tall, 2 another follows)
    constexpr int kTells = 8;  // more than the D + 1 tiles from the one that is read to the one that is aimed at
    __shared__ __align__(16) int tell[kTells][8];

    Share<BM, BN, kTall> share;
    share.init(a, upto, most);
    if (share.begin >= share.end) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int stages = (a.K + kStage - 1) / kStage;

    if (wave >= kMultipliers) {
        const int w = wave - kMultipliers, blocks = a.K / 32;
        const uint32_t xbytes = kMxX ? a.K / 2 : 2u * a.K, wbytes = kMxW ? a.K / 2 : 2u * a.K;
        const int64_t xs = kMxX ? static_cast<int64_t>(xbytes) : a.x_stride;
        const int64_t ws = kMxW ? static_cast<int64_t>(wbytes) : a.w_stride;
        uint32_t ahead = share.begin, steps = 0;  // steps: those whose copies are under way
        int stage = 0, buffer = 0, told = 0;
        bool tall = false;
        Rsrc rx, rw;
        const unsigned char* pw = nullptr;
        uint32_t wsize = 0, at[kJobs];
        int wrow0 = 0, wrow_step = 0;  // kCols: the row of a stage that this lane copies in w's first job, and from one job to the next
        const uint8_t* ps[kSJobs ? kSJobs : 1] = {};
        // the place in a row of the 16 bytes that this lane copies: the same in every job
        const uint32_t xpiece = 16u * (kXRow == 128   ? (lane & 7) ^ (lane >> 3)
                                       : kXRow == 256 ? lr ^ ((4 * w + q) & 15)
                                                      : (lane & 31) ^ ((2 * w + (lane >> 5)) & 7));
        const uint32_t wpiece = 16u * (kWRow == 128 ? (lane & 7) ^ (lane >> 3) : (lane & 3) ^ (lane >> 3 & 3));
        auto aim = [&] {  // at the tile ahead
            const Tile t = share.find(ahead);
            tall = t.tall;
            if (w == 0 && lane == 0) {
                int* const to = tell[told];
                to[0] = t.row;
                to[1] = t.rows;
                to[2] = t.n0;
                to[3] = t.cols;
                to[4] = (t.tall ? 1 : 0) | (share.next(ahead) < share.end ? 2 : 0);
            }
            told = (told + 1) & (kTells - 1);
            rx = make_rsrc(static_cast<const unsigned char*>(a.x) + t.row * xs, static_cast<uint32_t>((t.rows - 1) * xs) + xbytes);
            // rows and columns past the tile's are not read
            auto x_at = [&](int j) {
                const int r = 1024 / kXRow * (j * kCopiers + w) + lane / (kXRow / 16);
                return r < t.rows ? static_cast<uint32_t>(r) * static_cast<uint32_t>(xs) + xpiece : kOutside;
            };
            const int w_jobs = kTall && tall ? kXTall : kXJobs;  // the first of w's
            auto w_at = [&](int j) {
                const int job = (j - w_jobs) * kCopiers + w;
                if constexpr (kTurn) {
                    const int pieces = tall ? kLow / 8 : kWide / 8, r = job * (64 / pieces) + lane / pieces, p = lane % pieces;
                    const int col = 32 * ((p >> 1) ^ turn_key(r)) + 16 * (p & 1);
                    return col < 2 * t.cols ? static_cast<uint32_t>(r) * static_cast<uint32_t>(ws) + col : kOutside;
                } else {
                    const int n = column_of(1024 / kWRow * job + lane / (kWRow / 16));
                    return n < t.cols ? static_cast<uint32_t>(n) * static_cast<uint32_t>(ws) + wpiece : kOutside;
                }
            };
            if constexpr (kTurn) {
                pw = static_cast<const unsigned char*>(a.w) + t.expert * a.w_expert + 2 * static_cast<int64_t>(t.n0);
                wsize = static_cast<uint32_t>(2 * t.cols);
                const int pieces = tall ? kLow / 8 : kWide / 8;
                wrow0 = w * (64 / pieces) + lane / pieces;
                wrow_step = kCopiers * (64 / pieces);
            } else {
                const int64_t we = kMxW ? ws * a.N : a.w_expert;
                rw = make_rsrc(static_cast<const unsigned char*>(a.w) + t.expert * we + t.n0 * ws,
                               static_cast<uint32_t>((t.cols - 1) * ws) + wbytes);
            }
#pragma unroll
            for (int j = 0; j < kJobs; ++j) at[j] = j < kXJobs ? x_at(j) : j >= kXTall ? w_at(j) : tall ? x_at(j) : w_at(j);
            const int x_rows = kMxX ? (tall ? kWide : kLow) : 0;
#pragma unroll
            for (int j = 0; j < kSJobs; ++j) {
                const int i = min(j * 64 * kCopiers + static_cast<int>(threadIdx.x) - 64 * kMultipliers, kSRows - 1), r = i - x_rows;
                ps[j] = r < 0 ? a.xs + static_cast<int64_t>(t.row + min(i, t.rows - 1)) * blocks
                              : a.ws + (static_cast<int64_t>(t.expert) * a.N + t.n0 + min(column_of(r), t.cols - 1)) * blocks;
            }
        };
        u32x2 fresh[kSJobs ? kSJobs : 1] = {};  // scales on their way
        int fresh_at = 0, fresh_to = -1;
        auto issue = [&] {
            if constexpr (kMxW) {
                fresh_at = kSB * stage;
                fresh_to = buffer;
#pragma unroll
                for (int j = 0; j < kSJobs; ++j) fresh[j] = take_scales<kSB, kShort>(ps[j], fresh_at, blocks);
                __builtin_amdgcn_sched_barrier(0);  // before the copies: their count says that these are there
            }
            const uint32_t xk = static_cast<uint32_t>(kXRow) * stage, wk = static_cast<uint32_t>(kWRow) * stage;
            const bool xin = xk + xpiece < xbytes, win = wk + wpiece < wbytes;
            unsigned char* const to = buffers[buffer] + 1024 * w;
            int rows = 0;
            if constexpr (kTurn) {  // the stage's rows of w, a resource of its own: K rows may pass 32 bits
                rows = min(kStage, a.K - kStage * stage);
                rw = make_rsrc(pw + static_cast<int64_t>(kStage) * stage * ws, static_cast<uint32_t>((rows - 1) * ws) + wsize);
            }
            auto copy_x = [&](int j) { copy16(rx, to + 1024 * kCopiers * j, xin ? at[j] : kOutside, xk); };
            auto copy_w = [&](int j, int first) {
                if constexpr (kTurn)
                    copy16<kOnce>(rw, to + 1024 * kCopiers * j, wrow0 + wrow_step * (j - first) < rows ? at[j] : kOutside, 0);
                else
                    copy16<kOnce>(rw, to + 1024 * kCopiers * j, win ? at[j] : kOutside, wk);
            };
#pragma unroll
            for (int j = 0; j < kXJobs; ++j) copy_x(j);
            if (kTall && tall) {
#pragma unroll
                for (int j = kXJobs; j < kXTall; ++j) copy_x(j);
#pragma unroll
                for (int j = kXTall; j < kJobs; ++j) copy_w(j, kXTall);
            } else {
#pragma unroll
                for (int j = kXJobs; j < kJobs; ++j) copy_w(j, kXJobs);
            }
            buffer = buffer + 1 == D ? 0 : buffer + 1;
            ++steps;
            if (++stage == stages) {
                stage = 0;
                ahead = share.next(ahead);
                if (ahead < share.end) aim();
            }
        };
        auto put_scales = [&] {  // those of the last stage issued
            if constexpr (kMxW) {
                if (fresh_to < 0) return;
#pragma unroll
                for (int j = 0; j < kSJobs; ++j) {
                    const int i = j * 64 * kCopiers + static_cast<int>(threadIdx.x) - 64 * kMultipliers;
                    const u32x2 v = place_scales<kSB, kShort>(fresh[j], fresh_at, blocks);
                    if (i < kSRows) {
                        if constexpr (kSB == 8)
                            *reinterpret_cast<u32x2*>(scales[fresh_to] + 8 * i) = v;
                        else
                            *reinterpret_cast<uint32_t*>(scales[fresh_to] + 4 * i) = v[0];
                    }
                }
                fresh_to = -1;
            }
        };
        aim();
        for (int i = 0; i < D - 1 && ahead < share.end; ++i) {
            issue();
            if (i < D - 2) put_scales();
        }
        for (uint32_t i = 0; i < steps; ++i) {
            if (ahead < share.end)
                wait_copies<(D - 2) * kJobs>();
            else
                wait_copies<0>();
            put_scales();
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): scales and tile are in LDS
            step_barrier();
            if (ahead < share.end) issue();
        }
        return;
    }

    f32x4 acc[FN][FM];
    int buffer = 0, told = 0;
    for (bool more = true; more;) {
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int m = 0; m < FM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        step_barrier();
        Tile t;
        t.row = __builtin_amdgcn_readfirstlane(tell[told][0]);
        t.rows = __builtin_amdgcn_readfirstlane(tell[told][1]);
        t.n0 = __builtin_amdgcn_readfirstlane(tell[told][2]);
        t.cols = __builtin_amdgcn_readfirstlane(tell[told][3]);
        const int flags = __builtin_amdgcn_readfirstlane(tell[told][4]);
        told = (told + 1) & (kTells - 1);
        more = flags & 2;
        const bool tall = kTall && (flags & 1);
        const int wm = kLow < 128 ? 0 : tall || kBig ? wave >> 1 : wave >> 2, wn = kLow < 128 ? wave : tall || kBig ? wave & 1 : wave & 3;
        const int x_rows = tall ? kWide : kLow, columns = tall ? kLow : kWide;
        const int x_from = 64 * wm * kXRow, w_from = x_rows * kXRow + (kTurn ? 0 : kColumns * wn * kWRow);
        int turned[kTurn ? FN : 1];  // of columns 16 f of row 8 q + lr / 4
        if constexpr (kTurn) {
            const int r = 8 * q + (lr >> 2);
#pragma unroll
            for (int f = 0; f < FN; ++f) turned[f] = w_from + r * 2 * columns + 32 * ((wn * FN + f) ^ turn_key(r)) + 8 * (lr & 3);
        }
        auto multiply = [&](auto rows_16, const unsigned char* b, const unsigned char* sc) {
            constexpr int M = decltype(rows_16)::value;
            if constexpr (kMixed) {
                // lane quarter q holds one block of 128 of K (kLong: one of each 128): its
                // 16 bytes of codes become four operands, word i against x's values 8 i .. + 7
                // of the block (codes under their scale are exact in bf16)
#pragma unroll
                for (int s = 0; s < kStage / 128; ++s) {
                    const int block = kLong ? 2 * q + s : q;
                    u32x4 codes[FN];
                    float unit[FN];
#pragma unroll
                    for (int f = 0; f < FN; ++f) {
                        const int row = 16 * f + lr;
                        codes[f] = read16(b, w_from + kWRow * row + 16 * (block ^ (kLong ? lr & 7 : lr >> 1 & 3)));
                        unit[f] = mx_scale(sc[kSB * (kColumns * wn + row) + block]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u32x4 xf[M];
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            xf[m] = read16(b, x_from + kXRow * (16 * m + lr) + 16 * ((4 * block + i) ^ (kLong ? lr & 7 : lr)));
#pragma unroll
                        for (int f = 0; f < FN; ++f) {
                            const u32x4 w = mx_as_bf16(codes[f][i], unit[f]);
#pragma unroll
                            for (int m = 0; m < M; ++m) acc[f][m] = mfma_bf16(w, xf[m], acc[f][m]);
                        }
                    }
                }
                return;
            }
            uint32_t sx[kMxX ? M : 1], sw[kMxX ? FN : 1];
            if constexpr (kMxX) {  // blocks 2 q and 2 q + 1 of the stage
                const int x_at = 8 * (64 * wm + lr) + 2 * q, w_at = 8 * (x_rows + kColumns * wn + lr) + 2 * q;
#pragma unroll
                for (int m = 0; m < M; ++m) sx[m] = *reinterpret_cast<const uint16_t*>(sc + (x_at + 128 * m));
#pragma unroll
                for (int f = 0; f < FN; ++f) sw[f] = *reinterpret_cast<const uint16_t*>(sc + (w_at + 128 * f));
            }
            auto half = [&](auto which) {
                constexpr int S = decltype(which)::value;
                const int piece = 128 * lr + 16 * ((kMxX ? 2 * q + S : 4 * S + q) ^ (lr & 7));
                if constexpr (kBig) {  // the results take most registers: w's operands come one by one
                    u32x4 xf[M];
#pragma unroll
                    for (int m = 0; m < M; ++m) xf[m] = read16(b, x_from + piece + 2048 * m);
#pragma unroll
                    for (int f = 0; f < FN; ++f) {
                        u32x4 w;
                        if constexpr (kTurn) {
                            const u32x2 lo = read_turned(b, turned[f] + 64 * S * columns), hi = read_turned(b, turned[f] + 64 * S * columns + 8 * columns);
                            w = u32x4{lo[0], lo[1], hi[0], hi[1]};
                        } else {
                            w = read16(b, w_from + piece + 2048 * f);
                        }
#pragma unroll
                        for (int m = 0; m < M; ++m) {
                            if constexpr (kMxX)
                                acc[f][m] = mfma_mx<S, S>(w, xf[m], acc[f][m], sw[f], sx[m]);
                            else
                                acc[f][m] = mfma_bf16(w, xf[m], acc[f][m]);
                        }
                    }
                    if constexpr (F == Form::kRows && M == FM) {
                        // w's reads three operands ahead of the products: 332 us against 339 with the
                        // compiler's order (16381 rows of 8 experts by 2816 x 4096); kMx 160 against 121
                        __builtin_amdgcn_sched_group_barrier(0x100, M + 3, 0);
                        __builtin_amdgcn_sched_group_barrier(0x8, M, 0);
#pragma unroll
                        for (int f = 3; f < FN; ++f) {
                            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x8, M, 0);
                        }
                        __builtin_amdgcn_sched_group_barrier(0x8, 2 * M, 0);
                    }
                    return;
                }
                u32x4 wf[FN], xf[M];
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    if constexpr (kTurn) {
                        const u32x2 lo = read_turned(b, turned[f] + 64 * S * columns), hi = read_turned(b, turned[f] + 64 * S * columns + 8 * columns);
                        wf[f] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                    } else {
                        wf[f] = read16(b, w_from + piece + 2048 * f);
                    }
                }
#pragma unroll
                for (int m = 0; m < M; ++m) xf[m] = read16(b, x_from + piece + 2048 * m);
#pragma unroll
                for (int f = 0; f < FN; ++f)
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        if constexpr (kMxX)
                            acc[f][m] = mfma_mx<S, S>(wf[f], xf[m], acc[f][m], sw[f], sx[m]);
                        else
                            acc[f][m] = mfma_bf16(wf[f], xf[m], acc[f][m]);
                    }
            };
            half(std::integral_constant<int, 0>());
            half(std::integral_constant<int, 1>());
        };
        // the stages, with products of 16 M rows (branches inside would take the results
        // apart in registers)
        auto run = [&](auto rows_16) {
            for (int stage = 0; stage < stages; ++stage) {
                if (stage > 0) step_barrier();
                if constexpr (decltype(rows_16)::value > 0) multiply(rows_16, buffers[buffer], scales[buffer]);
                buffer = buffer + 1 == D ? 0 : buffer + 1;
            }
        };
        const int rows_here = t.rows - 64 * wm;
        if (rows_here <= 0 || kColumns * wn >= t.cols) {  // nothing here for this wave
            run(std::integral_constant<int, 0>());
            continue;
        }
        if (rows_here <= 16)
            run(std::integral_constant<int, 1>());
        else if (FM == 2 || rows_here <= 32)
            run(std::integral_constant<int, 2>());
        else
            run(std::integral_constant<int, FM>());
        store_tile<FM, FN, kTurn, kF32>(a, t, acc, 64 * wm, kColumns * wn, lr, q);
    }
}

template <Form F, int kLow, bool kOnce>
void launch_product(const GroupedArgs& a, hipStream_t s) {
    const int64_t most = most_strips(a, kLow == 128 && F != Form::kBf16Mx ? 256 : kLow), units = most * ((a.N + kUnit - 1) / kUnit);
    const dim3 grid(static_cast<unsigned>(units < 256 ? (units + 7) / 8 * 8 : 256)), block(64 * (kCopiers + kMultipliers));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, a, static_cast<uint32_t>(most)); };
    if constexpr (F == Form::kMx || F == Form::kBf16Mx) {
        if (a.K < (F == Form::kBf16Mx && kLow == 128 ? 128 : 256)) {
            a.out_f32 ? go(moe_grouped_product<F, kLow, kOnce, true, true>) : go(moe_grouped_product<F, kLow, kOnce, false, true>);
            return;
        }
    }
    a.out_f32 ? go(moe_grouped_product<F, kLow, kOnce, true, false>) : go(moe_grouped_product<F, kLow, kOnce, false, false>);
}
template <Form F, int kLow>
void launch_product(const GroupedArgs& a, bool once, hipStream_t s) {
    once ? launch_product<F, kLow, true>(a, s) : launch_product<F, kLow, false>(a, s);
}

// Whether w's rows pass the GPU once and come from memory: then non-temporal loads are faster, 188 | 174 us for
// 4096 rows of 128 experts by 1408 x 2816 in bf16.  Where strips share weights they are slower (16381 rows of 8
// experts by 2816 x 4096, 340 | 362 us), and for 8 rows of 2816 x 704, whose 32 MB stay in a cache (11.1 | 12.6 us).
// From 128 MB to the 256 MB that the cache behind the L2s holds it depends on what ran since the last call with them.
// The next layer's weights push them out (three sets in turn): 72 rows of 18 experts by 1408 x 2816 (143 MB) 30 | 27 us,
// 512 rows of 32 (254 MB) 49 | 44, codes of 120 experts with 480 bf16 rows (253 MB) 55 | 50.  One set again and again: 24
// | 26, 41 | 44, 41 | 46.  A model has many layers, so the first is what counts.
inline bool read_once(const GroupedArgs& a, int64_t expert_bytes) {
    return a.A <= 192 * static_cast<int64_t>(a.E) && (a.A < a.E ? a.A : a.E) * expert_bytes > 128 << 20;
}

// Whether strips of 32 rows are faster, with x and w of one kind.  32 | 128, 128 experts by 1408 x
// 2816: 64 rows in bf16 68 | 79 us, 1024 rows 169 | 168 us, 4096 rows 213 | 174 us; both
// microscaled 24 | 26, 49 | 50 and 70 | 58 us.
inline bool low_strips(const GroupedArgs& a) { return a.A <= 8 * static_cast<int64_t>(a.E); }

// Whether tiles of 256 x 256 are faster: strips mostly full, rounds of tiles mostly full or many, and K long enough that
// a tile's start and its 256 x 256 results do not count.  Tiles at most 128 wide | 256 x 256, us, bf16 out, then fp32:
// 16381 rows of 8 experts by 2816 x 4096 (748 tiles) 343 | 330, 362 | 359, w turned 347 | 327, 370 | 345, both
// microscaled 139 | 119, 161 | 142; 16384 rows of 32 experts by 1408 x 2816 (480) 171 | 162, 186 | 176, w turned 174 |
// 157, 186 | 172, 67 | 59, 81 | 70; 16384 rows of one by 4096 x 4096 (1040) 443 | 429, 489 | 466, w turned 457 | 429,
// 491 | 459, 172 | 151, 230 | 198.  But 8192 rows of 8 by 2816 x 2816 (396) 129 | 143, 142 | 159, w turned 130 | 141, 141
// | 159, 48 | 52, 59 | 61, and with 256 rows an expert, 64 by 1408 x 2816, 185 | 220, 197 | 233, w turned 183 | 211, 196 |
// 225, 71 | 75, 81 | 86.  Short K, bf16 out: 65536 rows of 16 experts by 1024 x 128, 256, 512, 768: 37 | 46, 53 | 63, 92
// | 95, 128 | 131; w turned 38 | 43, 55 | 59, 92 | 90, 126 | 125; both microscaled 43 | 38, 34 | 38, 42 | 46, 55 | 55.  16381
// rows of 8 by 2816 x 64, 256, 512, 768: 26 | 27, 39 | 42, 56 | 58, 77 | 78; w turned 26 | 26, 40 | 38, 57 | 54, 82 | 74;
// both microscaled 31 | 26, 27 | 27, 32 | 31, 40 | 37.
inline bool big_tiles(const GroupedArgs& a) {
    const int32_t least = a.ws ? 0 : a.w_kn ? 256 : 640;
    return a.K >= least && a.A >= 512 * static_cast<int64_t>(a.E) &&
           (a.A / 256 + a.E / 2) * static_cast<int64_t>((a.N + 255) / 256) >= 448;
}

}  // namespace
}  // namespace moe
