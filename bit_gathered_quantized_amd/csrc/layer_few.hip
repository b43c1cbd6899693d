// A whole mixture-of-experts layer for at most 16 tokens in two launches.
//
//   1. moe_layer_few_route: logits = rstd (x . Wr^T), one workgroup an expert;
//      n = rms(x) w, one workgroup a token, as bf16 hi + lo (16 bits) in the order
//      of the matmul operand, with its sums over groups; the second launch's
//      counters are cleared.
//   2. moe_layer_few_experts: top-k in every workgroup (it is cheaper than a wait),
//      gate|up with the activation, down, and per token the weighted sum over its
//      experts with the norms and the residual around it.
//
// The time is that of reading each touched expert's weights once.  So the second
// launch holds the chip from the first byte to the last: one workgroup of eight
// waves a CU, whose waves have the weights of their next 32 rows in flight while
// they multiply the present ones, through the whole list of experts.  128 experts
// top-8, hidden 2816, expert width 704, one launch after the other: 8 tokens of
// 4-bit codes 66 us (174 MB), of which the weights stream for 40 us at 4.5 TB/s and
// 7 us are the first launch, 5 the lists, 4 the first loads, 4 the turn from gate|up
// to down, 5 the tokens; one token 31 us, 16 tokens of 8-bit codes 135 us (550 MB).
//
// Tiles.  An expert's rows go in tiles of at most 8: a 16-row MFMA operand holds
// the hi parts of 8 rows and their lo parts below, so 16-bit activations cost no
// MFMA more than 8-bit ones, and the two halves of a product are added at its end.
// The codes are exact operands (OFF + q).  With P = x . (OFF + q) over a group of
// columns and X the group's sum of x, the accumulator takes s P per group, and
// sum_g b X - s OFF X once per unit on MFMAs: a wave's slice has at most 8 groups
// (16 of 32 columns), s and b are bf16 as they are, and X goes in as three bf16
// parts in three of the four 8-value pieces of K, exact to its last bit.
//
// A unit is 32 weight rows (gate|up: 16 columns of h, both halves; down: 32
// output columns) by all of K, cut over 1, 2, 4 or 8 waves that hold at most 4
// chunks of 128 columns each, so that a wave keeps its slice of the tile's
// activations in registers for all units of the tile.  Few waves to a unit and long
// slices: a unit costs a wave 2 us whatever it holds, so 3 chunks instead of 2 in the
// down matmul above (2 waves, not 4) took it from 18 to 11 us.  Units are numbered
// tile by tile, and workgroup b takes the b-th of 256 equal ranges of them.
//
// Nothing in a range makes its waves wait for one another but the places for their
// shares of a unit, and those are four deep; a barrier a unit cost 8 tokens 8 us, and
// outputs made by whoever came last (the slowest wave, ever later) 8 us as well.
// Scales and biases are loaded by the wave that needs them, through its own LDS.
//
// Order between the phases without a barrier.  A range is taken by an exchange on
// its own flag.  A workgroup takes its own range of both matmuls when it starts,
// then, at the end of a phase, any range of it that is still untaken, and only when
// all ranges of a phase are taken does it go on: in the down matmul it waits for the
// counters (gate|up units done) of its range's tiles, and workgroup t, which makes
// token t's output at last, for those of the token's tiles.  So whoever waits waits
// for running workgroups, for ranges of an earlier phase than its own, and the first
// phase waits for nobody: every wait ends, however few workgroups the GPU holds at
// once.  (Waits are also bounded: calls that overlap on one workspace give undefined
// values, but no hang.)
//
// What one workgroup writes and another reads within the launch (h and its sums,
// y) is stored and loaded past the L2 of the XCD (sc1), rows of whole 128-byte
// lines; a writer counts its units only after its stores have been acknowledged
// (vmcnt 0).  Nothing else is shared, so no L2 write-back or invalidation is
// needed.
#include "block_norm.h"
#include "gemm_kernels.h"
#include "layer_cut.h"
#include "router_few.h"
#include "topk.h"

namespace moe {
namespace {

using cut::kDepth;
using cut::kLag;
using cut::kRanges;
using cut::kTileRows;
using cut::kWaves;
constexpr int kFewThreads = 64 * kWaves;
static_assert(kRanges == kLayerRanges, "ranges");
constexpr int kMaxSlots = kLayerFewTokens * kRouterMaxK;  // assignments, and so tiles
constexpr int kSc1 = 16;                                  // buffer access past the XCD's L2
constexpr int kPad = kLayerCounterStride;                 // counters lie on cache lines of their own
constexpr int kSpinLimit = 1 << 22;                       // polls: of memory about 1 us each, of LDS about 0.1 us

// ------------------------------------------------------------ first launch
template <int TM>
__device__ __forceinline__ void logits_of(const LayerArgs& a, int e, float (&part)[2][4][16]) {
    if (a.router.weight_f32)
        router::few_tokens<TM, true>(a.router, e, part);
    else
        router::few_tokens<TM, false>(a.router, e, part);
}

template <int TM>
__global__ __launch_bounds__(256) void moe_layer_few_route(LayerArgs a) {
    __shared__ float part[2][4][16];
    for (int i = blockIdx.x * 256 + threadIdx.x; i < a.num_counters; i += gridDim.x * 256) a.counters[i] = 0;
    if (static_cast<int>(blockIdx.x) < a.E) {
        logits_of<TM>(a, blockIdx.x, part);
        return;
    }
    // n of one token: two pieces of 8 columns a thread (H <= 4096)
    const int t = blockIdx.x - a.E, H = a.H;
    const norm::Rsrc sx = norm::row_rsrc(a.x, 2 * static_cast<int64_t>(H), t, H, 2);
    const norm::Rsrc sw = norm::row_rsrc(a.norm_weight, 0, 0, H, a.norm_f32 ? 4 : 2);
    const norm::Rsrc hw = a.norm_f32 ? sw : norm::row_rsrc(nullptr, 0, 0, 0, 0);
    norm::Raw<8> rx[2], rw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 8 * (threadIdx.x + 256 * i);
        rx[i] = norm::load_raw<8, false>(sx, c);
        rw[i] = norm::load_raw<8>(sw, hw, c, a.norm_f32);
    }
    float v[2][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] = norm::value(rx[i], j, false);
            ss = fmaf(v[i][j], v[i][j], ss);
        }
    const float rstd = a.norm ? 1.f / sqrtf(norm::row_sum<4>(ss, part[0][0]) / H + a.eps) : 1.f;
    const int gs = a.gs, per = gs / 8;  // threads of a group
    uint16_t* const n = a.n + static_cast<size_t>(2 * t) * H;
    float* const sums = a.nsum + static_cast<size_t>(2 * t) * (H / gs);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 8 * (threadIdx.x + 256 * i);
        uint32_t hi[4], lo[4];
        float shi = 0.f, slo = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (a.norm) v[i][j] *= rstd;
            if (a.norm_weight) v[i][j] *= a.weight_offset + norm::value(rw[i], j, a.norm_f32);
        }
        // operand order: 0,4,1,5,2,6,3,7
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = pack_bf16x2(v[i][j], v[i][j + 4]);
            const float h0 = __uint_as_float(hi[j] << 16), h1 = __uint_as_float(hi[j] & 0xFFFF0000u);
            lo[j] = pack_bf16x2(v[i][j] - h0, v[i][j + 4] - h1);
            shi += h0 + h1;
            slo += __uint_as_float(lo[j] << 16) + __uint_as_float(lo[j] & 0xFFFF0000u);
        }
        for (int off = 1; off < per; off <<= 1) {
            shi += __shfl_xor(shi, off);
            slo += __shfl_xor(slo, off);
        }
        if (c < H) {
            *reinterpret_cast<u32x4*>(n + c) = u32x4{hi[0], hi[1], hi[2], hi[3]};
            *reinterpret_cast<u32x4*>(n + H + c) = u32x4{lo[0], lo[1], lo[2], lo[3]};
            if (c % gs == 0) {
                sums[c / gs] = shi;
                sums[H / gs + c / gs] = slo;
            }
        }
    }
}

// ----------------------------------------------------------- second launch
// The lists that every workgroup makes of the chosen experts.  The assignments lie
// in h, its sums and y in the order of the tiles: row `start` + r is row r of a tile.
struct Lists {
    int32_t tiles;                    // tiles in all
    uint32_t tokens[kMaxSlots];       // the tokens of a tile's rows, 4 bits each
    uint16_t what[kMaxSlots];         // 16 * its expert + its rows
    uint16_t start[kMaxSlots];        // its first row
    uint16_t slot_tile[kMaxSlots];    // the tile of assignment t * k + j
    uint16_t slot_row[kMaxSlots];     // and its row in h and y
    float weight[kMaxSlots];          // and its routing weight
};

// Buffers in which a wave turns its weights: a unit's chunks at once where there is room.
template <int BITS>
constexpr int kBuffers = BITS == 4 ? 4 : 2;

template <int GS>
constexpr int kTablePieces = cut::table_pieces(GS);

template <int GS, int BITS>
struct alignas(16) FewSmem {
    uint32_t w[kWaves][kBuffers<BITS>][2 * 16 * 4 * BITS];   // weight transposition, a wave's own
    u32x4 tables[kWaves][2][2][16][kTablePieces<GS>];        // scales, biases of its slice of a unit
    float red[kDepth][kWaves][2][kTileRows][16];             // the waves' shares of the units' outputs
    int32_t arrived[kDepth][kWaves], finished[kDepth][kWaves];
    union {
        struct {                             // while the lists are made
            uint32_t mask[MOE_MAX_EXPERTS];  // tokens of each expert
            uint16_t tile[MOE_MAX_EXPERTS];  // its first tile
            uint16_t row[MOE_MAX_EXPERTS];   // and row
            uint16_t id[kMaxSlots];
            uint32_t scan[kWaves];
        };
        float lds[2][16];                    // sums of the last phase
    };
    int32_t pick, own[2];
    Lists l;
};

// A value that is the same in every lane, as a scalar (one read from LDS is not
// known to be).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One relaxed device-wide read of *p, polled until it reaches `want`.
__device__ __forceinline__ bool wait_for(const int32_t* p, int32_t want) {
    bool ok = false;
    for (int i = 0; i < kSpinLimit && !ok; ++i) {
        ok = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= want;
        if (!ok) __builtin_amdgcn_s_sleep(1);
    }
    asm volatile("" ::: "memory");
    return ok;
}

// The same in LDS, for another wave of the workgroup.
__device__ __forceinline__ bool wait_lds(const int32_t* p, int32_t want) {
    bool ok = false;
    for (int i = 0; i < kSpinLimit && !ok; ++i) {
        ok = uniform(__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) >= want;
        if (!ok) __builtin_amdgcn_s_sleep(1);
    }
    asm volatile("" ::: "memory");
    return ok;
}

// A wait ran out: the tokens that are finished after this become NaN.
__device__ __forceinline__ void give_up(const LayerArgs& a) {
    __hip_atomic_store(a.failed, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Takes any untaken range of a phase; -1 once all are taken.  Called by the whole
// workgroup.
template <class Smem>
__device__ __forceinline__ int take(Smem& sm, int32_t* flags) {
    for (;;) {
        __syncthreads();
        if (threadIdx.x == 0) sm.pick = INT32_MAX;
        __syncthreads();
        for (int i = threadIdx.x; i < kRanges; i += kFewThreads)
            if (!__hip_atomic_load(flags + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMin(&sm.pick, i);
        __syncthreads();
        const int want = sm.pick;
        if (want == INT32_MAX) return -1;
        __syncthreads();
        if (threadIdx.x == 0 && __hip_atomic_exchange(flags + want, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
            sm.pick = -1;  // another workgroup was first: look again
        __syncthreads();
        if (sm.pick >= 0) return want;
    }
}

// top-k of all tokens, then the tiles in expert order (rows in token order).
template <class Smem>
__device__ __forceinline__ void make_lists(const LayerArgs& a, Smem& sm) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int T = a.T, k = a.k, E = a.E;
    // the last wave (the first ones have most tokens) takes the workgroup's ranges
    if (wave == kWaves - 1 && lane < 2)
        sm.own[lane] = !__hip_atomic_exchange((lane ? a.claim_down : a.claim_gateup) + blockIdx.x, 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
    for (int e = threadIdx.x; e < E; e += kFewThreads) sm.mask[e] = 0;
    // tokens wave, wave + 8; the factors of the weights, and they, are needed at last
    TopK c[kLayerFewTokens / kWaves];
    float factor[kLayerFewTokens / kWaves], first[kLayerFewTokens / kWaves][2];
    const Rsrc logits = make_rsrc(a.logits, 4u * T * E);
#pragma unroll
    for (int i = 0; i < kLayerFewTokens / kWaves; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
            first[i][n] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(logits, 4u * ((wave + kWaves * i) * E + lane + 64 * n), 0, 0));
#pragma unroll
    for (int i = 0; i < kLayerFewTokens / kWaves; ++i) {
        const int t = wave + kWaves * i;
        if (t >= T) break;
        const float* row = a.logits + static_cast<size_t>(t) * E;
        if (E <= 128 && k <= 16) {
            c[i] = wave_topk_128(first[i][0], first[i][1], E, k);
        } else {
            float v[MOE_MAX_EXPERTS / 64];
#pragma unroll
            for (int n = 0; n < MOE_MAX_EXPERTS / 64; ++n) v[n] = lane + 64 * n < E ? row[lane + 64 * n] : -INFINITY;
            c[i] = wave_topk<MOE_MAX_EXPERTS / 64>(v, E, k, nullptr);
        }
        if (lane < k) sm.id[t * k + lane] = static_cast<uint16_t>(c[i].id);
        factor[i] = a.expert_scale && lane < k ? a.expert_scale[c[i].id] : 1.f;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < T * k; s += kFewThreads) atomicOr(&sm.mask[sm.id[s]], 1u << (s / k));
    __syncthreads();
    // tiles and rows before expert kPer i, by thread i: rows << 16 | tiles
    constexpr int kPer = MOE_MAX_EXPERTS / kFewThreads;
    const int e0 = kPer * threadIdx.x;
    uint32_t of[kPer], incl = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t rows = e0 + i < E ? __popc(sm.mask[e0 + i]) : 0;
        of[i] = rows << 16 | (rows + kTileRows - 1) / kTileRows;
        incl += of[i];
    }
    const uint32_t own = incl;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 63) sm.scan[wave] = incl;
    __syncthreads();
    uint32_t before = incl - own;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before += w < wave ? sm.scan[w] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e0 + i < E) {
            sm.tile[e0 + i] = static_cast<uint16_t>(before);
            sm.row[e0 + i] = static_cast<uint16_t>(before >> 16);
        }
        before += of[i];
    }
    if (threadIdx.x == kFewThreads - 1) sm.l.tiles = before & 0xFFFF;
    __syncthreads();
    for (int s = threadIdx.x; s < T * k; s += kFewThreads) {
        const int e = sm.id[s], t = s / k;
        uint32_t m = sm.mask[e];
        const int rank = __popc(m & ((1u << t) - 1u)), rows = __popc(m), tile = sm.tile[e] + rank / kTileRows;
        sm.l.slot_tile[s] = static_cast<uint16_t>(tile);
        sm.l.slot_row[s] = static_cast<uint16_t>(sm.row[e] + rank);
        if (rank % kTileRows == 0) {  // the tile's first row writes the tile
            const int count = min(kTileRows, rows - rank);
            m >>= t;
            uint32_t tokens = 0;
            for (int r = 0; r < count; ++r) {
                tokens |= static_cast<uint32_t>(t + __ffs(m) - 1) << (4 * r);
                m &= m - 1;
            }
            sm.l.tokens[tile] = tokens;
            sm.l.what[tile] = static_cast<uint16_t>(16 * e + count);
            sm.l.start[tile] = static_cast<uint16_t>(sm.row[e] + rank);
        }
    }
#pragma unroll
    for (int i = 0; i < kLayerFewTokens / kWaves; ++i) {
        const int s = (wave + kWaves * i) * k + lane;
        if (wave + kWaves * i >= T || lane >= k) break;
        const float w = c[i].weight * factor[i];
        sm.l.weight[s] = w;
        if (blockIdx.x == 0 && a.out_ids) a.out_ids[s] = c[i].id;
        if (blockIdx.x == 0 && a.out_weights) a.out_weights[s] = w;
    }
    __syncthreads();
}

// The sums over groups g0 .. g0 + 7 of one operand row, those from the n-th on
// zeros.  gate|up: from n's group sums; down: from h's sums over 16 columns.  `at`
// is the byte offset of group g0's.
template <int GS, bool kDown>
__device__ __forceinline__ void load_sums(float (&v)[8], Rsrc all, uint32_t at, int n) {
    constexpr int B = kDown ? GS / 16 : 1;  // floats of a group
    const Rsrc none = make_rsrc(nullptr, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Rsrc r = j < n ? all : none;
        const uint32_t o = at + 4 * B * j;
        if constexpr (B == 1) {
            v[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
        } else if constexpr (B == 2) {
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, kSc1));
            v[j] = __uint_as_float(b[0]) + __uint_as_float(b[1]);
        } else {
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < B / 4; ++h) {
                const f32x4 b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o + 16 * h, 0, kSc1));
                sum = (((sum + b[0]) + b[1]) + b[2]) + b[3];
            }
            v[j] = sum;
        }
    }
}

// v as a value that the compiler forms anew here: what follows from it is computed
// where it is used, not kept in registers through the loop.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+s"(v));
    return v;
}

// Waits until all loads of the wave have returned.  The compiler tracks loads per
// register over branches: one that may still be under way on one side of a branch
// makes every later use wait for whatever was issued since.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

// One phase (kDown: the down matmul, else gate|up) of one range of units; a wave's
// slice is CPW chunks of 128 columns (the last of a row may be missing: zeros).
// Returns whether `flags`, the phase's, still hold an untaken range.
//
// The loop over units has no branch around a load: what does not exist (a chunk
// past the row, a unit past the range) is read through an empty resource.
template <int GS, int BITS, bool kDown, int CPW>
__device__ __forceinline__ bool run_range(const LayerArgs& a, FewSmem<GS, BITS>& sm, int any_range, const int32_t* flags) {
    const int range = uniform(any_range);
    constexpr int CH = Geo<GS>::kChains, SH = Geo<GS>::kShift;
    constexpr int OFF = kCodeOffset<BITS, true>;
    constexpr int NS = (CPW * 128 / GS + 7) / 8;  // bias steps of a wave's slice
    constexpr int NP = kTablePieces<GS>;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, lr = lane & 15;
    const int K = kDown ? a.I : a.H, G = K / GS, row_words = K / 32 * BITS;
    const int rows_e = cut::expert_rows(kDown, a.H, a.I);
    const int upt = cut::units_of_tile(kDown, a.H, a.I);
    const int nch = cut::chunks(K);
    const int log_split = cut::split_log(nch), split = 1 << log_split;
    const int nu = kWaves >> log_split;           // units at work at a time
    const int wu = wave >> log_split, ws = wave & (split - 1);
    const int ch0 = cut::first_chunk(nch, log_split, ws), nc = cut::first_chunk(nch, log_split, ws + 1) - ch0;  // <= CPW
    const int N = uniform(sm.l.tiles) * upt;
    static_assert(kWaves == 1 << 3, "shares");
    auto first = [&](int share) { return cut::first_unit(N, share, 3 - log_split); };
    const int r0 = range * nu, lo = first(r0), hi = first(r0 + nu);
    const int u0 = first(r0 + wu), u1 = first(r0 + wu + 1);
    const uint32_t magic = kDown ? a.magic_down : a.magic_gateup;
    auto tile_of = [&](int u) { return cut::tile_of_unit(u, magic); };
    const int block_rows = cut::block_rows(kDown, a.I);
    const int g0 = cut::slice_group(GS, ch0), ng = cut::slice_groups(GS, G, ch0, nc);
    const int cols = cut::slice_columns(K, ch0, nc);
    // The tables' rows of a slice: lane (block, row, piece) loads pieces of 16 bytes.
    // Where the slice begins in its first piece is the same for all units (16 rows are
    // a multiple of 16 bytes).
    const int tb_ = lane >> 5, tr_ = lane >> 1 & 15, tp_ = lane & 1;
    const uint32_t tat = cut::table_load(G, g0, block_rows, tb_, tr_, tp_);
    WaveW<2, GS, BITS> ww;
    Rsrc rts, rtb;
    // loads are of unit u from now on, or of nothing from u1 on
    int ahead = 0;  // what[] of the unit to load next
    auto look = [&](int u) { ahead = sm.l.what[tile_of(min(u, u1 - 1))]; };
    auto aim = [&](int u) {
        const bool some = u < u1;
        // its first weight row
        const uint32_t r = cut::unit_row(kDown, rows_e, uniform(ahead >> 4), u - tile_of(u) * upt);
        const uint32_t* const w = (kDown ? a.w_d : a.w_gu) + static_cast<size_t>(r) * row_words;
        const uint32_t* const blk[2] = {w, w + static_cast<size_t>(block_rows) * row_words};
        ww.init(sm.w[wave][0], blk, row_words);
        const uint32_t left = 2u * G * (static_cast<uint32_t>(a.E) * rows_e - r);
        rts = make_rsrc((kDown ? a.s_d : a.s_gu) + static_cast<size_t>(r) * G, some ? left : 0);
        rtb = make_rsrc((kDown ? a.b_d : a.b_gu) + static_cast<size_t>(r) * G, some ? left : 0);
        if (!some) ww.blk[0] = ww.blk[1] = make_rsrc(w, 0);
    };
    u32x4 tv[2][NP / 2];
    auto load_tables = [&] {
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            tv[0][i] = load16(rts, tat, 32 * i);
            tv[1][i] = load16(rtb, tat, 32 * i);
        }
    };
    auto store_tables = [&] {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) sm.tables[wave][t][tb_][tr_][2 * i + tp_] = tv[t][i];
    };

    // a tile's activations for this wave's slice: operand row lr is part lr / 8 of
    // the tile's row lr % 8; rows past the tile and columns past K are zeros
    const uint32_t slots = static_cast<uint32_t>(kDown ? a.T * a.k : a.T);
    const Rsrc rx = make_rsrc(kDown ? a.h : a.n, 4u * K * slots);
    const Rsrc rs = kDown ? make_rsrc(a.hsum, 8u * (K / 16) * slots) : make_rsrc(a.nsum, 8u * G * slots);
    const Rsrc none = make_rsrc(a.n, 0);
    u32x4 x[CPW][4], xb[NS];
    float sums[NS][8];
    auto load_x = [&](int tile) {
        const int ng_ = fresh(ng), cols_ = fresh(cols);
        const int count = uniform(sm.l.what[tile]) & 15, r = lr & 7;
        const uint32_t from = kDown ? sm.l.start[tile] + r : sm.l.tokens[tile] >> (4 * r) & 15;
        const uint32_t src = 2u * from + (lr >> 3);
        // rows past the tile lie past every resource
        const bool mine = r < count;
        constexpr int B = kDown ? GS / 16 : 1;
#pragma unroll
        for (int st = 0; st < NS; ++st)
            load_sums<GS, kDown>(sums[st], rs, mine ? 4u * B * (src * G + g0 + 8 * st) : 0xFFFFF000u, ng_ - 8 * st);
        const uint32_t base = mine ? 2u * (K * src + 128 * ch0 + (Geo<GS>::kChain == 64 ? 16 : 8) * q) : 0xFFFFF000u;
#pragma unroll
        for (int i = 0; i < CPW; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const Rsrc rh = 128 * i + 64 * half < cols_ ? rx : none;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    x[i][2 * half + s] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   rh, base + 256 * i + 128 * half + (Geo<GS>::kChain == 64 ? 16 : 64) * s, 0, kDown ? kSc1 : 0));
            }
    };
    // lane (lr, q) brings part q of the sums of row lr: X = hi + mid + lo
    auto split_sums = [&] {
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            xb[st] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t pk = pack_bf16x2(sums[st][2 * j], sums[st][2 * j + 1]);
                    const float p0 = __uint_as_float(pk << 16), p1 = __uint_as_float(pk & 0xFFFF0000u);
                    sums[st][2 * j] -= p0;
                    sums[st][2 * j + 1] -= p1;
                    xb[st][j] = q == part ? pk : xb[st][j];
                }
        }
    };
    // eight entries of a table row of the slice, those past the slice as zeros
    const int tsub = cut::table_start(G, g0, lr);
    auto table8 = [&](int t, int b, int st, int ng) {
        u32x4 v;
        __builtin_memcpy(&v, reinterpret_cast<const char*>(sm.tables[wave][t][b][lr]) + tsub + 16 * st, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = ng - 8 * st - 2 * j;
            v[j] &= left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u;
        }
        return v;
    };
    u32x4 rv[CPW][2][BITS / 4];
    // chunk i of the slice, or one past every row if the slice is shorter
    auto chunk = [&](int i) { return i < nc ? ch0 + i : 1 << 20; };
    auto load_weights = [&] {
#pragma unroll
        for (int i = 0; i < CPW; ++i) ww.load(chunk(i), rv[i]);
    };

    // A wave's loads return in order.  So first what is needed first: the tables,
    // and gate|up's activations; down's have to wait for gate|up, and the wave that
    // waits (all others have their weights in flight meanwhile) keeps its weights
    // back.
    const bool idle = u0 == u1;
    int tile_now = idle ? -1 : tile_of(u0);
    if (tid < kDepth * kWaves) sm.arrived[tid / kWaves][tid % kWaves] = sm.finished[tid / kWaves][tid % kWaves] = 0;
    if (!idle) {
        look(u0);
        aim(u0);
        look(u0 + 1);
        load_tables();
        if constexpr (!kDown) load_x(tile_now);
        if (!kDown || wave != 0) load_weights();
        if constexpr (!kDown) split_sums();
    }
    if constexpr (kDown) {
        const int t = tile_of(lo) + lane;  // at most 5 tiles
        if (wave == 0 && lo < hi && t * upt < hi)
            if (!wait_for(a.done_gateup + t * kPad, a.I / 16)) give_up(a);
        __syncthreads();
        if (!idle) {
            load_x(tile_now);
            if (wave == 0) load_weights();
            split_sums();
        }
    } else {
        __syncthreads();
    }
    if (!idle) loads_done();
    const CodeConsts<OFF> kc = code_consts<OFF>(a.zero);
    // The outputs of the share's unit j: the sums of its waves' shares.
    auto finish = [&](int j) {
        const int slot = j % kDepth, u = u0 + j, tile = tile_of(u);
        if (!wait_lds(&sm.arrived[slot][wu], (j / kDepth + 1) << log_split)) give_up(a);
        const int count = uniform(sm.l.what[tile]) & 15, col = u - tile * upt;
        const uint32_t start = uniform(sm.l.start[tile]);
        const float(*const red)[2][kTileRows][16] = sm.red[slot] + wu * split;
        if constexpr (kDown) {  // 2 rows of 32 columns at a time
            const Rsrc ry = make_rsrc(a.y + static_cast<size_t>(start) * a.H, 4u * a.H * count);
            for (int r0 = 0; r0 < count; r0 += 2) {
                const int r = r0 + (lane >> 5), c = lane & 31;
                float o = 0.f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    const float p = red[min(v, split - 1)][c >> 4][r][c & 15];
                    o = v < split ? o + p : o;
                }
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o), ry, 4u * (r * a.H + 32 * col + c), 0, kSc1);
            }
        } else {  // 4 rows of 16 columns, both halves
            const Rsrc rh = make_rsrc(a.h + static_cast<size_t>(start) * 2 * a.I, 4u * a.I * count);
            const Rsrc rq = make_rsrc(a.hsum + static_cast<size_t>(start) * 2 * (a.I / 16), 8u * (a.I / 16) * count);
            for (int r0 = 0; r0 < count; r0 += 4) {
                const int r = r0 + q, c = lr;
                float o[2] = {0.f, 0.f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p = red[min(v, split - 1)][h][r][c];
                        o[h] = v < split ? o[h] + p : o[h];
                    }
                const float hv = (a.swiglu ? silu(o[0]) : gelu_tanh(o[0])) * o[1];
                const uint16_t hi16 = f32_to_bf16(hv), lo16 = f32_to_bf16(hv - bf16_to_f32(hi16));
                const uint32_t at = 2u * (2 * r * a.I + 16 * col + (c & ~7) + permuted_pos(c & 7));
                __builtin_amdgcn_raw_buffer_store_b16(hi16, rh, at, 0, kSc1);
                __builtin_amdgcn_raw_buffer_store_b16(lo16, rh, at + 2u * a.I, 0, kSc1);
                const float shi = sum16(bf16_to_f32(hi16)), slo = sum16(bf16_to_f32(lo16));
                // rows past the count lie past every resource
                if (c < 2)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(c ? slo : shi), rq,
                                                          4u * ((2 * r + c) * (a.I / 16) + col), 0, kSc1);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (lane == 0)
            __hip_atomic_store(&sm.finished[slot][wu], j / kDepth + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    // The waves of a unit are not in step.  Each leaves its share in one of kDepth
    // places in turn and counts itself; the waves take turns at making the outputs,
    // kLag units later, when all shares are there as a rule, and count that too: then
    // the place may be written again.
    for (int it = 0; it < u1 - u0 + kLag; ++it) {
        if (it >= kLag && ((it - kLag) & (split - 1)) == ws) finish(it - kLag);
        const int u = u0 + it;
        if (u >= u1) continue;
        const int tile = tile_of(u);
        if (tile != tile_now) {
            tile_now = tile;
            load_x(tile);
            split_sums();
            loads_done();
        }
        store_tables();
        aim(u + 1);
        load_tables();
        look(u + 2);
        const int free = __hip_atomic_load(&sm.finished[it % kDepth][wu], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        const int ngl = fresh(ng);
        u32x4 sc[2][NS];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int st = 0; st < NS; ++st) sc[b][st] = table8(0, b, st, ngl);
        // chunk i of this unit into its buffer, of the next unit into its registers
        constexpr bool kAll = CPW <= kBuffers<BITS>;
        auto turn = [&](int i) {
            ww.lds = sm.w[wave][i % kBuffers<BITS>];
            ww.put(rv[i]);
            ww.load(chunk(i), rv[i]);
        };
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < (kAll ? CPW : 1); ++i) turn(i);
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            if (!kAll || i == 0) {
                chunk_fence();
                if (!kAll && i + 1 < CPW) turn(i + 1);
                __builtin_amdgcn_wave_barrier();
            }
            ww.lds = sm.w[wave][i % kBuffers<BITS>];
            WLane<BITS> wv[2];
            float s16[2][CH];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                wv[b] = ww.get(b, lr, q);
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    const int g = (i * CH + j) >> SH;
                    const uint32_t pair = sc[b][g >> 3][(g & 7) >> 1];
                    s16[b][j] = __uint_as_float(g & 1 ? pair & 0xFFFF0000u : pair << 16);
                }
            }
            // columns past the slice have zeros in x
            chunk_steps<GS, 2, 4, BITS>(acc, x[i], wv, s16, kc);
            if (!kAll || i + 1 == CPW) __builtin_amdgcn_wave_barrier();
        }
        // + sum_g b X - OFF s X
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x4& o = acc[b];
            f32x4 sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                o = mfma16(xb[st], table8(1, b, st, ngl), o);
                if constexpr (OFF != 0) sx = mfma16(xb[st], sc[b][st], sx);
            }
            if constexpr (OFF != 0) {
#pragma unroll
                for (int v = 0; v < 4; ++v) o[v] = fmaf(-static_cast<float>(OFF), sx[v], o[v]);
            }
        }
        const int slot = it % kDepth;
        if (uniform(free) < it / kDepth && !wait_lds(&sm.finished[slot][wu], it / kDepth)) give_up(a);
        // operand rows 8..15 are the lo parts of rows 0..7, in the wave's upper half:
        // the halves of two blocks trade places so that the lower half adds up the
        // first one, the upper half the second
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const u32x2 t = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[0][v]), __float_as_uint(acc[1][v]), false, false));
            sm.red[slot][wave][lane >> 5][4 * (q & 1) + v][lr] = __uint_as_float(t[0]) + __uint_as_float(t[1]);
        }
        asm volatile("" ::: "memory");  // the LDS operations of a wave keep their order
        if (lane == 0) __hip_atomic_fetch_add(&sm.arrived[slot][wu], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    // the range is done once its stores have been acknowledged; the phase's flags
    // are read meanwhile
    static_assert(kRanges <= kFewThreads, "a flag a thread");
    const int taken = tid < kRanges ? __hip_atomic_load(flags + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const bool left = __syncthreads_or(!taken);
    const int t0 = tile_of(lo) + tid;
    if (lo < hi && t0 * upt < hi) {
        const int n = min(hi, (t0 + 1) * upt) - max(lo, t0 * upt);
        __hip_atomic_fetch_add((kDown ? a.done_down : a.done_gateup) + t0 * kPad, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    return left;
}

// The same with the chunks of a wave's slice known: up to 2, 3 or 4.
template <int GS, int BITS, bool kDown>
__device__ __forceinline__ bool run_range(const LayerArgs& a, FewSmem<GS, BITS>& sm, int range, const int32_t* flags) {
    const int most = cut::most_chunks(cut::chunks(kDown ? a.I : a.H));
    if (most <= 2) return run_range<GS, BITS, kDown, 2>(a, sm, range, flags);
    return most <= 3 ? run_range<GS, BITS, kDown, 3>(a, sm, range, flags)
                     : run_range<GS, BITS, kDown, 4>(a, sm, range, flags);
}

// out and normed of one token.
template <int GS, int BITS>
__device__ __forceinline__ void finish_token(const LayerArgs& a, FewSmem<GS, BITS>& sm, int t) {
    constexpr int NV = 4096 / (8 * kFewThreads), kStep = 8 * kFewThreads;
    const int c0 = 8 * threadIdx.x, k = a.k, H = a.H;
    norm::Row<kWaves, NV, 8, -1> row;
    row.load(a.tail, t, c0);
    if (static_cast<int>(threadIdx.x) < k)  // lanes of the first wave
        if (!wait_for(a.done_down + sm.l.slot_tile[t * k + threadIdx.x] * kPad, H / 32)) give_up(a);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int failed = __hip_atomic_load(a.failed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float z[NV][8] = {};
    const Rsrc ry = make_rsrc(a.y, 4u * H * static_cast<uint32_t>(a.T * k));
    constexpr int J = 8;  // experts in flight
    for (int j0 = 0; j0 < k; j0 += J) {
        u32x4 v[J][NV][2];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t row = sm.l.slot_row[t * k + min(j0 + j, k - 1)];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = c0 + kStep * i;
                    const uint32_t at = c < H ? 4u * (row * H + c + 4 * h) : 0xFFFFFFF0u;
                    v[j][i][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, at, 0, kSc1));
                }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float wt = sm.l.weight[t * k + min(j0 + j, k - 1)];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float p = wt * __uint_as_float(v[j][i][n >> 2][n & 3]);
                    z[i][n] = j0 + j < k ? z[i][n] + p : z[i][n];
                }
        }
    }
    if (failed) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int n = 0; n < 8; ++n) z[i][n] = __uint_as_float(0x7FC00000u);
    }
    row.finish(a.tail, t, c0, z, sm.lds);
}

template <int GS, int BITS>
__global__ __launch_bounds__(kFewThreads, 1) void moe_layer_few_experts(LayerArgs a) {
    __shared__ FewSmem<GS, BITS> sm;
    make_lists(a, sm);
    // usually one range of each phase; more if workgroups have not started yet
    for (int r = sm.own[0] ? blockIdx.x : take(sm, a.claim_gateup); r >= 0;)
        r = run_range<GS, BITS, false>(a, sm, r, a.claim_gateup) ? take(sm, a.claim_gateup) : -1;
    for (int r = sm.own[1] ? blockIdx.x : take(sm, a.claim_down); r >= 0;)
        r = run_range<GS, BITS, true>(a, sm, r, a.claim_down) ? take(sm, a.claim_down) : -1;
    if (static_cast<int>(blockIdx.x) < a.T) finish_token(a, sm, blockIdx.x);
}

template <int GS, int BITS>
hipError_t launch_experts(const LayerArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((moe_layer_few_experts<GS, BITS>), dim3(kRanges), dim3(kFewThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_few(const LayerArgs& a, hipStream_t s) {
    const dim3 grid(a.E + a.T), block(256);
    if (a.T <= 1)
        hipLaunchKernelGGL(moe_layer_few_route<1>, grid, block, 0, s, a);
    else if (a.T <= 2)
        hipLaunchKernelGGL(moe_layer_few_route<2>, grid, block, 0, s, a);
    else if (a.T <= 4)
        hipLaunchKernelGGL(moe_layer_few_route<4>, grid, block, 0, s, a);
    else if (a.T <= 8)
        hipLaunchKernelGGL(moe_layer_few_route<8>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(moe_layer_few_route<16>, grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.bits == 4)
        return a.gs == 32 ? launch_experts<32, 4>(a, s) : a.gs == 64 ? launch_experts<64, 4>(a, s) : launch_experts<128, 4>(a, s);
    return a.gs == 32 ? launch_experts<32, 8>(a, s) : a.gs == 64 ? launch_experts<64, 8>(a, s) : launch_experts<128, 8>(a, s);
}

}  // namespace moe
