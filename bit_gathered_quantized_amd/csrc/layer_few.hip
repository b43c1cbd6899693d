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
// they multiply the present ones, through the whole list of experts.
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
// output columns) by all of K, cut over SPLIT waves that hold at most 4 chunks of
// 128 columns each, so that a wave keeps its slice of the tile's activations in
// registers for all units of the tile.  Units are numbered tile by tile, and
// workgroup b takes the b-th of 256 equal ranges of them.
//
// Order between the phases without a barrier.  A range is taken by an exchange on
// its own flag.  A workgroup takes its own range of both matmuls when it starts,
// then, at the end of a phase, any range of it that is still untaken, and only
// when all ranges of a phase are taken does it wait for the counters (units done
// per tile) of that phase; workgroup t finishes token t at last.  So whoever waits waits for running workgroups, for
// ranges of an earlier phase than its own, and the first phase waits for nobody:
// every wait ends, however few workgroups the GPU holds at once.  (Waits are also bounded: a workspace that another call writes to gives
// NaN, not a hang.)
//
// What one workgroup writes and another reads within the launch (h and its sums,
// y) is stored and loaded past the L2 of the XCD (sc1), rows of whole 128-byte
// lines; a writer counts its units only after its stores have been acknowledged
// (vmcnt 0).  Nothing else is shared, so no L2 write-back or invalidation is
// needed.
#include "block_norm.h"
#include "gemm_kernels.h"
#include "router_few.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kWaves = 8, kFewThreads = 64 * kWaves;
constexpr int kRanges = kLayerRanges;
constexpr int kTileRows = 8;
constexpr int kMaxSlots = kLayerFewTokens * kRouterMaxK;  // assignments, and so tiles
constexpr int kChunks = 4;                                // chunks of 128 columns a wave holds
constexpr int kSc1 = 16;                                  // buffer access past the XCD's L2
constexpr int kPad = kLayerCounterStride;                 // counters lie on cache lines of their own
constexpr int kSpinLimit = 1 << 22;                       // polls of about 1 us

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
// The lists that every workgroup makes of the chosen experts.
struct Lists {
    int32_t tiles;                             // tiles in all
    uint16_t rows[kMaxSlots][kTileRows];       // 64 t + j of a tile's rows
    uint16_t expert[kMaxSlots];                // a tile's expert
    uint8_t count[kMaxSlots];                  // and its rows
    uint16_t slot_tile[kMaxSlots];             // the tile of an assignment
    float weight[kMaxSlots];                   // its routing weight
};

// Chunks that a wave turns at a time: all of a unit with 4-bit codes, half of it
// with 8-bit ones (LDS).
template <int BITS>
constexpr int kBuffers = BITS == 4 ? kChunks : kChunks / 2;

// 16-byte pieces of scales (or biases) of the units at work per thread of half a
// workgroup: units times columns are at most 4096.
template <int GS>
constexpr int kTablePieces = 4 * 4096 / GS / (kFewThreads / 2) > 0 ? 4 * 4096 / GS / (kFewThreads / 2) : 1;

// A row of nch chunks is cut over 1 << split_log waves.
__device__ __forceinline__ int split_log(int nch) { return nch <= 4 ? 0 : nch <= 8 ? 1 : nch <= 16 ? 2 : 3; }

template <int GS, int BITS>
struct alignas(16) FewSmem {
    uint32_t w[kWaves][kBuffers<BITS>][2 * 16 * 4 * BITS];  // weight transposition, a wave's own
    uint16_t tables[2][2][kTablePieces<GS> * kFewThreads / 2 * 8];  // scales, biases of the units at work, of the next ones
    float red[2][kWaves][2][kTileRows][16];         // the waves' shares of the units' outputs
    union {
        struct {
            uint32_t mask[MOE_MAX_EXPERTS];     // tokens of each expert
            uint16_t base[MOE_MAX_EXPERTS];     // its first tile
            uint16_t id[kMaxSlots];
            uint32_t scan[kWaves];
        };
        float lds[2][16];                       // sums of the last phase
    };
    int32_t pick, own[2];
    Lists l;
};

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

// A wait ran out: every token becomes NaN.
__device__ __forceinline__ void give_up(const LayerArgs& a) {
    __hip_atomic_store(a.failed, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Takes any untaken one of n <= kFewThreads flags; -1 once all are taken.  Called
// by the whole workgroup.
template <class Smem>
__device__ __forceinline__ int take(Smem& sm, int32_t* flags, int n) {
    for (;;) {
        __syncthreads();
        if (threadIdx.x == 0) sm.pick = INT32_MAX;
        __syncthreads();
        const int i = threadIdx.x;
        if (i < n && !__hip_atomic_load(flags + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMin(&sm.pick, i);
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
    // the last wave (the first ones have a token each) takes the workgroup's ranges
    if (wave == kWaves - 1 && lane < 2)
        sm.own[lane] = !__hip_atomic_exchange((lane ? a.claim_down : a.claim_gateup) + blockIdx.x, 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
    for (int e = threadIdx.x; e < E; e += kFewThreads) sm.mask[e] = 0;
    for (int t = wave; t < T; t += kWaves) {
        const float* row = a.logits + static_cast<size_t>(t) * E;
        TopK c;
        if (E <= 128) {
            float v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
            c = wave_topk<2>(v, E, k, a.expert_scale);
        } else {
            float v[MOE_MAX_EXPERTS / 64];
#pragma unroll
            for (int i = 0; i < MOE_MAX_EXPERTS / 64; ++i) v[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
            c = wave_topk<MOE_MAX_EXPERTS / 64>(v, E, k, a.expert_scale);
        }
        if (lane < k) {
            sm.id[t * k + lane] = static_cast<uint16_t>(c.id);
            sm.l.weight[t * k + lane] = c.weight;
            if (blockIdx.x == 0 && a.out_ids) a.out_ids[t * k + lane] = c.id;
            if (blockIdx.x == 0 && a.out_weights) a.out_weights[t * k + lane] = c.weight;
        }
    }
    __syncthreads();
    for (int s = threadIdx.x; s < T * k; s += kFewThreads) atomicOr(&sm.mask[sm.id[s]], 1u << (s / k));
    __syncthreads();
    // tiles before expert 2 i, by thread i (E <= 1024 = 2 kFewThreads)
    const int e0 = 2 * threadIdx.x;
    auto tiles_of = [&](int e) { return e < E ? (__popc(sm.mask[e]) + kTileRows - 1) / kTileRows : 0; };
    const int n0 = tiles_of(e0), n1 = tiles_of(e0 + 1);
    int incl = n0 + n1;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 63) sm.scan[wave] = incl;
    __syncthreads();
    int before = incl - n0 - n1;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before += w < wave ? sm.scan[w] : 0;
    if (e0 < E) sm.base[e0] = static_cast<uint16_t>(before);
    if (e0 + 1 < E) sm.base[e0 + 1] = static_cast<uint16_t>(before + n0);
    if (threadIdx.x == kFewThreads - 1) sm.l.tiles = before + n0 + n1;
    __syncthreads();
    for (int s = threadIdx.x; s < T * k; s += kFewThreads) {
        const int e = sm.id[s], t = s / k;
        const uint32_t m = sm.mask[e];
        const int rank = __popc(m & ((1u << t) - 1u)), tile = sm.base[e] + rank / kTileRows;
        sm.l.rows[tile][rank % kTileRows] = static_cast<uint16_t>(64 * t + s - t * k);
        sm.l.slot_tile[s] = static_cast<uint16_t>(tile);
        if (rank % kTileRows == 0) {
            sm.l.expert[tile] = static_cast<uint16_t>(e);
            sm.l.count[tile] = static_cast<uint8_t>(min(kTileRows, __popc(m) - rank));
        }
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

// A value that is the same in every lane, as a scalar (one read from LDS is not
// known to be).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

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
    const int rows_e = kDown ? a.H : 2 * a.I;     // weight rows of an expert
    const int upt = kDown ? a.H / 32 : a.I / 16;  // units of a tile
    const int nch = (K + 127) / 128;
    const int log_split = split_log(nch), split = 1 << log_split;
    const int nu = kWaves >> log_split;           // units at work at a time
    const int wu = wave >> log_split, ws = wave & (split - 1);
    const int ch0 = nch * ws >> log_split, nc = (nch * (ws + 1) >> log_split) - ch0;  // this wave's chunks, <= CPW
    const int N = uniform(sm.l.tiles) * upt, shift = 8 + 3 - log_split;  // kRanges * nu shares, N share < 2^30
    static_assert(kRanges == 1 << 8 && kWaves == 1 << 3, "shift");
    auto first = [&](int share) { return N * share >> shift; };
    const int r0 = range * nu, lo = first(r0), hi = first(r0 + nu);
    const int u0 = first(r0 + wu), u1 = first(r0 + wu + 1);
    // the shares of a range differ by one unit at most
    int steps = 0;
    for (int i = 0; i < nu; ++i) steps = max(steps, first(r0 + i + 1) - first(r0 + i));

    // u / upt for u < 2^18, upt <= 256: u (m upt - 2^32) < 2^26 errs by less than 1 / upt
    const uint32_t magic = kDown ? a.magic_down : a.magic_gateup;
    auto tile_of = [&](int u) { return static_cast<int>(__umulhi(static_cast<uint32_t>(u), magic)); };
    // the first weight row of block b of unit u
    auto row_of = [&](int u, int b) {
        const int tile = tile_of(u), i = u - tile * upt;
        const uint32_t e = sm.l.expert[tile];
        return e * rows_e + (kDown ? 32 * i + 16 * b : 16 * i + (b ? a.I : 0));
    };
    WaveW<2, GS, BITS> ww;
    // ww loads unit u from now on, or nothing from u1 on
    auto aim = [&](int u) {
        const uint32_t* const w = kDown ? a.w_d : a.w_gu;
        const uint32_t* blk[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t r = uniform(row_of(min(u, u1 - 1), b));
            blk[b] = w + static_cast<size_t>(r) * row_words;
        }
        ww.init(sm.w[wave][0], blk, row_words);
        if (u >= u1) ww.blk[0] = ww.blk[1] = make_rsrc(w, 0);
    };
    // Tables: the scales of the units at work, then their biases, 2 G pieces of 16
    // bytes a block of 16 rows.  The first half of the workgroup loads scales, the
    // other biases, NP pieces a thread.
    constexpr int kHalf = kFewThreads / 2;
    const bool biases = wave >= kWaves / 2;
    const uint16_t* const tab = kDown ? (biases ? a.b_d : a.s_d) : (biases ? a.b_gu : a.s_gu);
    const Rsrc rt = make_rsrc(tab, 2u * a.E * rows_e * G);
    int tu[NP];        // a piece's unit, its block and its place in the block
    uint32_t tblk[NP], tat[NP];
#pragma unroll
    for (int h = 0; h < NP; ++h) {
        const int p = (tid & (kHalf - 1)) + kHalf * h, i = p / (4 * G), r = p - i * 4 * G;
        tu[h] = i;
        tblk[h] = r / (2 * G);
        tat[h] = 16 * (r - tblk[h] * 2 * G);
    }
    u32x4 tv[NP];
    auto load_tables = [&](int step) {
#pragma unroll
        for (int h = 0; h < NP; ++h) {
            const int u = first(r0 + tu[h]) + step, end = first(r0 + tu[h] + 1);
            const uint32_t at = 2u * G * row_of(max(min(u, end - 1), 0), tblk[h]) + tat[h];
            tv[h] = load16(rt, tu[h] < nu && u < end ? at : 0xFFFFFFF0u, 0);
        }
    };
    auto store_tables = [&](int step) {
#pragma unroll
        for (int h = 0; h < NP; ++h)
            *reinterpret_cast<u32x4*>(sm.tables[step & 1][biases] + 8 * ((tid & (kHalf - 1)) + kHalf * h)) = tv[h];
    };

    // a tile's activations for this wave's slice: operand row lr is part lr / 8 of
    // the tile's row lr % 8; rows past the tile and columns past K are zeros
    const uint32_t slots = static_cast<uint32_t>(kDown ? a.T * a.k : a.T);
    const Rsrc rx = make_rsrc(kDown ? a.h : a.n, 4u * K * slots);
    const Rsrc rs = kDown ? make_rsrc(a.hsum, 8u * (K / 16) * slots) : make_rsrc(a.nsum, 8u * G * slots);
    const Rsrc none = make_rsrc(a.n, 0);
    u32x4 x[CPW][4], xb[NS], xo[NS];
    float sums[NS][8];
    const int g0 = ch0 * 128 / GS, ng = min(nc * 128 / GS, G - g0);  // the slice's groups
    const int cols = min(nc * 128, K - 128 * ch0);                   // and columns
    auto load_x = [&](int tile) {
        const int ng_ = fresh(ng), cols_ = fresh(cols);
        const int count = sm.l.count[tile], r = lr & 7;
        const int slot = sm.l.rows[tile][min(r, count - 1)];
        const uint32_t src = 2u * static_cast<uint32_t>(kDown ? (slot >> 6) * a.k + (slot & 63) : slot >> 6) + (lr >> 3);
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
            xo[st] = xb[st];
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t pk = pack_bf16x2(sums[st][2 * j], sums[st][2 * j + 1]);
                    const float p0 = __uint_as_float(pk << 16), p1 = __uint_as_float(pk & 0xFFFF0000u);
                    sums[st][2 * j] -= p0;
                    sums[st][2 * j + 1] -= p1;
                    const uint32_t off = pack_bf16x2(-static_cast<float>(OFF) * p0, -static_cast<float>(OFF) * p1);
                    xb[st][j] = q == part ? pk : xb[st][j];
                    xo[st][j] = q == part ? off : xo[st][j];
                }
        }
    };
    // eight entries of a table row, those past the slice as zeros
    auto table8 = [&](const uint16_t* t, int st, int ng) {
        u32x4 v;
        __builtin_memcpy(&v, t + g0 + 8 * st, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = ng - 8 * st - 2 * j;
            v[j] &= left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u;
        }
        return v;
    };
    u32x4 rv[CPW][2][BITS / 4];
    auto load_weights = [&] {
#pragma unroll
        for (int i = 0; i < CPW; ++i) ww.load(ch0 + i, rv[i]);
    };

    // A wave's loads return in order.  So first what is needed first: the tables,
    // and gate|up's activations; down's have to wait for gate|up, and the wave that
    // waits (all others have their weights in flight meanwhile) keeps its weights
    // back.
    const bool idle = u0 == u1;
    int tile_now = idle ? -1 : tile_of(u0);
    if (!idle) {
        load_tables(0);
        if constexpr (!kDown) load_x(tile_now);
        aim(u0);
        if (!kDown || wave != 0) load_weights();
        store_tables(0);
        if constexpr (!kDown) {
            split_sums();
            loads_done();
        }
    } else {
        load_tables(0);
        store_tables(0);
    }
    if constexpr (kDown) {
        const int t = tile_of(lo) + lane;  // at most 6 tiles
        if (wave == 0 && lo < hi && t * upt < hi)
            if (!wait_for(a.done_gateup + t * kPad, a.I / 16)) give_up(a);
        __syncthreads();
        if (!idle) {
            load_x(tile_now);
            if (wave == 0) load_weights();
            split_sums();
            loads_done();
        }
    }
    const CodeConsts<OFF> kc = code_consts<OFF>(a.zero);
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        const int u = u0 + step;
        load_tables(step + 1);
        if (!idle) {
            const int tile = tile_of(min(u, u1 - 1));
            if (tile != tile_now) {
                tile_now = tile;
                load_x(tile);
                split_sums();
                loads_done();
            }
            aim(u + 1);
            const uint16_t* const ts = sm.tables[step & 1][0] + (32 * wu + lr) * G;
            const uint16_t* const tb = sm.tables[step & 1][1] + (32 * wu + lr) * G;
            const int ngl = fresh(ng);
            f32x4 acc[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int st = 0; st < NS; ++st) {
                    acc[b] = mfma16(xb[st], table8(tb + 16 * b * G, st, ngl), acc[b]);
                    if constexpr (OFF != 0) acc[b] = mfma16(xo[st], table8(ts + 16 * b * G, st, ngl), acc[b]);
                }
            }
            constexpr int NB = kBuffers<BITS>;
#pragma unroll
            for (int h = 0; h < CPW; h += NB) {
                // the weights of this unit through LDS, those of the next into their place
#pragma unroll
                for (int i = h; i < h + NB && i < CPW; ++i) {
                    ww.lds = sm.w[wave][i - h];
                    ww.put(rv[i]);
                    ww.load(ch0 + i, rv[i]);
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = h; i < h + NB && i < CPW; ++i) {
                    chunk_fence();  // one chunk's operands at a time: registers
                    ww.lds = sm.w[wave][i - h];
                    WLane<BITS> wv[2];
                    float s[2][CH];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        wv[b] = ww.get(b, lr, q);
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            s[b][j] = bf16_to_f32(ts[16 * b * G + min(g0 + ((i * CH + j) >> SH), G - 1)]);
                    }
                    // columns past the slice have zeros in x
                    chunk_steps<GS, 2, 4, BITS>(acc, x[i], wv, s, kc);
                }
                __builtin_amdgcn_wave_barrier();
            }
            // operand rows 8..15 are the lo parts of rows 0..7, in the wave's upper half:
            // the halves trade places so that the lower one adds up block 0, the upper
            // one block 1
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const u32x2 t = __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[0][v]), __float_as_uint(acc[1][v]), false, false));
                sm.red[step & 1][wave][lane >> 5][4 * (q & 1) + v][lr] = __uint_as_float(t[0]) + __uint_as_float(t[1]);
            }
        }
        store_tables(step + 1);
        __syncthreads();
        // the units' outputs: wave r adds up the shares of row r, 16 columns of both
        // halves of gate|up by 4 lanes each, 32 of down by 2
        constexpr int kCols = kDown ? 32 : 16;
        const int r = wave, c = lane % kCols;
        for (int i = 0; i < nu; ++i) {
            const int uu = first(r0 + i) + step;
            if (uu >= first(r0 + i + 1)) continue;
            const int t = tile_of(uu), col = uu - t * upt;
            if (r >= uniform(sm.l.count[t])) continue;
            const int id = uniform(sm.l.rows[t][r]);
            const size_t slot = (id >> 6) * a.k + (id & 63);
            float o[2] = {0.f, 0.f};
            for (int v = lane / kCols; v < split; v += 64 / kCols) {
                const auto& red = sm.red[step & 1][(i << log_split) + v];
                if constexpr (kDown) {
                    o[0] += red[c >> 4][r][c & 15];
                } else {
                    o[0] += red[0][r][c];
                    o[1] += red[1][r][c];
                }
            }
#pragma unroll
            for (int off = kCols; off < 64; off <<= 1) {
                o[0] += __shfl_xor(o[0], off);
                if constexpr (!kDown) o[1] += __shfl_xor(o[1], off);
            }
            if constexpr (kDown) {
                const Rsrc ry = make_rsrc(a.y + slot * a.H, 4u * a.H);
                if (lane < kCols)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), ry, 4 * (32 * col + c), 0, kSc1);
            } else {
                const float hv = (a.swiglu ? silu(o[0]) : gelu_tanh(o[0])) * o[1];
                const uint16_t hi16 = f32_to_bf16(hv), lo16 = f32_to_bf16(hv - bf16_to_f32(hi16));
                const float shi = sum16(bf16_to_f32(hi16)), slo = sum16(bf16_to_f32(lo16));
                // lanes 0..15 store the hi parts, 16..31 the lo parts
                const Rsrc rh = make_rsrc(a.h, 4u * a.I * static_cast<uint32_t>(a.T * a.k));
                const uint32_t part = 2 * static_cast<uint32_t>(slot) + (lane >> 4);
                if (lane < 32)
                    __builtin_amdgcn_raw_buffer_store_b16(lane < 16 ? hi16 : lo16, rh,
                                                          2u * (part * a.I + 16 * col + (c & 8) + permuted_pos(c & 7)), 0, kSc1);
                const Rsrc rq = make_rsrc(a.hsum, 8u * (a.I / 16) * static_cast<uint32_t>(a.T * a.k));
                if (lane == 0 || lane == 16)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lane ? slo : shi), rq, 4u * (part * (a.I / 16) + col), 0,
                                                          kSc1);
            }
        }
    }
    // the range is done once its stores have been acknowledged; the phase's flags
    // are read meanwhile
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

// The same with the chunks of a wave's slice known: 3, or 4.
template <int GS, int BITS, bool kDown>
__device__ __forceinline__ bool run_range(const LayerArgs& a, FewSmem<GS, BITS>& sm, int range, const int32_t* flags) {
    const int nch = ((kDown ? a.I : a.H) + 127) / 128;
    const int log_split = split_log(nch), most = (nch + (1 << log_split) - 1) >> log_split;
    return most <= 3 ? run_range<GS, BITS, kDown, 3>(a, sm, range, flags)
                     : run_range<GS, BITS, kDown, 4>(a, sm, range, flags);
}

// out and normed of one token.
template <int GS, int BITS>
__device__ __forceinline__ void finish_token(const LayerArgs& a, FewSmem<GS, BITS>& sm, int t) {
    const int c0 = 8 * threadIdx.x, k = a.k, H = a.H;
    norm::Row<kWaves, 1, 8, -1> row;
    row.load(a.tail, t, c0);
    if (static_cast<int>(threadIdx.x) < k)  // lanes of the first wave
        if (!wait_for(a.done_down + sm.l.slot_tile[t * k + threadIdx.x] * kPad, H / 32)) give_up(a);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int failed = __hip_atomic_load(a.failed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float z[1][8] = {};
    const Rsrc ry = make_rsrc(a.y + static_cast<size_t>(t) * k * H, 4u * H * k);
    for (int j0 = 0; j0 < k; j0 += 8) {
        u32x4 v[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = j0 + j < k && c0 < H ? 4u * ((j0 + j) * H + c0 + 4 * h) : 0xFFFFFFF0u;
                v[j][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, at, 0, kSc1));
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float wt = j0 + j < k ? sm.l.weight[t * k + j0 + j] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = wt * __uint_as_float(v[j][i >> 2][i & 3]);
                z[0][i] = j0 + j < k ? z[0][i] + p : z[0][i];
            }
        }
    }
    if (failed) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[0][i] = __uint_as_float(0x7FC00000u);
    }
    row.finish(a.tail, t, c0, z, sm.lds);
}

template <int GS, int BITS>
__global__ __launch_bounds__(kFewThreads, 1) void moe_layer_few_experts(LayerArgs a) {
    __shared__ FewSmem<GS, BITS> sm;
    make_lists(a, sm);
    // usually one range of each phase; more if workgroups have not started yet
    for (int r = sm.own[0] ? blockIdx.x : take(sm, a.claim_gateup, kRanges); r >= 0;)
        r = run_range<GS, BITS, false>(a, sm, r, a.claim_gateup) ? take(sm, a.claim_gateup, kRanges) : -1;
    for (int r = sm.own[1] ? blockIdx.x : take(sm, a.claim_down, kRanges); r >= 0;)
        r = run_range<GS, BITS, true>(a, sm, r, a.claim_down) ? take(sm, a.claim_down, kRanges) : -1;
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
