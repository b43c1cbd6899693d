// A whole mixture-of-experts layer for at most 16 tokens in two launches.
//
//   1. moe_layer_few_route: logits = rstd (x . Wr^T), one workgroup an expert;
//      n = rms(x) w, one workgroup a token, as bf16 hi + lo (16 bits) in the order
//      of the matmul operand, with its sums over chains of columns; the second
//      launch's counters are cleared.
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
// The codes are exact operands (OFF + q); with P = x . (OFF + q) - OFF X over a
// chain of columns, X the chain's sum of x, the accumulator takes s P + b X.
//
// A unit is 32 weight rows (gate|up: 16 columns of h, both halves; down: 32
// output columns) by all of K, cut over SPLIT waves that hold at most 4 chunks of
// 128 columns each, so that a wave keeps its slice of the tile's activations in
// registers for all units of the tile.  Units are numbered tile by tile, and
// workgroup b takes the b-th of 256 equal ranges of them.
//
// Order between the phases without a barrier.  A range is taken by an exchange on
// its own flag.  A workgroup takes its own range, then any range that it finds
// untaken, and only when all ranges of a phase are taken does it go on to the
// next phase, where it may wait for counters (units done per tile).  So whoever
// waits waits for running workgroups of an earlier phase, and the first phase
// waits for nobody: every wait ends, however few workgroups the GPU holds at
// once.  (Waits are also bounded: a workspace that another call writes to gives
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
constexpr int kSpinLimit = 1 << 22;                       // polls of about 1 us

template <int GS>
constexpr int kChainCols = Geo<GS>::kChain;

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
    const int chain = a.gs == 32 ? 32 : 64, per = chain / 8;  // threads of a chain
    uint16_t* const n = a.n + static_cast<size_t>(2 * t) * H;
    float* const sums = a.nsum + static_cast<size_t>(2 * t) * (H / chain);
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
            if (c % chain == 0) {
                sums[c / chain] = shi;
                sums[H / chain + c / chain] = slo;
            }
        }
    }
}

// ----------------------------------------------------------- second launch
// The lists that every workgroup makes of the chosen experts.
struct Lists {
    int32_t tiles;                             // tiles in all
    uint16_t rows[kMaxSlots][kTileRows];       // assignments t * k + j of a tile's rows
    uint16_t expert[kMaxSlots];                // a tile's expert
    uint8_t count[kMaxSlots];                  // and its rows
    uint16_t slot_tile[kMaxSlots];             // the tile of an assignment
    float weight[kMaxSlots];                   // its routing weight
};

template <int GS, int BITS>
struct alignas(16) FewSmem {
    uint32_t w[kWaves][2 * 16 * 4 * BITS];          // weight transposition, a wave's own
    uint16_t tables[2][8 * 4096 / GS * 8];          // scales and biases of the units at work, of the next ones
    float xs[kWaves][kChunks * Geo<GS>::kChains][16];  // chain sums of a wave's slice, per operand row
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
    int32_t pick;
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

// Takes flag `own`, or with own < 0 any untaken one of n <= kFewThreads flags; -1
// once all are taken.  Called by the whole workgroup.
template <class Smem>
__device__ __forceinline__ int take(Smem& sm, int32_t* flags, int n, int own) {
    for (;;) {
        __syncthreads();
        if (threadIdx.x == 0) sm.pick = own >= 0 ? own : INT32_MAX;
        __syncthreads();
        if (own < 0) {
            const int i = threadIdx.x;
            if (i < n && !__hip_atomic_load(flags + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
                atomicMin(&sm.pick, i);
            __syncthreads();
            if (sm.pick == INT32_MAX) return -1;
        }
        if (threadIdx.x == 0) {
            const int i = sm.pick;
            if (__hip_atomic_exchange(flags + i, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) sm.pick = -1;
        }
        __syncthreads();
        const int got = sm.pick;
        if (got >= 0) return got;
        own = -1;  // another workgroup was first: look for what is left
    }
}

// top-k of all tokens, then the tiles in expert order (rows in token order).
template <class Smem>
__device__ __forceinline__ void make_lists(const LayerArgs& a, Smem& sm) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int T = a.T, k = a.k, E = a.E;
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
        sm.l.rows[tile][rank % kTileRows] = static_cast<uint16_t>(s);
        sm.l.slot_tile[s] = static_cast<uint16_t>(tile);
        if (rank % kTileRows == 0) {
            sm.l.expert[tile] = static_cast<uint16_t>(e);
            sm.l.count[tile] = static_cast<uint8_t>(min(kTileRows, __popc(m) - rank));
        }
    }
    __syncthreads();
}

// One phase (kDown: the down matmul, else gate|up) of one range of units.
template <int GS, int BITS, bool kDown>
__device__ __forceinline__ void run_range(const LayerArgs& a, FewSmem<GS, BITS>& sm, int range) {
    constexpr int CH = Geo<GS>::kChains, MPG = Geo<GS>::kSlices, SH = Geo<GS>::kShift;
    constexpr int OFF = kCodeOffset<BITS, true>;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, lr = lane & 15;
    const int K = kDown ? a.I : a.H, G = K / GS, row_words = K / 32 * BITS, chains = K / kChainCols<GS>;
    const int upt = kDown ? a.H / 32 : a.I / 16;  // units of a tile
    const int nch = (K + 127) / 128;
    const int log_split = nch <= 4 ? 0 : nch <= 8 ? 1 : nch <= 16 ? 2 : 3, split = 1 << log_split;
    const int nu = kWaves >> log_split;           // units at work at a time
    const int wu = wave >> log_split, ws = wave & (split - 1);
    const int ch0 = nch * ws >> log_split, nc = (nch * (ws + 1) >> log_split) - ch0;  // this wave's chunks, <= 4
    const int N = sm.l.tiles * upt, groups = kRanges * nu;
    auto first = [&](int g) { return static_cast<int>(static_cast<int64_t>(N) * g / groups); };
    const int lo = first(range * nu), hi = first((range + 1) * nu);
    if (lo == hi) return;
    const int u0 = first(range * nu + wu), u1 = first(range * nu + wu + 1);
    int steps = 0;
    for (int i = 0; i < nu; ++i) steps = max(steps, first(range * nu + i + 1) - first(range * nu + i));

    const uint32_t* const w = kDown ? a.w_d : a.w_gu;
    const uint16_t* const s16 = kDown ? a.s_d : a.s_gu;
    const uint16_t* const b16 = kDown ? a.b_d : a.b_gu;
    // the first weight row of block b of unit u
    auto row_of = [&](int u, int b) {
        const int tile = u / upt, i = u - tile * upt;
        const size_t e = sm.l.expert[tile];
        return kDown ? e * a.H + 32 * i + 16 * b : e * 2 * a.I + 16 * i + (b ? a.I : 0);
    };
    WaveW<2, GS, BITS> ww;
    auto aim = [&](int u) {  // ww loads unit u from now on
        const uint32_t* blk[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const size_t r = row_of(u, b);
            const uint32_t rl = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(r)),
                           rh = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(r >> 32));
            blk[b] = w + ((static_cast<size_t>(rh) << 32 | rl)) * row_words;
        }
        ww.init(sm.w[wave], blk, row_words);
    };
    u32x4 rv[kChunks][2][BITS / 4];
    if (u0 < u1) {
        aim(u0);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (i < nc) ww.load(ch0 + i, rv[i]);
    }
    // tables: per unit the scales and then the biases of its 2 x 16 rows, 2 G
    // pieces of 16 bytes a block; at most 2 pieces a thread
    u32x4 tv[2];
    auto load_tables = [&](int step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = tid + kFewThreads * h, i = p / (8 * G), r = p - i * 8 * G, seg = r / (2 * G), at = r - seg * 2 * G;
            const int u = first(range * nu + min(i, nu - 1)) + step;
            if (i < nu && u < first(range * nu + i + 1))
                tv[h] = *reinterpret_cast<const u32x4*>((seg < 2 ? s16 : b16) + row_of(u, seg & 1) * G + 8 * at);
        }
    };
    auto store_tables = [&](int step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = tid + kFewThreads * h;
            if (p < nu * 8 * G) *reinterpret_cast<u32x4*>(sm.tables[step & 1] + 8 * p) = tv[h];
        }
    };
    load_tables(0);
    store_tables(0);

    const CodeConsts<OFF> kc = code_consts<OFF>(a.zero);
    const int parts_row = 2 * K;  // values of a row's hi and lo parts
    const Rsrc rx = make_rsrc(kDown ? a.h : a.n, 2u * parts_row * static_cast<uint32_t>(kDown ? a.T * a.k : a.T));
    u32x4 x[kChunks][4];
    int tile_now = -1;
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        const int u = u0 + step;
        const bool busy = u < u1, more = u + 1 < u1;
        if (step + 1 < steps) load_tables(step + 1);
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (busy) {
            const int tile = __builtin_amdgcn_readfirstlane(u / upt);
            if (tile != tile_now) {
                tile_now = tile;
                if constexpr (kDown) {
                    if (!wait_for(a.done_gateup + tile, a.I / 16)) give_up(a);
                }
                // operand row lr: part lr / 8 of the tile's row lr % 8; rows past the
                // tile and columns past K are zeros
                const int count = sm.l.count[tile], r = lr & 7;
                const int slot = sm.l.rows[tile][min(r, count - 1)];
                const uint32_t base = 2u * (static_cast<uint32_t>(kDown ? slot : slot / a.k) * parts_row + (lr >> 3) * K);
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int col = 128 * (ch0 + i) +
                                        (kChainCols<GS> == 64 ? 64 * (s >> 1) + 16 * q + 8 * (s & 1) : 32 * s + 8 * q);
                        const uint32_t at = i < nc && r < count && col < K ? base + 2u * col : 0xFFFFFFF0u;
                        x[i][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, kDown ? kSc1 : 0));
                    }
                // chain sums of the wave's slice
#pragma unroll
                for (int i = 0; i < kChunks * CH / 4; ++i) {
                    const int p = lane + 64 * i, c = p >> 4, row = p & 15, rr = row & 7;
                    const int chain = ch0 * CH + c;
                    float sum = 0.f;
                    if (c < nc * CH && chain < chains && rr < count) {
                        const int sl = sm.l.rows[tile][rr];
                        if constexpr (kDown) {
                            const int blocks = kChainCols<GS> / 16;
                            const Rsrc rs = make_rsrc(a.hsum, 8u * (K / 16) * static_cast<uint32_t>(a.T * a.k));
                            const uint32_t at = 4u * ((2 * sl + (row >> 3)) * (K / 16) + chain * blocks);
                            float v[kChainCols<GS> / 16];
#pragma unroll
                            for (int b = 0; b < blocks; ++b)
                                v[b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at + 4 * b, 0, kSc1));
#pragma unroll
                            for (int b = 0; b < blocks; ++b) sum += v[b];
                        } else {
                            sum = a.nsum[static_cast<size_t>(2 * (sl / a.k) + (row >> 3)) * chains + chain];
                        }
                    }
                    sm.xs[wave][c][row] = sum;
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (more) aim(u + 1);
            const uint16_t* const ts = sm.tables[step & 1] + wu * 64 * G + lr * G;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                if (i < nc) {
                    chunk_fence();
                    ww.put(rv[i]);
                    if (more) ww.load(ch0 + i, rv[i]);
                    __builtin_amdgcn_wave_barrier();
                    WLane<BITS> wv[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) wv[b] = ww.get(b, lr, q);
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const f32x4 X = *reinterpret_cast<const f32x4*>(&sm.xs[wave][i * CH + j][4 * q]);
                        const int g = min(((ch0 + i) * CH + j) >> SH, G - 1);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            f32x4 p;
#pragma unroll
                            for (int v = 0; v < 4; ++v) p[v] = -static_cast<float>(OFF) * X[v];
#pragma unroll
                            for (int m = 0; m < MPG; ++m)
                                p = mfma16(x[i][j * MPG + m], slice_operand<BITS, OFF>(wv[b], j * MPG + m, kc), p);
                            const float s = bf16_to_f32(ts[16 * b * G + g]), bias = bf16_to_f32(ts[(32 + 16 * b) * G + g]);
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[b][v] = fmaf(bias, X[v], fmaf(s, p[v], acc[b][v]));
                        }
                    }
                    __builtin_amdgcn_wave_barrier();
                }
            }
            // operand rows 8..15 are the lo parts of rows 0..7
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    acc[b][v] += __shfl_xor(acc[b][v], 32);
                    if (lane < 32) sm.red[step & 1][wave][b][4 * q + v][lr] = acc[b][v];
                }
        }
        if (step + 1 < steps) store_tables(step + 1);
        __syncthreads();
        // the units' outputs: 128 of gate|up, 256 of down each
        constexpr int kOut = kDown ? 256 : 128;
        for (int p = tid; p < nu * kOut; p += kFewThreads) {
            const int i = p / kOut, r = (p / (kOut / kTileRows)) % kTileRows, c = p % (kOut / kTileRows);
            const int uu = first(range * nu + i) + step;
            if (uu >= first(range * nu + i + 1)) continue;
            const int tile = uu / upt, col = uu - tile * upt;
            if (r >= sm.l.count[tile]) continue;
            const size_t slot = sm.l.rows[tile][r];
            float o[2] = {0.f, 0.f};
            for (int v = 0; v < split; ++v) {
                const auto& red = sm.red[step & 1][(i << log_split) + v];
                if constexpr (kDown) {
                    o[0] += red[c >> 4][r][c & 15];
                } else {
                    o[0] += red[0][r][c];
                    o[1] += red[1][r][c];
                }
            }
            if constexpr (kDown) {
                const Rsrc ry = make_rsrc(a.y + slot * a.H, 4u * a.H);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), ry, 4 * (32 * col + c), 0, kSc1);
            } else {
                const float hv = (a.swiglu ? silu(o[0]) : gelu_tanh(o[0])) * o[1];
                const uint16_t hi16 = f32_to_bf16(hv), lo16 = f32_to_bf16(hv - bf16_to_f32(hi16));
                const Rsrc rh = make_rsrc(a.h, 4u * a.I * static_cast<uint32_t>(a.T * a.k));
                const uint32_t at = 2u * (static_cast<uint32_t>(slot) * 2 * a.I + 16 * col + (c & 8) + permuted_pos(c & 7));
                __builtin_amdgcn_raw_buffer_store_b16(hi16, rh, at, 0, kSc1);
                __builtin_amdgcn_raw_buffer_store_b16(lo16, rh, at + 2u * a.I, 0, kSc1);
                const float shi = sum16(bf16_to_f32(hi16)), slo = sum16(bf16_to_f32(lo16));
                const Rsrc rs = make_rsrc(a.hsum, 8u * (a.I / 16) * static_cast<uint32_t>(a.T * a.k));
                const uint32_t sat = 4u * (static_cast<uint32_t>(slot) * 2 * (a.I / 16) + col);
                if (c < 2)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(c ? slo : shi), rs, sat + (c ? 4u * (a.I / 16) : 0), 0,
                                                          kSc1);
            }
        }
    }
    // the range is done once its stores have been acknowledged
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int t0 = lo / upt + tid;
    if (t0 * upt < hi) {
        const int n = min(hi, (t0 + 1) * upt) - max(lo, t0 * upt);
        __hip_atomic_fetch_add((kDown ? a.done_down : a.done_gateup) + t0, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// out and normed of one token.
template <int GS, int BITS>
__device__ __forceinline__ void finish_token(const LayerArgs& a, FewSmem<GS, BITS>& sm, int t) {
    const int c0 = 8 * threadIdx.x, k = a.k, H = a.H;
    norm::Row<kWaves, 1, 8, -1> row;
    row.load(a.tail, t, c0);
    if (static_cast<int>(threadIdx.x) < k)  // lanes of the first wave
        if (!wait_for(a.done_down + sm.l.slot_tile[t * k + threadIdx.x], H / 32)) give_up(a);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const bool ok = !__hip_atomic_load(a.failed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
    if (!ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[0][i] = __uint_as_float(0x7FC00000u);
    }
    row.finish(a.tail, t, c0, z, sm.lds);
}

template <int GS, int BITS>
__global__ __launch_bounds__(kFewThreads, 1) void moe_layer_few_experts(LayerArgs a) {
    __shared__ FewSmem<GS, BITS> sm;
    make_lists(a, sm);
    for (int r = take(sm, a.claim_gateup, kRanges, blockIdx.x); r >= 0; r = take(sm, a.claim_gateup, kRanges, -1))
        run_range<GS, BITS, false>(a, sm, r);
    for (int r = take(sm, a.claim_down, kRanges, blockIdx.x); r >= 0; r = take(sm, a.claim_down, kRanges, -1))
        run_range<GS, BITS, true>(a, sm, r);
    for (int t = take(sm, a.claim_token, a.T, blockIdx.x % a.T); t >= 0; t = take(sm, a.claim_token, a.T, -1))
        finish_token(a, sm, t);
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
