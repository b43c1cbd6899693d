// The k largest of a row of logits, by one wave.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

// Largest v of the wave, in every lane: within 16-lane rows by DPP moves (lane
// i ^ 1, i ^ 2, then mirrors of 8 and 16 once quads agree), across rows by
// scalar reads.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = max_dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
    v = max_dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
    v = max_dpp<0x141>(v);  // row_half_mirror
    v = max_dpp<0x140>(v);  // row_mirror
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < 64; r += 16)
        m = fmaxf(m, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), r)));
    return m;
}

struct TopK {
    int32_t id;    // lane j < k: the j-th largest logit's expert
    float weight;  // and its weight
};

// Lane l holds logits l, l + 64, ... in v (anything past E; NaN ranks as -inf).
// Each of the k rounds takes the largest logit left; among equal ones the lowest
// id, found from the ballots of the lanes that hold it.  Then the weights:
// softmax over the k, each times its expert's factor (expert_scale may be
// nullptr).  All lanes of the wave take part; 1 <= k <= min(E, 64), E <= 64 PER.
template <int PER>
__device__ __forceinline__ TopK wave_topk(float (&v)[PER], int E, int k, const float* expert_scale) {
    const int lane = threadIdx.x & 63;
    uint32_t left = 0;  // bit i: logit lane + 64 i exists and is not yet chosen
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (v[i] != v[i]) v[i] = -INFINITY;
        if (lane + 64 * i < E) left |= 1u << i;
    }
    float mine = -INFINITY, top = 0.f;
    int32_t my_id = 0;
    for (int j = 0; j < k; ++j) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = left >> i & 1u ? fmaxf(m, v[i]) : m;
        m = wave_max(m);
        int id = -1;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const uint64_t holds = __ballot((left >> i & 1u) && v[i] == m);
            if (holds) id = 64 * i + __ffsll(static_cast<unsigned long long>(holds)) - 1;
        }
        if ((id & 63) == lane) left &= ~(1u << (id >> 6));
        if (j == 0) top = m;
        if (lane == j) {
            mine = m;
            my_id = id;
        }
    }
    // lanes 0..k-1 hold the chosen logits in order
    const float ex = lane < k ? expf(mine - top) : 0.f;
    float sum = ex;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
    sum = __shfl(sum, 0);  // one rounding of the sum for every lane
    const float w = ex / sum;
    return TopK{my_id, expert_scale && lane < k ? w * expert_scale[my_id] : w};
}

// Largest v of the wave as a scalar; rows of 16 lanes as above, then each row's to
// the next and the first two rows' to the rest.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
    return max(v, static_cast<uint32_t>(
                      __builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    v = umax_dpp<0xB1, 0xF>(v);
    v = umax_dpp<0x4E, 0xF>(v);
    v = umax_dpp<0x141, 0xF>(v);
    v = umax_dpp<0x140, 0xF>(v);
    v = umax_dpp<0x142, 0xA>(v);  // row_bcast:15
    v = umax_dpp<0x143, 0xC>(v);  // row_bcast:31
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// The same for E <= 128 and k <= 16, without the factors, in the few-token layer (8 of
// 128: 1 us less there; the router's own launch has not been measured with it).  A
// lane's two logits lie in order, as keys that order like the floats and leave 0 for
// "none", so a round looks at one value a lane.  Bit for bit the same.
__device__ __forceinline__ TopK wave_topk_128(float v0, float v1, int E, int k) {
    const int lane = threadIdx.x & 63;
    auto key = [](float v) {
        const uint32_t u = __float_as_uint(v != v ? -INFINITY : v == 0.f ? 0.f : v);
        return u >> 31 ? ~u : u | 0x80000000u;
    };
    uint32_t a = lane < E ? key(v0) : 0, b = lane + 64 < E ? key(v1) : 0;
    const bool swap = b > a;
    if (swap) {
        const uint32_t t = a;
        a = b;
        b = t;
    }
    bool second = swap;  // a is logit lane + 64
    int mine = 0, my_id = 0;
    for (int j = 0; j < k; ++j) {
        const uint32_t m = wave_umax(a);
        const uint64_t lo = __ballot(a == m && !second), hi = __ballot(a == m && second);
        const int id = lo ? __ffsll(static_cast<unsigned long long>(lo)) - 1
                          : 63 + __ffsll(static_cast<unsigned long long>(hi));
        if (lane == j) {
            mine = static_cast<int>(m);
            my_id = id;
        }
        if (lane == (id & 63)) {
            a = b;
            b = 0;
            second = !second;
        }
    }
    const uint32_t u = static_cast<uint32_t>(mine);
    const float logit = __uint_as_float(u >> 31 ? u & 0x7FFFFFFFu : ~u);
    const float top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(logit), 0));
    const float ex = lane < k ? expf(logit - top) : 0.f;
    float sum = ex;  // over 16 lanes, in wave_topk's order
    sum += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(sum), 0xB1, 0xF, 0xF, true));
    sum += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(sum), 0x4E, 0xF, 0xF, true));
    sum += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(sum), 0x141, 0xF, 0xF, true));
    sum += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(sum), 0x140, 0xF, 0xF, true));
    return TopK{my_id, ex / sum};
}

}  // namespace
}  // namespace moe
