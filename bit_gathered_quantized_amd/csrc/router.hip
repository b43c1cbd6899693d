// Device router: softmax top-k with renormalised weights, the step that feeds
// the route/sort kernel.  The pages do not define the router; this is the
// usual top-k softmax gate (the fused top-k candidate selection of the
// mlx-node PR #168 page is its nearest relative there).
//
// One wave per token (topk.h): lane l holds logits l, l + 64, ...  Weights: w_j =
// exp(l_j - m) / sum over the k chosen of exp(l_i - m), with m the largest logit
// -- the softmax over all E experts renormalised over the chosen k (the full
// denominator cancels).  The sum runs in a fixed order, so results are
// deterministic.  NaN logits rank as -inf.
#include "topk.h"

namespace moe {
namespace {

constexpr int kRouterTokensPerBlock = 4;

template <int PER>
__global__ __launch_bounds__(64 * kRouterTokensPerBlock) void moe_router_topk_kernel(
    const float* __restrict__ logits, int32_t T, int32_t E, int32_t k,
    const float* __restrict__ expert_scale, int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const uint32_t t = grid_index() * kRouterTokensPerBlock + (threadIdx.x >> 6);
    if (t >= static_cast<uint32_t>(T)) return;  // whole wave; no barrier follows
    const float* row = logits + static_cast<size_t>(t) * E;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
    const TopK c = wave_topk<PER>(v, E, k, expert_scale);
    if (lane < k) {
        ids[static_cast<size_t>(t) * k + lane] = c.id;
        weights[static_cast<size_t>(t) * k + lane] = c.weight;
    }
}

}  // namespace

hipError_t launch_router_topk(const float* logits, int32_t T, int32_t E, int32_t k, const float* expert_scale,
                              int32_t* ids, float* weights, hipStream_t stream) {
    const dim3 grid = grid_of((static_cast<int64_t>(T) + kRouterTokensPerBlock - 1) / kRouterTokensPerBlock);
    const dim3 block(64 * kRouterTokensPerBlock);
    if (E <= 128)
        hipLaunchKernelGGL(moe_router_topk_kernel<2>, grid, block, 0, stream, logits, T, E, k, expert_scale, ids, weights);
    else if (E <= 256)
        hipLaunchKernelGGL(moe_router_topk_kernel<4>, grid, block, 0, stream, logits, T, E, k, expert_scale, ids, weights);
    else if (E <= 512)
        hipLaunchKernelGGL(moe_router_topk_kernel<8>, grid, block, 0, stream, logits, T, E, k, expert_scale, ids, weights);
    else
        hipLaunchKernelGGL(moe_router_topk_kernel<MOE_MAX_EXPERTS / 64>, grid, block, 0, stream, logits, T, E, k,
                           expert_scale, ids, weights);
    return hipGetLastError();
}

}  // namespace moe
