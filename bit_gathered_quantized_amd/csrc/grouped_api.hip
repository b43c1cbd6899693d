// C ABI of the products grouped by expert and of the microscaled values: argument checks,
// then the launches.
#include <limits.h>

#include <numeric>

#include "moe_internal.h"

namespace {

bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool plain_type(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_FP32; }
// A row stride of an input: 16-byte steps, 32-bit offsets inside a tile.
bool input_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s <= MOE_GROUPED_MAX_STRIDE; }

// The memory of an operand: `rows` runs of `width` bytes, `stride` bytes from one to the next.
struct Memory {
    uintptr_t at;
    int64_t span;    // from the first byte past the last
    int64_t width;
    int64_t stride;  // 0: one run
};
Memory memory(const void* p, int64_t rows, int64_t width, int64_t stride) {
    if (!p || rows < 1) return {0, 0, 0, 0};
    return {reinterpret_cast<uintptr_t>(p), (rows - 1) * stride + width, width, rows > 1 ? stride : 0};
}
Memory memory(const void* p, int64_t bytes) { return memory(p, 1, bytes, 0); }

// Whether two operands share bytes.  Their runs repeat with the strides' common divisor: one operand
// may lie between the other's rows.
bool meet(const Memory& a, const Memory& b) {
    if (a.span == 0 || b.span == 0 || a.at >= b.at + b.span || b.at >= a.at + a.span) return false;
    const int64_t step = std::gcd(a.stride, b.stride);
    if (step == 0) return true;  // two runs
    const int64_t ahead = b.at >= a.at ? static_cast<int64_t>((b.at - a.at) % step) : (step - static_cast<int64_t>((a.at - b.at) % step)) % step;
    return ahead < a.width || step - ahead < b.width;
}

// The same for w, an expert at a time where the memory of all of them meets it.
bool meet_weights(const Memory& b, const moe_grouped* g) {
    const bool kn = g->flags & MOE_G_W_KN;
    const int64_t rows = kn ? g->K : g->N, width = 2 * static_cast<int64_t>(kn ? g->N : g->K), stride = 2 * g->w_stride;
    const int64_t expert = 2 * (g->w_expert_stride < int64_t{1} << 48 ? g->w_expert_stride : int64_t{1} << 48);
    if (!meet(memory(g->w, (g->E - 1) * expert + (rows - 1) * stride + width), b)) return false;
    for (int e = 0; e < g->E; ++e)
        if (meet(memory(static_cast<const char*>(g->w) + e * expert, rows, width, stride), b)) return true;
    return false;
}

moe_status check_sizes(int32_t A, int32_t E, int32_t N, int32_t K, int32_t step) {
    if (A < 0 || A >= 1 << 30 || E < 1 || N < 1 || K < 1 || N % 8 || K % step) return MOE_ERR_SHAPE;
    if (E > MOE_MAX_EXPERTS || N > MOE_GROUPED_MAX_DIM || K > MOE_GROUPED_MAX_DIM) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status check(const moe_grouped* g) {
    if (!g) return MOE_ERR_NULL;
    const bool xm = g->x_type == MOE_T_MXFP4, wm = g->w_type == MOE_T_MXFP4, kn = g->flags & MOE_G_W_KN;
    if ((!xm && g->x_type != MOE_T_BF16) || (!wm && g->w_type != MOE_T_BF16) || (xm && !wm) || !plain_type(g->out_type) ||
        (g->flags & ~MOE_G_W_KN) || (kn && wm))
        return MOE_ERR_UNSUPPORTED;
    const moe_status st = check_sizes(g->A, g->E, g->N, g->K, wm ? 32 : 8);
    if (st != MOE_OK) return st;
    // strips of rows by units of 32 columns: the kernels' sums over them stay within 32 bits
    const int64_t strip = g->A <= moe::kGroupedLowRows * static_cast<int64_t>(g->E) ? 32 : 128;
    if ((g->A / strip + g->E) * ((g->N + 31) / 32) >= 1 << 24) return MOE_ERR_SHAPE;
    if (!xm && !input_stride(g->x_stride)) return MOE_ERR_SHAPE;
    if (!wm && (!input_stride(g->w_stride) || g->w_expert_stride < 0 || g->w_expert_stride % 8)) return MOE_ERR_SHAPE;
    if (g->out_stride < g->N || g->out_stride > MOE_GROUPED_MAX_STRIDE || g->out_stride % (g->out_type == MOE_T_FP32 ? 4 : 8))
        return MOE_ERR_SHAPE;
    if (g->A == 0) return MOE_OK;
    if (!g->x || !g->w || !g->out || (!g->offsets && g->E > 1) || (xm && !g->x_scales) || (wm && !g->w_scales))
        return MOE_ERR_NULL;
    if (!on(g->x, 16) || !on(g->w, 16) || !on(g->out, 16) || !on(g->offsets, 4)) return MOE_ERR_ALIGN;
    const int64_t A = g->A, K = g->K, size = g->out_type == MOE_T_FP32 ? 4 : 2, weights = static_cast<int64_t>(g->E) * g->N;
    const Memory out = memory(g->out, A, size * g->N, size * g->out_stride);
    if (meet(out, xm ? memory(g->x, A * K / 2) : memory(g->x, A, 2 * K, 2 * g->x_stride)) ||
        (wm ? meet(out, memory(g->w, weights * K / 2)) : meet_weights(out, g)) ||
        (xm && meet(out, memory(g->x_scales, A * K / 32))) || (wm && meet(out, memory(g->w_scales, weights * K / 32))) ||
        meet(out, memory(g->offsets, 4 * (static_cast<int64_t>(g->E) + 1))))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Sizes of a gradient of the weights: what the workspace depends on.
moe_status check_grad_sizes(const moe_grouped_grad* g) {
    const moe_status st = check_sizes(g->A, g->E, g->N, g->K, 8);
    if (st != MOE_OK) return st;
    return static_cast<int64_t>(g->E) * ((g->N + 63) / 64) * ((g->K + 63) / 64) >= INT32_MAX ? MOE_ERR_SHAPE : MOE_OK;
}

moe_status check(const moe_grouped_grad* g) {
    if (!g) return MOE_ERR_NULL;
    if (!plain_type(g->out_type)) return MOE_ERR_UNSUPPORTED;
    const moe_status st = check_grad_sizes(g);
    if (st != MOE_OK) return st;
    if (!input_stride(g->dy_stride) || !input_stride(g->x_stride)) return MOE_ERR_SHAPE;
    // without rows dw is zeros all the same
    if (!g->dw || (!g->offsets && g->E > 1) || (g->A > 0 && (!g->dy || !g->x))) return MOE_ERR_NULL;
    if (!on(g->dy, 16) || !on(g->x, 16) || !on(g->dw, 16) || !on(g->offsets, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

// Whether dw or the workspace (`ws_bytes` that the call uses) lies on an operand or on the other.
bool overlaps(const moe_grouped_grad* g, const void* ws, size_t ws_bytes) {
    const int64_t N = g->N, K = g->K;
    const Memory dw = memory(g->dw, (g->out_type == MOE_T_FP32 ? 4 : 2) * g->E * N * K);
    const Memory space = memory(ws_bytes > 0 ? ws : nullptr, static_cast<int64_t>(ws_bytes));
    const Memory inputs[] = {memory(g->dy, g->A, 2 * N, 2 * g->dy_stride), memory(g->x, g->A, 2 * K, 2 * g->x_stride),
                             memory(g->offsets, 4 * (static_cast<int64_t>(g->E) + 1))};
    for (const Memory& m : inputs)
        if (meet(dw, m) || meet(space, m)) return true;
    return meet(dw, space);
}

moe_status check(const moe_mx* q, bool quantize) {
    if (!q) return MOE_ERR_NULL;
    if (!plain_type(q->type) || (q->flags & ~(MOE_Q_GELU | MOE_Q_SILU)) || q->flags == (MOE_Q_GELU | MOE_Q_SILU) ||
        (!quantize && q->flags))
        return MOE_ERR_UNSUPPORTED;
    if (q->R < 0 || q->K < 1 || q->K % 32) return MOE_ERR_SHAPE;
    if (q->K > MOE_GROUPED_MAX_DIM) return MOE_ERR_UNSUPPORTED;
    if (q->R > ((int64_t{1} << 34) - 1) / q->K) return MOE_ERR_SHAPE;
    const int64_t row = q->flags ? 2 * static_cast<int64_t>(q->K) : q->K;
    if (q->stride < row || q->stride % (q->type == MOE_T_FP32 ? 4 : 8) || q->stride > int64_t{1} << 30) return MOE_ERR_SHAPE;
    if (q->R == 0) return MOE_OK;
    if (!q->values || !q->codes || !q->scales) return MOE_ERR_NULL;
    if (!on(q->values, 16) || !on(q->codes, 16)) return MOE_ERR_ALIGN;
    // either way a thread reads what another may have written by then
    const int64_t size = q->type == MOE_T_FP32 ? 4 : 2;
    const Memory values = memory(q->values, q->R, size * row, size * q->stride), codes = memory(q->codes, q->R * q->K / 2),
                 scales = memory(q->scales, q->R * q->K / 32);
    return meet(values, codes) || meet(values, scales) || meet(codes, scales) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe::MxArgs mx_args(const moe_mx* q) {
    moe::MxArgs a = {};
    a.R = q->R;
    a.K = q->K;
    a.f32 = q->type == MOE_T_FP32;
    a.glu = q->flags & MOE_Q_GELU ? 1 : q->flags & MOE_Q_SILU ? 2 : 0;
    a.values = q->values;
    a.codes = q->codes;
    a.scales = q->scales;
    a.stride = q->stride * (a.f32 ? 4 : 2);
    return a;
}

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(const moe_grouped* g, void* stream) {
    const moe_status st = check(g);
    if (st != MOE_OK || g->A == 0) return st;
    moe::GroupedArgs a = {};
    a.A = g->A;
    a.E = g->E;
    a.N = g->N;
    a.K = g->K;
    a.w_kn = g->flags & MOE_G_W_KN;
    a.out_f32 = g->out_type == MOE_T_FP32;
    a.offsets = g->offsets;
    a.x = g->x;
    a.w = g->w;
    a.xs = g->x_type == MOE_T_MXFP4 ? g->x_scales : nullptr;
    a.ws = g->w_type == MOE_T_MXFP4 ? g->w_scales : nullptr;
    a.out = g->out;
    a.x_stride = 2 * g->x_stride;
    a.w_stride = 2 * g->w_stride;
    a.w_expert = 2 * g->w_expert_stride;
    a.out_stride = g->out_stride * (a.out_f32 ? 4 : 2);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = moe::grouped_few_rows(a)    ? moe::launch_grouped_few(a, s)
                         : g->w_type == MOE_T_BF16 ? moe::launch_grouped_bf16(a, s)
                         : g->x_type == MOE_T_BF16 ? moe::launch_grouped_bf16_mx(a, s)
                                                   : moe::launch_grouped_mx(a, s);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_grouped_dw_workspace_bytes(const moe_grouped_grad* g) {
    return g && check_grad_sizes(g) == MOE_OK ? moe::grouped_dw_workspace(g->A, g->E, g->N, g->K) : 0;
}

moe_status moe_grouped_matmul_dw(const moe_grouped_grad* g, void* ws, size_t ws_bytes, void* stream) {
    const moe_status st = check(g);
    if (st != MOE_OK) return st;
    const size_t need = moe::grouped_dw_workspace(g->A, g->E, g->N, g->K);
    if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    if (need > 0 && !on(ws, 256)) return MOE_ERR_ALIGN;
    if (overlaps(g, ws, need)) return MOE_ERR_UNSUPPORTED;
    moe::GroupedGradArgs a = {};
    a.A = g->A;
    a.E = g->E;
    a.N = g->N;
    a.K = g->K;
    a.out_f32 = g->out_type == MOE_T_FP32;
    a.offsets = g->offsets;
    a.dy = g->dy;
    a.x = g->x;
    a.dw = g->dw;
    a.dy_stride = 2 * g->dy_stride;
    a.x_stride = 2 * g->x_stride;
    a.ws = static_cast<float*>(ws);
    return moe::launch_grouped_dw(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_mx_quantize(const moe_mx* q, void* stream) {
    const moe_status st = check(q, true);
    if (st != MOE_OK || q->R == 0) return st;
    return moe::launch_mx_quantize(mx_args(q), static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_mx_dequantize(const moe_mx* q, void* stream) {
    const moe_status st = check(q, false);
    if (st != MOE_OK || q->R == 0) return st;
    return moe::launch_mx_dequantize(mx_args(q), static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
