// C ABI of libmoeffn: argument checks, workspace layout and the launch
// sequence of the forward.  Nothing here allocates, frees or waits on the
// device; everything is enqueued on the caller's stream.
#include <limits.h>
#include <stddef.h>

#include <mutex>

#include "layer_cut.h"
#include "moe_internal.h"

// The built-in workspace of moe_expert_ffn_forward_noalloc: one copy per
// GPU, alive until the process ends.  Host code never passes `scratch`
// itself to a kernel or a copy (in host code it is a stand-in, not a device
// address): it takes the device address from hipGetSymbolAddress, once per
// device, with that device current.
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's scratch array (looked up on the
// first call on that device), or nullptr with *err set.
void* scratch_for_current_device(hipError_t* err) {
    int dev = 0;
    *err = hipGetDevice(&dev);
    if (*err != hipSuccess) return nullptr;
    if (dev < 0 || dev >= kMaxDevices) {
        *err = hipErrorInvalidDevice;
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (g_scratch_ptr[dev] == nullptr) {
        void* ptr = nullptr;
        *err = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (*err != hipSuccess) return nullptr;
        g_scratch_ptr[dev] = ptr;
    }
    return g_scratch_ptr[dev];
}

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Wide tiles of at most 64 rows (4 row blocks per wave), or 32 with an fp32 h (the
// down matmul carries two activation parts) or 8-bit codes (twice the weight words
// in flight).
int32_t big_rows(const moe_problem* p) {
    return (p->flags & MOE_F_FP32_INTERMEDIATE) || p->bits == 8 ? moe::kBmBigF32 : moe::kBmBig;
}

// Whether a one-dimensional launch of `groups` workgroups has fewer than 2^32 threads.
// HIP does not refuse more: it starts what is left of their number modulo 2^32.
bool fits_launch(int64_t groups, int64_t threads) { return groups * threads < (int64_t{1} << 32); }

// Shape checks shared by the forward's size queries and the forward itself.
moe_status check_problem(const moe_problem* p) {
    if (!p) return MOE_ERR_NULL;
    if (p->bits != 4 && p->bits != 8) return MOE_ERR_UNSUPPORTED;
    if (p->group_size != 32 && p->group_size != 64 && p->group_size != 128)
        return MOE_ERR_UNSUPPORTED;
    if (p->flags & ~(MOE_F_FP32_OUT | MOE_F_FP32_INTERMEDIATE | MOE_F_SWIGLU))
        return MOE_ERR_UNSUPPORTED;
    if (p->T < 0 || p->k < 1 || p->E < 1 || p->H < 1 || p->I < 1) return MOE_ERR_SHAPE;
    if (p->E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if (p->k > p->E) return MOE_ERR_SHAPE;
    // The kernels step through K in 64-column halves of 128-column chunks;
    // a group never straddles two of those steps.
    if (p->H % 64 || p->I % 64) return MOE_ERR_SHAPE;
    if (p->H % p->group_size || p->I % p->group_size) return MOE_ERR_SHAPE;
    if (p->H > moe::kMaxDim || p->I > moe::kMaxDim) return MOE_ERR_UNSUPPORTED;
    const int64_t A = static_cast<int64_t>(p->T) * p->k;
    if (A > INT32_MAX / 2) return MOE_ERR_SHAPE;
    // the route's launch (x in pieces of 8 columns) and the wide matmuls'
    const int64_t tiles = moe_max_tiles(A, p->E, big_rows(p)), T = p->T;
    const int64_t route = moe::route_count_wgs(A) + 1 + (T * (p->H / 8) + moe::kRouteThreads - 1) / moe::kRouteThreads;
    if (!fits_launch(route, moe::kRouteThreads) || !fits_launch(tiles * ((p->I + 127) / 128) + 7, moe::kWideThreads) ||
        !fits_launch(tiles * ((p->H + 255) / 256) + 7, moe::kWideThreads))
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

moe_ws_layout make_layout(const moe_problem* p) {
    moe_ws_layout l = {};
    const int64_t A = static_cast<int64_t>(p->T) * p->k;
    l.bm_big = big_rows(p);
    l.bm_small = moe::kBmSmall;
    l.max_tiles = moe_max_tiles(A, p->E, l.bm_big);
    l.max_skinny = moe_max_tiles(A, p->E, l.bm_small);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes);
        return at;
    };
    const size_t hbytes = (p->flags & MOE_F_FP32_INTERMEDIATE) ? 4 : 2;
    const size_t G = p->H / p->group_size;
    l.counts = take(sizeof(int32_t) * p->E);
    l.offsets = take(sizeof(int32_t) * (p->E + 1));
    l.perm = take(sizeof(int32_t) * A);
    l.inv_perm = take(sizeof(int32_t) * A);
    l.tiles = take(sizeof(moe_tile) * l.max_tiles);
    l.tiles_skinny = take(sizeof(moe_tile) * l.max_skinny);
    l.num_tiles = take(sizeof(int32_t) * 8);
    l.x_perm = take(sizeof(uint16_t) * p->T * p->H);
    l.x_sums = take(sizeof(float) * p->T * G);
    l.h = take(hbytes * A * p->I);
    l.h_sums = take(sizeof(float) * A * (p->I / 16));
    l.y = take(sizeof(float) * A * p->H);
    // per-segment key counts, then one order check per segment (pre-sorted entry)
    l.route_hist = take(sizeof(int32_t) * moe::route_count_wgs(A) * (static_cast<size_t>(p->E) + 2));
    // x as e4m3 hi + lo with block scales, for the wide gate|up kernel's fp8 operands
    const bool fp8 = moe::fp8_wide_gateup(p->T, p->group_size, p->bits, p->flags);
    l.x8_hi = take(fp8 ? static_cast<size_t>(p->T) * p->H : 0);
    l.x8_lo = take(fp8 ? static_cast<size_t>(p->T) * p->H : 0);
    l.x8_scales = take(fp8 ? static_cast<size_t>(p->T) * moe::x8_stride(p->H) : 0);
    l.total = off;
    return l;
}

moe_status forward_impl(const moe_problem* p, const void* x, const int32_t* ids,
                        const float* topk_w, const uint32_t* w_gu, const void* s_gu,
                        const void* b_gu, const uint32_t* w_d, const void* s_d,
                        const void* b_d, void* out, void* ws, size_t ws_bytes, void* stream,
                        void* const* events, const int32_t* presorted, bool want_presorted,
                        bool combine = true) {
    const moe_status st = check_problem(p);
    if (st != MOE_OK) return st;
    if (combine && !fits_launch((static_cast<int64_t>(p->T) * (p->H / 4) + moe::kCombineThreads - 1) / moe::kCombineThreads,
                                moe::kCombineThreads))
        return MOE_ERR_SHAPE;
    if (p->T == 0) return MOE_OK;
    if (!x || !ids || !topk_w || !w_gu || !s_gu || !b_gu || !w_d || !s_d || !b_d || (combine && !out))
        return MOE_ERR_NULL;
    if (want_presorted && !presorted) return MOE_ERR_NULL;
    if (presorted && !aligned(presorted, 4)) return MOE_ERR_ALIGN;
    if (!ws) return MOE_ERR_WORKSPACE;
    const moe_ws_layout l = make_layout(p);
    if (ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    const bool f32out = p->flags & MOE_F_FP32_OUT;
    if (!aligned(x, 16) || !aligned(w_gu, 16) || !aligned(w_d, 16) || !aligned(ids, 4) ||
        !aligned(topk_w, 4) || !aligned(s_gu, 16) || !aligned(b_gu, 16) || !aligned(s_d, 16) ||
        !aligned(b_d, 16) || !aligned(out, f32out ? 16 : 8) || !aligned(ws, kAlign))
        return MOE_ERR_ALIGN;

    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    // events[2i], events[2i+1]: start and stop of kernel i
    auto kt = [&](int i) {
        moe::KTiming t;
        if (events != nullptr) {
            t.start = static_cast<hipEvent_t>(events[2 * i]);
            t.stop = static_cast<hipEvent_t>(events[2 * i + 1]);
        }
        return t;
    };

    moe::RouteArgs r;
    r.ids = ids;
    r.A = p->T * p->k;
    r.E = p->E;
    r.bm_big = l.bm_big;
    r.bm_small = l.bm_small;
    r.max_tiles = l.max_tiles;
    r.max_skinny = l.max_skinny;
    // At most bm_small tokens: no expert has more rows unless a token repeats
    // an id, so every expert takes the skinny path (in tiles of bm_small) and
    // the wide launches are left out.
    const bool skinny_only = p->T <= l.bm_small;
    r.skinny_max_rows = skinny_only ? INT32_MAX : l.bm_small;
    r.counts = reinterpret_cast<int32_t*>(base + l.counts);
    r.offsets = reinterpret_cast<int32_t*>(base + l.offsets);
    r.perm = reinterpret_cast<int32_t*>(base + l.perm);
    r.inv_perm = reinterpret_cast<int32_t*>(base + l.inv_perm);
    r.tiles = reinterpret_cast<int32_t*>(base + l.tiles);
    r.tiles_skinny = reinterpret_cast<int32_t*>(base + l.tiles_skinny);
    r.num_tiles = reinterpret_cast<int32_t*>(base + l.num_tiles);
    r.presorted = presorted;
    r.count_wgs = moe::route_count_wgs(r.A);
    r.hist = reinterpret_cast<int32_t*>(base + l.route_hist);
    r.x = static_cast<const uint16_t*>(x);
    r.T = p->T;
    r.H = p->H;
    r.gs = p->group_size;
    r.xp = reinterpret_cast<uint16_t*>(base + l.x_perm);
    r.xs = reinterpret_cast<float*>(base + l.x_sums);
    const bool fp8 = moe::fp8_wide_gateup(p->T, p->group_size, p->bits, p->flags);
    r.x8hi = fp8 ? reinterpret_cast<uint8_t*>(base + l.x8_hi) : nullptr;
    r.x8lo = fp8 ? reinterpret_cast<uint8_t*>(base + l.x8_lo) : nullptr;
    r.x8s = fp8 ? reinterpret_cast<uint8_t*>(base + l.x8_scales) : nullptr;

    moe::FfnArgs f;
    f.T = p->T;
    f.k = p->k;
    f.E = p->E;
    f.H = p->H;
    f.I = p->I;
    f.gs = p->group_size;
    f.bits = p->bits;
    f.max_tiles = l.max_tiles;
    f.max_skinny = l.max_skinny;
    f.skinny_only = skinny_only ? 1 : 0;
    f.flags = p->flags;
    f.zero = 0;
    f.x = static_cast<const uint16_t*>(x);
    f.xp = r.xp;
    f.xs = r.xs;
    f.x8hi = r.x8hi;
    f.x8lo = r.x8lo;
    f.x8s = r.x8s;
    f.hs = reinterpret_cast<float*>(base + l.h_sums);
    f.ids = ids;
    f.topk_w = topk_w;
    f.w_gu = w_gu;
    f.s_gu = static_cast<const uint16_t*>(s_gu);
    f.b_gu = static_cast<const uint16_t*>(b_gu);
    f.w_d = w_d;
    f.s_d = static_cast<const uint16_t*>(s_d);
    f.b_d = static_cast<const uint16_t*>(b_d);
    f.perm = r.perm;
    f.tiles = r.tiles;
    f.tiles_skinny = r.tiles_skinny;
    f.num_tiles = r.num_tiles;
    f.h = base + l.h;
    f.y = reinterpret_cast<float*>(base + l.y);
    f.out = out;

    if (moe::launch_route(r, s, kt(0)) != hipSuccess) return MOE_ERR_HIP;
    if (moe::launch_gateup_skinny(f, s, kt(1)) != hipSuccess) return MOE_ERR_HIP;
    if (moe::launch_gateup_wide(f, s, kt(2)) != hipSuccess) return MOE_ERR_HIP;
    if (moe::launch_down_skinny(f, s, kt(3)) != hipSuccess) return MOE_ERR_HIP;
    if (moe::launch_down_wide(f, s, kt(4)) != hipSuccess) return MOE_ERR_HIP;
    if (combine && moe::launch_combine(f, s, kt(5)) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
}

bool known_type(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_FP32; }
size_t type_size(int32_t t) { return t == MOE_T_FP32 ? 4 : 2; }

// Whether an output lies on an input's address without being its very rows.
bool clashes(const void* out, int32_t type, int64_t stride, const void* in, int32_t in_type, int64_t in_stride, int32_t T) {
    return out && out == in && (type != in_type || (T > 1 && stride != in_stride));
}

// The checks of a block norm of y (nullptr: not an address of the caller's), whose
// pointer itself is left to do.
moe_status check_norm(const moe_norm* n, const void* y) {
    if (!n) return MOE_ERR_NULL;
    if (!known_type(n->y_type) || !known_type(n->stream_type) || !known_type(n->normed_type) ||
        !known_type(n->weight_type) || !known_type(n->gate_type) || (n->flags & ~MOE_N_POST))
        return MOE_ERR_UNSUPPORTED;
    if (n->T < 0 || n->H < 1) return MOE_ERR_SHAPE;
    if (n->H > MOE_NORM_MAX_H) return MOE_ERR_UNSUPPORTED;
    if (!(n->eps >= 0.f)) return MOE_ERR_SHAPE;
    if (n->T == 0) return MOE_OK;
    if (!n->out && !n->normed) return MOE_ERR_NULL;
    if (n->y_stride < 0 || (n->residual && n->residual_stride < 0) || (n->out && n->out_stride < n->H) ||
        (n->normed && n->normed_stride < n->H))
        return MOE_ERR_SHAPE;
    if (n->gate && (n->gate_stride_t < 0 || n->gate_stride_h < 0 || n->gate_stride_h > 1)) return MOE_ERR_SHAPE;
    if ((n->out && n->out == n->normed) ||
        clashes(n->out, n->stream_type, n->out_stride, y, n->y_type, n->y_stride, n->T) ||
        clashes(n->out, n->stream_type, n->out_stride, n->residual, n->stream_type, n->residual_stride, n->T) ||
        clashes(n->normed, n->normed_type, n->normed_stride, y, n->y_type, n->y_stride, n->T) ||
        clashes(n->normed, n->normed_type, n->normed_stride, n->residual, n->stream_type, n->residual_stride, n->T))
        return MOE_ERR_UNSUPPORTED;
    const size_t ws = type_size(n->weight_type), ss = type_size(n->stream_type);
    if (!aligned(n->residual, ss) || !aligned(n->out, ss) || !aligned(n->normed, type_size(n->normed_type)) ||
        !aligned(n->post_weight, ws) || !aligned(n->pre_weight, ws) || !aligned(n->gate, type_size(n->gate_type)))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

moe::NormArgs norm_args(const moe_norm* n, const void* y) {
    moe::NormArgs a = {};
    a.T = n->T;
    a.H = n->H;
    a.post = n->flags & MOE_N_POST;
    a.y_f32 = n->y_type == MOE_T_FP32;
    a.stream_f32 = n->stream_type == MOE_T_FP32;
    a.normed_f32 = n->normed_type == MOE_T_FP32;
    a.weight_f32 = n->weight_type == MOE_T_FP32;
    a.gate_f32 = n->gate_type == MOE_T_FP32;
    a.eps = n->eps;
    a.residual_scale = n->residual_scale;
    a.gate_scale = n->gate_scale;
    a.weight_offset = n->weight_offset;
    a.y = y;
    a.residual = n->residual;
    a.post_weight = a.post ? n->post_weight : nullptr;
    a.gate = n->gate;
    a.pre_weight = n->normed ? n->pre_weight : nullptr;
    a.out = n->out;
    a.normed = n->normed;
    a.y_stride = n->y_stride;
    a.residual_stride = n->residual ? n->residual_stride : 0;
    a.out_stride = n->out ? n->out_stride : 0;
    a.normed_stride = n->normed ? n->normed_stride : 0;
    a.gate_stride_t = n->gate ? n->gate_stride_t : 0;
    a.gate_stride_h = n->gate ? n->gate_stride_h : 0;
    return a;
}

// A router's checks apart from its outputs.
moe_status check_router(const moe_router* r) {
    if (!r) return MOE_ERR_NULL;
    if (!known_type(r->weight_type) || (r->flags & ~MOE_R_NORM)) return MOE_ERR_UNSUPPORTED;
    if (r->T < 0 || r->H < 1 || r->E < 1 || r->k < 1 || r->k > r->E || r->H % 64) return MOE_ERR_SHAPE;
    if (r->E > MOE_MAX_EXPERTS || r->k > moe::kRouterMaxK || r->H > MOE_NORM_MAX_H) return MOE_ERR_UNSUPPORTED;
    if (!(r->eps >= 0.f)) return MOE_ERR_SHAPE;
    if (r->x_stride < r->H || r->x_stride > MOE_ROUTER_MAX_STRIDE) return MOE_ERR_SHAPE;
    if (static_cast<int64_t>(r->T) * r->E > INT32_MAX || r->T > MOE_ROUTER_MAX_TOKENS) return MOE_ERR_SHAPE;
    if (r->T == 0) return MOE_OK;
    if (!r->weight) return MOE_ERR_NULL;
    if (r->x_stride % 8 || !aligned(r->weight, 16) || !aligned(r->expert_scale, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

moe::RouterArgs router_args(const moe_router* r, const void* x, float* logits) {
    moe::RouterArgs a;
    a.T = r->T;
    a.H = r->H;
    a.E = r->E;
    a.weight_f32 = r->weight_type == MOE_T_FP32;
    a.norm = r->flags & MOE_R_NORM;
    a.eps = r->eps;
    a.x_stride = r->x_stride;
    a.x = static_cast<const uint16_t*>(x);
    a.weight = r->weight;
    a.logits = logits;
    return a;
}

hipError_t enqueue_router(const moe_router* r, const void* x, float* logits, int32_t* ids, float* weights,
                          hipStream_t s) {
    const hipError_t e = moe::launch_router_product(router_args(r, x, logits), s);
    if (e != hipSuccess) return e;
    return moe::launch_router_topk(logits, r->T, r->E, r->k, r->expert_scale, ids, weights, s);
}

static_assert(moe::kLayerFewTokens == MOE_LAYER_FEW_TOKENS, "few-token limit");

// Byte offsets in the layer's workspace.
struct LayerLayout {
    size_t counters, logits, ids, weights, n, nsum, h, hsum, y, ffn, total;
    int32_t num_counters;
    bool few;
};
LayerLayout layer_layout(const moe_problem* p) {
    LayerLayout l = {};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes);
        return at;
    };
    const size_t T = p->T, A = T * p->k, H = p->H, I = p->I;
    l.few = p->T <= MOE_LAYER_FEW_TOKENS;
    l.logits = take(4 * T * p->E);
    if (l.few) {
        l.num_counters = static_cast<int32_t>(2 * moe::kLayerRanges + 2 * moe::kLayerCounterStride * A + 1);
        l.counters = take(4 * static_cast<size_t>(l.num_counters));
        l.n = take(4 * T * H);
        l.nsum = take(8 * T * (H / 32));
        l.h = take(4 * A * I);
        l.hsum = take(8 * A * (I / 16));
        l.y = take(4 * A * H);
    } else {
        l.ids = take(4 * A);
        l.weights = take(4 * A);
        l.n = take(2 * T * H);
        l.ffn = take(make_layout(p).total);
    }
    l.total = off;
    if (!l.few) {
        // never less than a smaller batch takes: the few-token form keeps n and h wider
        moe_problem most = *p;
        most.T = MOE_LAYER_FEW_TOKENS;
        const size_t few = layer_layout(&most).total;
        if (l.total < few) l.total = few;
    }
    return l;
}

moe_status check_layer_problem(const moe_problem* p) {
    const moe_status st = check_problem(p);
    if (st != MOE_OK) return st;
    if ((p->flags & MOE_F_FP32_OUT) || p->k > moe::kRouterMaxK) return MOE_ERR_UNSUPPORTED;
    return static_cast<int64_t>(p->T) * p->E > INT32_MAX ? MOE_ERR_SHAPE : MOE_OK;
}

bool rows16(const void* q, int64_t stride, int32_t type) {
    return !q || (aligned(q, 16) && stride * static_cast<int64_t>(type_size(type)) % 16 == 0);
}

}  // namespace

extern "C" {

size_t moe_layer_workspace_bytes(const moe_problem* p) {
    return check_layer_problem(p) == MOE_OK ? layer_layout(p).total : 0;
}

moe_status moe_layer_forward(const moe_problem* p, const moe_layer* l, const void* x, const moe_norm* tail, void* ws,
                             size_t ws_bytes, void* stream) {
    moe_status st = check_layer_problem(p);
    if (st != MOE_OK) return st;
    if (!l || !tail) return MOE_ERR_NULL;
    if (!known_type(l->norm_type) || (l->flags & ~MOE_L_NORM)) return MOE_ERR_UNSUPPORTED;
    moe_router r;
    r.T = p->T;
    r.H = p->H;
    r.E = p->E;
    r.k = p->k;
    r.weight_type = l->router_type;
    r.flags = l->router_flags;
    r.eps = l->eps;
    r.x_stride = p->H;
    r.weight = l->router_weight;
    r.expert_scale = l->expert_scale;
    if ((st = check_router(&r)) != MOE_OK) return st;
    moe_norm t = *tail;
    t.y_type = MOE_T_FP32;
    t.y_stride = p->H;
    if (t.T != p->T || t.H != p->H) return MOE_ERR_SHAPE;
    if ((st = check_norm(&t, nullptr)) != MOE_OK) return st;
    if (p->T == 0) return MOE_OK;
    if (!x || !l->w_gateup || !l->s_gateup || !l->b_gateup || !l->w_down || !l->s_down || !l->b_down) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(l->norm_weight, 16) || !aligned(l->w_gateup, 16) || !aligned(l->s_gateup, 16) ||
        !aligned(l->b_gateup, 16) || !aligned(l->w_down, 16) || !aligned(l->s_down, 16) || !aligned(l->b_down, 16) ||
        !aligned(l->topk_ids, 4) || !aligned(l->topk_weights, 4) || !aligned(ws, kAlign) ||
        !rows16(t.residual, t.residual_stride, t.stream_type) || !rows16(t.out, t.out_stride, t.stream_type) ||
        !rows16(t.normed, t.normed_stride, t.normed_type) || !rows16(t.post_weight, 0, 0) ||
        !rows16(t.pre_weight, 0, 0) || (t.gate && t.gate_stride_h && !rows16(t.gate, t.gate_stride_t, t.gate_type)))
        return MOE_ERR_ALIGN;
    const LayerLayout y = layer_layout(p);
    if (!ws || ws_bytes < y.total) return MOE_ERR_WORKSPACE;

    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    float* const logits = reinterpret_cast<float*>(base + y.logits);
    if (y.few) {
        moe::LayerArgs a = {};
        a.T = p->T;
        a.k = p->k;
        a.E = p->E;
        a.H = p->H;
        a.I = p->I;
        a.gs = p->group_size;
        a.bits = p->bits;
        a.swiglu = p->flags & MOE_F_SWIGLU;
        a.norm = l->flags & MOE_L_NORM;
        a.norm_f32 = l->norm_type == MOE_T_FP32;
        a.eps = l->eps;
        a.weight_offset = l->weight_offset;
        a.magic_gateup = moe::cut::unit_magic(moe::cut::units_of_tile(false, p->H, p->I));
        a.magic_down = moe::cut::unit_magic(moe::cut::units_of_tile(true, p->H, p->I));
        a.router = router_args(&r, x, logits);
        a.expert_scale = l->expert_scale;
        a.x = static_cast<const uint16_t*>(x);
        a.norm_weight = a.norm ? l->norm_weight : nullptr;
        a.w_gu = l->w_gateup;
        a.w_d = l->w_down;
        a.s_gu = static_cast<const uint16_t*>(l->s_gateup);
        a.b_gu = static_cast<const uint16_t*>(l->b_gateup);
        a.s_d = static_cast<const uint16_t*>(l->s_down);
        a.b_d = static_cast<const uint16_t*>(l->b_down);
        a.out_ids = l->topk_ids;
        a.out_weights = l->topk_weights;
        a.tail = norm_args(&t, nullptr);
        const int A = p->T * p->k;
        a.counters = reinterpret_cast<int32_t*>(base + y.counters);
        a.num_counters = y.num_counters;
        a.claim_gateup = a.counters;
        a.claim_down = a.claim_gateup + moe::kLayerRanges;
        a.done_gateup = a.claim_down + moe::kLayerRanges;
        a.done_down = a.done_gateup + moe::kLayerCounterStride * A;
        a.failed = a.done_down + moe::kLayerCounterStride * A;
        a.logits = logits;
        a.n = reinterpret_cast<uint16_t*>(base + y.n);
        a.nsum = reinterpret_cast<float*>(base + y.nsum);
        a.h = reinterpret_cast<uint16_t*>(base + y.h);
        a.hsum = reinterpret_cast<float*>(base + y.hsum);
        a.y = reinterpret_cast<float*>(base + y.y);
        return moe::launch_layer_few(a, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
    }

    const void* n = x;
    if (l->flags & MOE_L_NORM) {
        moe::NormArgs a = {};
        a.T = p->T;
        a.H = p->H;
        a.weight_f32 = l->norm_type == MOE_T_FP32;
        a.eps = l->eps;
        a.gate_scale = 1.f;
        a.weight_offset = l->weight_offset;
        a.y = x;
        a.y_stride = p->H;
        a.pre_weight = l->norm_weight;
        a.normed = base + y.n;
        a.normed_stride = p->H;
        if (moe::launch_block_norm(a, s) != hipSuccess) return MOE_ERR_HIP;
        n = base + y.n;
    }
    int32_t* const ids = l->topk_ids ? l->topk_ids : reinterpret_cast<int32_t*>(base + y.ids);
    float* const weights = l->topk_weights ? l->topk_weights : reinterpret_cast<float*>(base + y.weights);
    if (enqueue_router(&r, x, logits, ids, weights, s) != hipSuccess) return MOE_ERR_HIP;
    const moe_ws_layout f = make_layout(p);
    st = forward_impl(p, n, ids, weights, l->w_gateup, l->s_gateup, l->b_gateup, l->w_down, l->s_down, l->b_down, nullptr,
                      base + y.ffn, f.total, stream, nullptr, nullptr, false, false);
    if (st != MOE_OK) return st;
    moe::NormArgs a = norm_args(&t, base + y.ffn + f.y);
    a.ids = ids;
    a.k = p->k;
    a.E = p->E;
    return moe::launch_block_norm(a, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_router_forward(const moe_router* r, const void* x, float* logits, int32_t* topk_ids,
                              float* topk_weights, void* stream) {
    const moe_status st = check_router(r);
    if (st != MOE_OK) return st;
    if (r->T == 0) return MOE_OK;
    if (!x || !logits || !topk_ids || !topk_weights) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return MOE_ERR_ALIGN;
    const hipError_t e =
        enqueue_router(r, x, logits, topk_ids, topk_weights, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_block_norm(const moe_norm* n, const void* y, void* stream) {
    const moe_status st = check_norm(n, y);
    if (st != MOE_OK) return st;
    if (n->T == 0) return MOE_OK;
    if (!y) return MOE_ERR_NULL;
    if (!aligned(y, type_size(n->y_type))) return MOE_ERR_ALIGN;
    const hipError_t e = moe::launch_block_norm(norm_args(n, y), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int32_t moe_max_tiles(int64_t A, int32_t E, int32_t bm_big) {
    if (A < 0 || E < 1 || bm_big < 1) return -1;
    const int64_t v = A / bm_big + (A < E ? A : E);
    return v > INT32_MAX ? -1 : static_cast<int32_t>(v);
}

moe_status moe_sort_build_tiles(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E,
                                int32_t bm_big, int32_t bm_small, int32_t* counts,
                                int32_t* offsets, int32_t* perm, int32_t* inv_perm,
                                moe_tile* tiles, int32_t max_tiles, int32_t* num_tiles,
                                void* stream) {
    if (T < 0 || k < 1 || E < 1) return MOE_ERR_SHAPE;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if (bm_small < 1 || bm_big < bm_small) return MOE_ERR_SHAPE;
    const int64_t A = static_cast<int64_t>(T) * k;
    if (A > INT32_MAX / 2) return MOE_ERR_SHAPE;
    if (!counts || !offsets || !num_tiles || !tiles) return MOE_ERR_NULL;
    if (A > 0 && (!topk_ids || !perm || !inv_perm)) return MOE_ERR_NULL;
    const int32_t need = moe_max_tiles(A, E, bm_big);
    if (need < 0 || max_tiles < need) return MOE_ERR_WORKSPACE;
    if (!aligned(tiles, 16) || !aligned(counts, 4) || !aligned(offsets, 4) ||
        !aligned(num_tiles, 4) || (A > 0 && (!aligned(topk_ids, 4) || !aligned(perm, 4) ||
                                             !aligned(inv_perm, 4))))
        return MOE_ERR_ALIGN;
    moe::RouteArgs r;
    r.ids = topk_ids;
    r.A = static_cast<int32_t>(A);
    r.E = E;
    r.bm_big = bm_big;
    r.bm_small = bm_small;
    r.max_tiles = max_tiles;
    r.counts = counts;
    r.offsets = offsets;
    r.perm = perm;
    r.inv_perm = inv_perm;
    r.tiles = reinterpret_cast<int32_t*>(tiles);
    r.tiles_skinny = nullptr;
    r.max_skinny = 0;
    r.skinny_max_rows = bm_small;
    r.presorted = nullptr;
    r.count_wgs = 0;
    r.hist = nullptr;
    r.num_tiles = num_tiles;
    r.x = nullptr;
    r.gs = 0;
    r.T = T;
    r.H = 0;
    r.xp = nullptr;
    r.xs = nullptr;
    r.x8hi = nullptr;
    r.x8lo = nullptr;
    r.x8s = nullptr;
    return moe::launch_route(r, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK
                                                                               : MOE_ERR_HIP;
}

size_t moe_ffn_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK) return 0;
    return make_layout(p).total;
}

moe_status moe_ffn_workspace_layout(const moe_problem* p, moe_ws_layout* layout) {
    if (!layout) return MOE_ERR_NULL;
    const moe_status st = check_problem(p);
    if (st != MOE_OK) return st;
    *layout = make_layout(p);
    return MOE_OK;
}

moe_status moe_expert_ffn_forward(const moe_problem* p, const void* x, const int32_t* topk_ids,
                                  const float* topk_weights, const uint32_t* w_gateup,
                                  const void* s_gateup, const void* b_gateup,
                                  const uint32_t* w_down, const void* s_down, const void* b_down,
                                  void* out, void* ws, size_t ws_bytes, void* stream) {
    return forward_impl(p, x, topk_ids, topk_weights, w_gateup, s_gateup, b_gateup, w_down,
                        s_down, b_down, out, ws, ws_bytes, stream, nullptr, nullptr, false);
}

moe_status moe_expert_ffn_forward_noalloc(const moe_problem* p, const void* x,
                                          const int32_t* topk_ids, const float* topk_weights,
                                          const uint32_t* w_gateup, const void* s_gateup,
                                          const void* b_gateup, const uint32_t* w_down,
                                          const void* s_down, const void* b_down, void* out,
                                          void* stream) {
    const moe_status st = check_problem(p);
    if (st != MOE_OK) return st;
    if (p->T == 0) return MOE_OK;
    if (make_layout(p).total > MOE_NOALLOC_SCRATCH_BYTES) return MOE_ERR_SCRATCH;
    hipError_t err = hipSuccess;
    void* ws = scratch_for_current_device(&err);
    if (ws == nullptr) return MOE_ERR_HIP;
    return forward_impl(p, x, topk_ids, topk_weights, w_gateup, s_gateup, b_gateup, w_down, s_down,
                        b_down, out, ws, MOE_NOALLOC_SCRATCH_BYTES, stream, nullptr, nullptr, false);
}

moe_status moe_expert_ffn_forward_presorted(const moe_problem* p, const void* x,
                                            const int32_t* topk_ids, const float* topk_weights,
                                            const int32_t* sorted_order,
                                            const uint32_t* w_gateup, const void* s_gateup,
                                            const void* b_gateup, const uint32_t* w_down,
                                            const void* s_down, const void* b_down, void* out,
                                            void* ws, size_t ws_bytes, void* stream) {
    return forward_impl(p, x, topk_ids, topk_weights, w_gateup, s_gateup, b_gateup, w_down,
                        s_down, b_down, out, ws, ws_bytes, stream, nullptr, sorted_order, true);
}

moe_status moe_expert_ffn_forward_timed(const moe_problem* p, const void* x,
                                        const int32_t* topk_ids, const float* topk_weights,
                                        const uint32_t* w_gateup, const void* s_gateup,
                                        const void* b_gateup, const uint32_t* w_down,
                                        const void* s_down, const void* b_down, void* out,
                                        void* ws, size_t ws_bytes, void* stream,
                                        void* const* events) {
    return forward_impl(p, x, topk_ids, topk_weights, w_gateup, s_gateup, b_gateup, w_down,
                        s_down, b_down, out, ws, ws_bytes, stream, events, nullptr, false);
}

moe_status moe_router_topk(const float* logits, int32_t T, int32_t E, int32_t k,
                           int32_t* topk_ids, float* topk_weights, void* stream) {
    if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_SHAPE;
    if (E > MOE_MAX_EXPERTS || k > moe::kRouterMaxK) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_weights) return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return MOE_ERR_ALIGN;
    if (static_cast<int64_t>(T) * E > INT32_MAX) return MOE_ERR_SHAPE;
    const hipError_t e = moe::launch_router_topk(logits, T, E, k, nullptr, topk_ids, topk_weights,
                                                  static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

const char* moe_status_string(moe_status s) {
    switch (s) {
        case MOE_OK: return "ok";
        case MOE_ERR_NULL: return "a required pointer is NULL";
        case MOE_ERR_SHAPE: return "invalid or inconsistent sizes";
        case MOE_ERR_UNSUPPORTED: return "unsupported configuration (bits, group size, flags or expert count)";
        case MOE_ERR_ALIGN: return "a pointer is misaligned";
        case MOE_ERR_WORKSPACE: return "workspace or tile buffer missing or too small";
        case MOE_ERR_HIP: return "HIP runtime error while enqueueing work";
        case MOE_ERR_SCRATCH:
            return "problem needs more workspace than the built-in scratch buffer of the allocation-free entry point holds";
        default: return "unknown status";
    }
}

}  // extern "C"
