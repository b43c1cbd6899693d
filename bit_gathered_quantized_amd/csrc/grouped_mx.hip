// Grouped products on microscaled weights, with microscaled or bf16 rows.
#include "grouped_product.h"

namespace moe {

hipError_t launch_grouped_mx(const GroupedArgs& a, hipStream_t s) {
    const bool once = read_once(a, static_cast<int64_t>(a.N) * a.K / 2);
    if (big_tiles(a))
        launch_product<Form::kMx, 256, false>(a, s);
    else
        low_strips(a) ? launch_product<Form::kMx, 32>(a, once, s) : launch_product<Form::kMx, 128>(a, once, s);
    return hipGetLastError();
}

hipError_t launch_grouped_bf16_mx(const GroupedArgs& a, hipStream_t s) {
    // Strips of 32 rows up to kGroupedLowRows rows an expert: whole lines of w at a time (with 128 rows there is
    // room for half lines).  32 | 128 rows, 128 experts by 1408 x 2816: 64 rows 25 | 35 us, 4096 rows
    // 78 | 85 us, 16384 rows 193 | 198 us; 16384 rows of 32 experts by 2816 x 2816 299 | 253 us.
    if (a.A <= kGroupedLowRows * static_cast<int64_t>(a.E))
        launch_product<Form::kBf16Mx, 32>(a, read_once(a, static_cast<int64_t>(a.N) * a.K / 2), s);
    else
        launch_product<Form::kBf16Mx, 128, false>(a, s);  // half lines of w: not non-temporal
    return hipGetLastError();
}

}  // namespace moe
