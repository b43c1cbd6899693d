// Grouped products on microscaled weights, with microscaled or bf16 rows.
#include "grouped_product.h"

namespace moe {

hipError_t launch_grouped_mx(const GroupedArgs& a, hipStream_t s) {
    if (read_once(a, static_cast<int64_t>(a.N) * a.K / 2))
        launch_product<Form::kMx, true>(a, s);
    else
        launch_product<Form::kMx, false>(a, s);
    return hipGetLastError();
}

hipError_t launch_grouped_bf16_mx(const GroupedArgs& a, hipStream_t s) {
    // Strips of 64 rows up to 24 rows an expert: whole lines of w at a time.  Low | not, 128 experts
    // by 1408 x 2816: 64 rows 36 | 39 us, 2048 rows 68 | 76 us, 4096 rows 99 | 83 us.
    if (a.A <= 24 * static_cast<int64_t>(a.E))
        launch_product<Form::kBf16MxLow, false>(a, s);
    else
        launch_product<Form::kBf16Mx, false>(a, s);
    return hipGetLastError();
}

}  // namespace moe
