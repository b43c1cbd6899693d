// Grouped products of bf16 rows and bf16 weights.
#include "grouped_product.h"

namespace moe {

hipError_t launch_grouped_bf16(const GroupedArgs& a, hipStream_t s) {
    const bool once = read_once(a, 2 * static_cast<int64_t>(a.N) * a.K);
    if (a.w_kn)
        once ? launch_product<Form::kCols, true>(a, s) : launch_product<Form::kCols, false>(a, s);
    else
        once ? launch_product<Form::kRows, true>(a, s) : launch_product<Form::kRows, false>(a, s);
    return hipGetLastError();
}

}  // namespace moe
