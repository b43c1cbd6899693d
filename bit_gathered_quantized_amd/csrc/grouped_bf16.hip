// Grouped products of bf16 rows and bf16 weights.
#include "grouped_product.h"

namespace moe {

hipError_t launch_grouped_bf16(const GroupedArgs& a, hipStream_t s) {
    const bool once = read_once(a, 2 * static_cast<int64_t>(a.N) * a.K), low = low_strips(a);
    if (big_tiles(a))
        a.w_kn ? launch_product<Form::kCols, 256, false>(a, s) : launch_product<Form::kRows, 256, false>(a, s);
    else if (a.w_kn)
        low ? launch_product<Form::kCols, 32>(a, once, s) : launch_product<Form::kCols, 128>(a, once, s);
    else
        low ? launch_product<Form::kRows, 32>(a, once, s) : launch_product<Form::kRows, 128>(a, once, s);
    return hipGetLastError();
}

}  // namespace moe
