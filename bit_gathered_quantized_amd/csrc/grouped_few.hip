// Grouped products for few rows: the rule and the launches.
#include "grouped_few.h"

namespace moe {

// Few rows an expert and not many weights: then a call is bound by latency, and streams
// of its own for every 16 columns and eighth of K are faster than tiles that step through K.
// Few | tiles: 1 row of 4096 x 4096 in bf16 9.4 | 29 us, 8 rows of 8 of 128 experts by 1408 x
// 2816 15 | 22 us (codes, bf16 rows 9.8 | 15 us); where reading the weights takes long the
// tiles read them faster (64 rows of 51 of these experts, 405 MB, 95 | 79 us), and for a short
// K they have few steps (8 rows, K 704, N 2816, 12 | 11 us).
bool grouped_few_rows(const GroupedArgs& a) {
    const int64_t row = a.ws ? a.K / 2 : 2 * static_cast<int64_t>(a.K), touched = (a.A < a.E ? a.A : a.E) * a.N * row;
    return !a.w_kn && a.K >= 1024 && (a.A <= 64 || a.A <= 4 * static_cast<int64_t>(a.E)) && touched <= 80 << 20;
}

hipError_t launch_grouped_few(const GroupedArgs& a, hipStream_t s) {
    if (!a.ws)
        launch_few<Form::kRows>(a, s);
    else if (a.xs)
        launch_few<Form::kMx>(a, s);
    else
        launch_few<Form::kBf16Mx>(a, s);
    return hipGetLastError();
}

}  // namespace moe
