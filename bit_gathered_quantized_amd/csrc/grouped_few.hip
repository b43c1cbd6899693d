// Grouped products for few rows: the rule and the launches.
#include "grouped_few.h"

namespace moe {

// Few rows an expert, and workgroups of 64 columns for about one round: then a call is bound by
// latency, and streams of its own for every 16 columns and eighth of K are faster than tiles that
// step through K.  Few | tiles, us: 1 row of 4096 x 4096 in bf16 9.2 | 29; 8 rows of 8 experts by 1408 x
// 2816 (176 workgroups) 15 | 22, codes with bf16 rows 9.8 | 13.6, both as codes 8.9 | 11.0; 12 such
// experts (264) 15 | 22; 64 rows of 1 expert by 4096 x 4096 (320) 22 | 30.  More workgroups: 8
// experts by 4096 x 2816 (512) 37 | 34, codes of 4096 x 4096 with bf16 rows 23 | 17; 64 rows by 8192
// x 4096 (640) 41 | 31; 64 experts by 1408 x 2816 (1408) 90 | 70.  For a shorter K the tiles have few
// steps (8 rows, K 704, N 2816, 12 | 11).
bool grouped_few_rows(const GroupedArgs& a) {
    return !a.w_kn && a.K >= 1024 && (a.A <= 64 || a.A <= 4 * static_cast<int64_t>(a.E)) && most_strips(a, 16) * ((a.N + 63) / 64) <= 320;
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
