// Launchers of the few-row kernels (few_rows.h, few_int4.h), one translation unit per kind of
// weights, type of x and number of matrices (-DFG_ROWS_INT4, -DFG_ROWS_BF16,
// -DFG_ROWS_MATRICES), so that they compile side by side.
#include "few_int4.h"

namespace fg {

#define FG_ROWS_NAME_(i, b, m) launch_rows_##i##b##m
#define FG_ROWS_NAME(i, b, m) FG_ROWS_NAME_(i, b, m)

hipError_t FG_ROWS_NAME(FG_ROWS_INT4, FG_ROWS_BF16, FG_ROWS_MATRICES)(const RowsParams& p,
                                                                      hipStream_t stream) {
#if FG_ROWS_INT4
    return launch_int4<FG_ROWS_BF16 != 0, FG_ROWS_MATRICES>(p, stream);
#else
    return launch<FG_ROWS_BF16 != 0>(p, stream);
#endif
}

}  // namespace fg
