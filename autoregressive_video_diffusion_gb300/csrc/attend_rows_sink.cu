// The attention of few rows and of fp32 caches under a window whose first positions stay visible.
#include "attend_rows.cuh"

namespace dcp {

cudaError_t launch_rows_sink(const RowParams& p, int rows, cudaStream_t s) { return launch_form<kSink>(p, rows, s); }

}  // namespace dcp
