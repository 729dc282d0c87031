// The attention of few rows and of fp32 caches of all sequences of a group over the prefix they share.
#include "attend_rows.cuh"

namespace dcp {

cudaError_t launch_rows_prefix(const RowParams& p, int rows, cudaStream_t s) { return launch_form<kPrefix>(p, rows, s); }

}  // namespace dcp
