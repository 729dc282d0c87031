// The attention of few rows and of fp32 caches of sequences behind a shared prefix.
#include "attend_rows.cuh"

namespace dcp {

cudaError_t launch_rows_rest(const RowParams& p, int rows, cudaStream_t s) { return launch_form<kRest>(p, rows, s); }

}  // namespace dcp
