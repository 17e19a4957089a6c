// Sums over the rows that the CTAs of a kernel have left in a workspace (the gradients of weights).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace selscan {

// out[j] = Σ_{i<n} part[i·ld + j] for j < cols: the first `split` columns to out0, the others to out1.  The
// order of the additions is the same in every call.
// Follows the kernel that leaves the rows on the same stream (chained.cuh).
cudaError_t launch_column_sum(const float* part, int n, int64_t ld, int cols, int split, float* out0, float* out1,
                              cudaStream_t stream);

}  // namespace selscan
