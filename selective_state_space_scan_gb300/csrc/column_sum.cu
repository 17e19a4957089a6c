// Second pass of the gradients of weights: every CTA of the first has left a row of sums.  A warp takes every
// 32nd row of 32 columns, so that a read is 128 bytes wide and several are in flight; the warps' sums meet in
// shared memory.
#include "column_sum.h"

#include "chained.cuh"

namespace selscan {
namespace {

// (part is not restrict: the kernel before still writes it when this one comes up)
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int n, int64_t ld, int cols, int split,
                                                          float* out0, float* out1) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = blockIdx.x * 32 + lane;
    float v = 0.f;
    wait_for_earlier();
    if (j < cols) {
#pragma unroll 4
        for (int i = warp; i < n; i += 32) v += part[i * ld + j];
    }
    s[warp][lane] = v;
    __syncthreads();
    v = s[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int c = blockIdx.x * 32 + warp;
    if (lane == 0 && c < cols) {
        if (c < split) out0[c] = v;
        else if (out1) out1[c - split] = v;
    }
}

}  // namespace

cudaError_t launch_column_sum(const float* part, int n, int64_t ld, int cols, int split, float* out0, float* out1, cudaStream_t stream) {
    return launch_chained(column_sum_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(1024), 0, stream, part, n, ld, cols, split, out0, out1);
}

}  // namespace selscan
