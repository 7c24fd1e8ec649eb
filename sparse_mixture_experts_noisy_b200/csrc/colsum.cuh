// Column sums of a pass whose blocks left partial rows: gamma's and beta's
// gradients of the layer norm, the bias's of the dense layer.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

// out0[c] = sum over g of part[g][0][c], out1[c] of part[g][1][c], for one or two
// arrays a row: 32 columns per block, each of 32 warps every 32nd partial row, then
// a tree over the warps.  An out that is null is skipped.
__global__ void __launch_bounds__(1024)
col_reduce_kernel(const float *part, int64_t groups, int n, float *out0, float *out1) {
    __shared__ float red[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float *out = blockIdx.y == 0 ? out0 : out1;
    if (out == nullptr) return;
    float a = 0.0f;
    if (col < n) {
#pragma unroll 4
        for (int64_t g = warp; g < groups; g += 32) a += part[(gridDim.y * g + blockIdx.y) * n + col];
    }
    red[warp][lane] = a;
    __syncthreads();
    a = red[lane][warp];  // warp w now sums column w
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0 && blockIdx.x * 32 + warp < n) out[blockIdx.x * 32 + warp] = a;
}

cudaError_t launch_col_reduce(const float *part, int64_t groups, int n, int arrays, float *out0, float *out1,
                              cudaStream_t s) {
    return launch_pdl(col_reduce_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(n) + 31) / 32), arrays),
                      dim3(1024), 0, s, part, groups, n, out0, out1);
}

}  // namespace

}  // namespace moe
