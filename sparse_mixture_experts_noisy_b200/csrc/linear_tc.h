// Tensor-core products of the dense layer (linear_tc.cu), used by linear.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "linear.cuh"

namespace moe {

// D[m][n] = sum_k Q(m, k) P(n, k), D row-major [M][Nn].  P: [Nn][K] or, p_mn,
// [K][Nn]; Q: [M][K] or, q_mn, [K][M]; bf16, rows padded with zeros to a multiple
// of 8 elements.  For fp32 products both are three planes of that shape, one
// behind the other: the values' bf16 parts.
struct TcProduct {
    const void *P, *Q;
    int64_t M;
    int Nn, K;
    bool p_mn, q_mn;
    LinearEpi epi;
};

// One product, or two that share a launch where both have tiles enough.
// full: bias, activation, residual and z of the epilogue; else out alone.
cudaError_t launch_tc_products(const TcProduct *t, int count, bool fp32, bool full, uint64_t timeout_ns, int num_sms,
                               cudaStream_t s);

}  // namespace moe
