// Products of the dense layer, used by linear.cu: on the tensor cores
// (linear_tc.cu) and, for a few tokens, on CUDA cores (linear_skinny.cu).
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

// One product, or two that share a launch where they run on the same kernel.  A
// product whose out is null is not computed, but counts in the choice of the
// other's K split.
// full: bias, activation, residual and z of the epilogue; else out alone.
cudaError_t launch_tc_products(const TcProduct *t, int count, bool fp32, bool full, uint64_t timeout_ns, int num_sms,
                               cudaStream_t s);

// For a few tokens; rows dense, of any width.  dz: dZ in the storage type.
constexpr int kSkinnyRows = 16;   // dx at most; forward: a block's
constexpr int kSkinnyDwRows = 4;  // dW at most
template <typename T>
cudaError_t launch_skinny_fwd(const T *x, const T *W, int64_t M, int K, int Nn, const LinearEpi &epi, cudaStream_t s);
template <typename T>
cudaError_t launch_skinny_dx(const T *dz, const T *W, int64_t M, int Ni, int No, T *dx, cudaStream_t s);
template <typename T>
cudaError_t launch_skinny_dw(const T *dz, const T *x, int64_t M, int Ni, int No, T *dW, cudaStream_t s);

}  // namespace moe
