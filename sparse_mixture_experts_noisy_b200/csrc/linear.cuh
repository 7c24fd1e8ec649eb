// Epilogue and activation arithmetic shared by the dense layer's kernels.
#pragma once

#include "common.cuh"

namespace moe {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2 };

// ReLU keeps a NaN (v < 0 is false for it).
__device__ __forceinline__ float act_value(float v, int act) {
    if (act == kActGelu) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752440f));
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;
    return v;
}

// dy act'(z): ReLU'(z) = [z > 0] (a masked dy does not reach the result, even
// an infinite one), GELU'(z) = Phi(z) + z phi(z).  The product is rounded by
// itself, so that db's sums have the same bits whether or not dZ is stored.
__device__ __forceinline__ float act_backward(float dy, float z, int act) {
    if (act == kActGelu)
        return __fmul_rn(dy, fmaf(z * 0.39894228040143267794f, expf(-0.5f * z * z),
                                  0.5f * (1.0f + erff(z * 0.70710678118654752440f))));
    if (act == kActRelu) return z > 0.0f ? dy : 0.0f;
    return dy;
}

// What happens to one accumulated value on its way out.  All nullable but out.
struct LinearEpi {
    const float *bias;
    int act;
    const void *residual;
    void *out;
    void *z_out;
};

template <typename T>
__device__ __forceinline__ void linear_store(const LinearEpi &e, int64_t i, int64_t j, int64_t ld, float v) {
    const int64_t at = i * ld + j;
    if (e.bias != nullptr) v += e.bias[j];
    if (e.z_out != nullptr) static_cast<T *>(e.z_out)[at] = from_f32<T>(v);
    v = act_value(v, e.act);
    if (e.residual != nullptr) v += to_f32<T>(static_cast<const T *>(e.residual)[at]);
    static_cast<T *>(e.out)[at] = from_f32<T>(v);
}

}  // namespace moe
