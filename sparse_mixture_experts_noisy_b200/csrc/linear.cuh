// Epilogue and activation arithmetic shared by the dense layer's kernels.
#pragma once

#include "common.cuh"

namespace moe {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2 };

// Phi(z) of the standard normal, and e = exp(-z^2 / 2), from one exponential:
// 1 - erf(x) = (a1 t + ... + a5 t^5) exp(-x^2) with t = 1 / (1 + 0.3275911 x),
// x = |z| / sqrt(2) >= 0 (Abramowitz and Stegun, 7.1.26; error of erf below
// 1.5e-7, about that of fp32's 1 + erf).  Over [-13, 13] GELU is off by 4.1e-7 at
// most and its derivative by 2.5e-7; z / 2 (1 + erf) in fp32 by 4.7e-7.  The experts
// call erff, so a shared expert's GELU differs from theirs by such amounts.
// GELU passes are bound by its arithmetic: db alone at 32768 x 1408 bf16 takes 55 us
// (113 with erff and expf; its two arrays' bytes take 28), and 59 with the write of
// dZ (42).
//
// The reciprocal and the exponential are the hardware's approximations (about
// 2^-23 and 2^-22 relative); their arguments lie in [1, inf) and (-inf, 0], where
// flushing denormals changes nothing.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = fabsf(z) * 0.70710678118654752440f;
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3275911f, x, 1.0f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * x * -1.4426950408889634f));  // exp(-x^2)
    // half the polynomial's coefficients: Phi(-|z|) = erfc(x) / 2
    float p = fmaf(0.5307027145f, t, -0.7265760135f);
    p = fmaf(p, t, 0.7107068705f);
    p = fmaf(p, t, -0.142248368f);
    p = fmaf(p, t, 0.127414796f);
    const float tail = p * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

// ReLU keeps a NaN (v < 0 is false for it).
__device__ __forceinline__ float act_value(float v, int act) {
    if (act == kActGelu) {
        float e;
        return __fmul_rn(v, normal_cdf(v, e));  // by itself: the same bits with and without a residual or z
    }
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;
    return v;
}

// dy act'(z): ReLU'(z) = [z > 0] (a masked dy does not reach the result, even
// an infinite one), GELU'(z) = Phi(z) + z phi(z).  The product is rounded by
// itself, so that db's sums have the same bits whether or not dZ is stored.
__device__ __forceinline__ float act_backward(float dy, float z, int act) {
    if (act == kActGelu) {
        float e;
        const float c = normal_cdf(z, e);
        return __fmul_rn(dy, fmaf(z * 0.39894228040143267794f, e, c));
    }
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
