// Layer norm in front of the layer ("nanoMoEの深層解剖" slide 4: each block is
// attention + normalization, then the MoE layer + normalization), with the
// residual add folded in, and its backward pass.
//
//   h = round(x + r)            (h = x without a residual; stored, rounded to the storage type)
//   mu = sum h / d,  var = sum (h - mu)^2 / d,  rstd = 1 / sqrt(var + eps)
//   y = (h - mu) rstd gamma + beta
// and, with xh = (h - mu) rstd and g = gamma dy,
//   dx = dres + rstd (g - sum(g) / d - xh sum(g xh) / d)
//   dgamma = sum over rows of dy xh,   dbeta = sum over rows of dy
// Statistics, row sums and column sums are fp32; each output is rounded once.
// The mean is taken first and the variance from the centred values, so a row
// with a large common offset loses nothing.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kRowThreads = 256;

// Sums over the block; every thread gets the totals.  red: 2 x 32 floats.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    __syncthreads();  // the previous totals have been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float2 v = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

// ---------------------------------------------------------------- any width
// One block per row, three passes over the row (the second and third hit the
// caches).  A thread reads and writes the same elements in every pass, so y,
// sum_out, x and residual may be the same arrays.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
norm_rows_kernel(const T *x, const T *residual, const float *__restrict__ gamma, const float *__restrict__ beta,
                 float eps, int64_t N, int d, T *y, T *sum_out, float *mean_out, float *rstd_out) {
    __shared__ float2 red[32];
    pdl_trigger();
    pdl_wait();
    const float inv_d = 1.0f / static_cast<float>(d);
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
        const int64_t base = row * d;
        const T *h = (residual != nullptr) ? sum_out + base : x + base;
        float s = 0.0f;
        for (int i = threadIdx.x; i < d; i += kRowThreads) {
            if (residual != nullptr)
                sum_out[base + i] = from_f32<T>(to_f32<T>(x[base + i]) + to_f32<T>(residual[base + i]));
            s += to_f32<T>(h[i]);
        }
        const float mu = block_sum2(s, 0.0f, red).x * inv_d;
        float q = 0.0f;
        for (int i = threadIdx.x; i < d; i += kRowThreads) {
            const float c = to_f32<T>(h[i]) - mu;
            q += c * c;
        }
        const float rstd = 1.0f / sqrtf(block_sum2(q, 0.0f, red).x * inv_d + eps);
        for (int i = threadIdx.x; i < d; i += kRowThreads) {
            float v = (to_f32<T>(h[i]) - mu) * rstd;
            if (gamma != nullptr) v *= gamma[i];
            if (beta != nullptr) v += beta[i];
            y[base + i] = from_f32<T>(v);
        }
        if (threadIdx.x == 0) {
            if (mean_out != nullptr) mean_out[row] = mu;
            if (rstd_out != nullptr) rstd_out[row] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
norm_bwd_rows_kernel(const T *dy, const T *h, const float *__restrict__ gamma, const float *__restrict__ mean,
                     const float *__restrict__ rstd, const T *dres, int64_t N, int d, T *dx) {
    __shared__ float2 red[32];
    pdl_trigger();
    pdl_wait();
    const float inv_d = 1.0f / static_cast<float>(d);
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
        const int64_t base = row * d;
        const float mu = mean[row], rs = rstd[row];
        float a = 0.0f, b = 0.0f;
        for (int i = threadIdx.x; i < d; i += kRowThreads) {
            const float g = to_f32<T>(dy[base + i]) * (gamma != nullptr ? gamma[i] : 1.0f);
            a += g;
            b += g * ((to_f32<T>(h[base + i]) - mu) * rs);
        }
        const float2 t = block_sum2(a, b, red);
        const float ma = t.x * inv_d, mb = t.y * inv_d;
        for (int i = threadIdx.x; i < d; i += kRowThreads) {
            const float g = to_f32<T>(dy[base + i]) * (gamma != nullptr ? gamma[i] : 1.0f);
            const float xh = (to_f32<T>(h[base + i]) - mu) * rs;
            float v = rs * (g - ma - xh * mb);
            if (dres != nullptr) v += to_f32<T>(dres[base + i]);
            dx[base + i] = from_f32<T>(v);
        }
    }
}

// Column sums of dy xh and dy over a chunk of rows: a block takes 32 columns,
// its 8 warps every eighth row of the chunk.  part: [chunks][2][d].
template <typename T>
__global__ void __launch_bounds__(256)
norm_bwd_cols_kernel(const T *__restrict__ dy, const T *__restrict__ h, const float *__restrict__ mean,
                     const float *__restrict__ rstd, int64_t N, int d, int64_t chunk_rows, float *part) {
    __shared__ float2 red[8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * chunk_rows;
    const int64_t r1 = r0 + chunk_rows < N ? r0 + chunk_rows : N;
    float a = 0.0f, b = 0.0f;
    if (col < d)
        for (int64_t r = r0 + warp; r < r1; r += 8) {
            const float v = to_f32<T>(dy[r * d + col]);
            a += v * ((to_f32<T>(h[r * d + col]) - mean[r]) * rstd[r]);
            b += v;
        }
    red[warp][lane] = make_float2(a, b);
    __syncthreads();
    if (warp == 0 && col < d) {
        for (int w = 1; w < 8; ++w) {
            a += red[w][lane].x;
            b += red[w][lane].y;
        }
        float *p = part + static_cast<int64_t>(blockIdx.y) * 2 * d;
        p[col] = a;
        p[d + col] = b;
    }
}

// dgamma[c] = sum over g of part[g][0][c], dbeta[c] of part[g][1][c]: 32
// columns per block, each warp every eighth partial row, then the 8 warps in
// order.  out0/out1 nullable.
__global__ void __launch_bounds__(256)
col_reduce_kernel(const float *part, int64_t groups, int d, float *out0, float *out1) {
    __shared__ float red[8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float *out = blockIdx.y == 0 ? out0 : out1;
    if (out == nullptr) return;
    float a = 0.0f;
    if (col < d)
        for (int64_t g = warp; g < groups; g += 8) a += part[(2 * g + blockIdx.y) * d + col];
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < d) {
        for (int w = 1; w < 8; ++w) a += red[w][lane];
        out[col] = a;
    }
}

constexpr int kMaxChunks = 64;

int64_t col_chunks(int64_t N) {
    int64_t c = (N + 255) / 256;
    return c < 1 ? 1 : c > kMaxChunks ? kMaxChunks : c;
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t N, int d) {
    return align_up(static_cast<size_t>(col_chunks(N)) * 2 * d * sizeof(float), 256);
}

cudaError_t launch_norm(const void *x, const void *residual, int dt, const float *gamma, const float *beta, float eps,
                        int64_t N, int d, void *y, void *sum_out, float *mean, float *rstd, int num_sms,
                        cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(N < cap ? N : cap));
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return launch_pdl(norm_rows_kernel<T>, grid, dim3(kRowThreads), 0, s, static_cast<const T *>(x),
                          static_cast<const T *>(residual), gamma, beta, eps, N, d, static_cast<T *>(y),
                          static_cast<T *>(sum_out), mean, rstd);
    };
    return dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

cudaError_t launch_norm_bwd(const void *dy, const void *h, int dt, const float *gamma, const float *mean,
                            const float *rstd, const void *dres, int64_t N, int d, void *dx, float *dgamma,
                            float *dbeta, void *ws, int num_sms, cudaStream_t s) {
    if (N == 0) {
        cudaError_t e = cudaSuccess;
        if (dgamma != nullptr) e = cudaMemsetAsync(dgamma, 0, sizeof(float) * static_cast<size_t>(d), s);
        if (e == cudaSuccess && dbeta != nullptr) e = cudaMemsetAsync(dbeta, 0, sizeof(float) * static_cast<size_t>(d), s);
        return e;
    }
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(N < cap ? N : cap));
    float *part = static_cast<float *>(ws);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        cudaError_t e = cudaSuccess;
        if (dgamma != nullptr || dbeta != nullptr) {
            // the column sums first: dx may be the array dy or h
            const int64_t chunks = col_chunks(N);
            const unsigned cols = static_cast<unsigned>((static_cast<int64_t>(d) + 31) / 32);
            e = launch_pdl(norm_bwd_cols_kernel<T>, dim3(cols, static_cast<unsigned>(chunks)), dim3(256), 0, s,
                           static_cast<const T *>(dy), static_cast<const T *>(h), mean, rstd, N, d,
                           (N + chunks - 1) / chunks, part);
            if (e != cudaSuccess) return e;
            e = launch_pdl(col_reduce_kernel, dim3(cols, 2), dim3(256), 0, s, part, chunks, d, dgamma, dbeta);
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(norm_bwd_rows_kernel<T>, grid, dim3(kRowThreads), 0, s, static_cast<const T *>(dy),
                          static_cast<const T *>(h), gamma, mean, rstd, static_cast<const T *>(dres), N, d,
                          static_cast<T *>(dx));
    };
    return dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace moe
