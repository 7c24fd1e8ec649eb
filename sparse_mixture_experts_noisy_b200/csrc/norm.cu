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
#include "colsum.cuh"
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

// ---------------------------------------------------------------- rows held in registers
// A group of TPR threads (a warp or several; several groups to a block) takes
// rows g, g + G, g + 2G, ... and holds the row it works on in registers as
// 16-byte vectors, thread t the vectors t, t + TPR, ...  The vectors of the next
// DEPTH rows are on their way into shared memory meanwhile (cp.async).  Each
// thread copies only what it will read itself, so the ring needs no barrier.
//
// Rows of any width use full vectors.  Vectors are aligned in memory, so a row
// whose start is `off` elements past a vector boundary covers a first and a
// last vector in part; the elements outside are masked out of the sums, and
// those vectors are stored element by element.  G is a multiple of
// P = VEC / gcd(d, VEC), the period of off over the rows, so off is the same for
// all rows of a group and a thread's columns never move: gamma, beta and the
// column sums stay in registers for the whole kernel.  A vector that reaches
// past the row's end reads the next row's first elements; past the end of the
// array itself the copy stops and fills with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Launch shapes by threads a row and elements a thread.  A warp that holds 24
// elements a lane needs up to 190 registers in the backward: 256 threads.
template <int TPR, int EPT> struct NormCfg {
    static constexpr bool LONG = TPR == 32 && EPT > 16;
    static constexpr bool HOLD = TPR < 512 || EPT <= 16;  // gamma, beta, column sums in registers
    static constexpr int THREADS = LONG ? 256 : 512, FWD_PER_SM = (LONG || EPT == 8) ? 2 : 1;
};
// Rows on their way: six, or as many as `budget` bytes of shared memory hold.
// The budget is what keeps HBM busy, 64 KB an SM of forward rows and 112 KB of
// backward rows: 32768 x 2048 forward takes 92.5 us with 64 KB, 96 with 32 and 98
// with 100; 16384 x 4096 backward 82.7 us with 112 KB, 104 with 80, 84.3 with 200.
constexpr int ring_depth(int arrays, int ch, int threads, int budget) {
    const int n = budget / (arrays * ch * threads * 16);
    return n > 6 ? 6 : n < 1 ? 1 : n;
}
template <int TPR, int EPT> constexpr int fwd_depth(int arrays, int ch) {
    return ring_depth(arrays, ch, NormCfg<TPR, EPT>::THREADS, 64 * 1024 / NormCfg<TPR, EPT>::FWD_PER_SM);
}
template <int TPR, int EPT> constexpr int bwd_depth(int arrays, int ch) {
    return ring_depth(arrays, ch, NormCfg<TPR, EPT>::THREADS, 112 * 1024);
}

template <typename T, int TPR, int CH, bool AL>
struct RowLayout {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    static constexpr int EPT = VEC * CH;
    static constexpr uint32_t FULL = (1u << VEC) - 1;
    int d, off, t;
    uint32_t keep[AL ? 1 : CH];  // which elements of vector c lie inside the row
    __device__ __forceinline__ RowLayout(int d_, int off_, int t_) : d(d_), off(off_), t(t_) {
        if constexpr (!AL) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int lo = -first(c), hi = d - first(c);  // elements [lo, hi)
                uint32_t m = hi >= VEC ? FULL : hi > 0 ? (1u << hi) - 1u : 0u;
                if (lo > 0) m &= FULL << lo;
                keep[c] = m;
            }
        }
    }
    __device__ __forceinline__ int first(int c) const { return (t + c * TPR) * VEC - (AL ? 0 : off); }
    __device__ __forceinline__ bool any(int c) const { return AL ? first(c) < d : keep[AL ? 0 : c] != 0u; }
    __device__ __forceinline__ bool whole(int c) const { return AL ? first(c) < d : keep[AL ? 0 : c] == FULL; }
    __device__ __forceinline__ bool in(int c, int i) const {
        return AL ? first(c) < d : ((keep[AL ? 0 : c] >> i) & 1u) != 0u;
    }
    // v with zeros in place of what lies outside the row (the vector may never
    // have been fetched).
    __device__ __forceinline__ void inside(float (&v)[VEC], int c) const {
        if (!whole(c)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = (!AL && in(c, i)) ? v[i] : 0.0f;
        }
    }
    // Starts the copy of the row at p (its first element) into this thread's
    // slots, `step` bytes apart; left: elements from p to the array's end.
    __device__ __forceinline__ void fetch(const T *p, int64_t left, uint32_t slot, uint32_t step) const {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (any(c)) {
                int n = 16;
                if (!AL && first(c) + VEC > left) n = static_cast<int>(left - first(c)) * static_cast<int>(sizeof(T));
                copy16(slot + c * step, p + first(c), n);
            }
    }
    __device__ __forceinline__ void store(T *p, int c, const uint4 &raw) const {
        if (whole(c)) {
            *reinterpret_cast<uint4 *>(p + first(c)) = raw;
        } else if (any(c)) {
            const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (in(c, i)) p[first(c) + i] = e[i];
        }
    }
    // This thread's columns of an fp32 vector of length d (`other` outside it and
    // when w is null).  Inside the row they come in aligned 16-byte pieces,
    // shifted by the row's offset (off mod 4, the same for the whole group).
    __device__ __forceinline__ void columns(const float *w, float other, int c, float (&v)[VEC]) const {
        if (w == nullptr || !whole(c)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = (!AL && w != nullptr && in(c, i)) ? w[first(c) + i] : other;
            return;
        }
        const int shift = AL ? 0 : (4 - (off & 3)) & 3;  // first(c) mod 4
        const float4 *q = reinterpret_cast<const float4 *>(w + first(c) - shift);
        float f[VEC + 4];
#pragma unroll
        for (int k = 0; k < VEC / 4 + (AL ? 0 : 1); ++k) {
            float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < VEC / 4 || shift != 0) {
                if (k < VEC / 4 || first(c) - shift + VEC + 4 <= d) {
                    u = q[k];
                } else {  // the last piece would leave the vector
                    const float *r = reinterpret_cast<const float *>(q + k);
                    u.x = r[0];
                    if (shift > 1) u.y = r[1];
                    if (shift > 2) u.z = r[2];
                }
            }
            f[4 * k] = u.x;
            f[4 * k + 1] = u.y;
            f[4 * k + 2] = u.z;
            f[4 * k + 3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] = AL ? f[i] : shift == 0 ? f[i] : shift == 1 ? f[i + 1] : shift == 2 ? f[i + 2] : f[i + 3];
    }
};

template <typename T> __device__ __forceinline__ float elem(const uint4 &raw, int i);
template <> __device__ __forceinline__ float elem<float>(const uint4 &raw, int i) {
    return __uint_as_float(i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w);
}
template <> __device__ __forceinline__ float elem<__nv_bfloat16>(const uint4 &raw, int i) {
    const uint32_t w = i < 2 ? raw.x : i < 4 ? raw.y : i < 6 ? raw.z : raw.w;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
template <typename T> __device__ __forceinline__ uint4 pack(const float *v);
template <> __device__ __forceinline__ uint4 pack<float>(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <> __device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float *v) {
    uint4 r;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return r;
}

// Sum over a group.  Groups of several warps use a named barrier of their own
// and one of two buffers in turn: a thread that writes a buffer again has passed
// the other one's barrier, so everyone has read it.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float (*red)[NV][32], int buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = threadIdx.x / TPR;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) red[buf][k][warp] = v[k];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "n"(TPR) : "memory");
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = red[buf][k][grp * W + (lane & (W - 1))];
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < NV; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// Rows too wide to HOLD gamma and beta read them again for each row, from the L1 cache.
// ADD: with a residual.
template <typename T, int TPR, int CH, bool AL, bool ADD>
__global__ void __launch_bounds__(NormCfg<TPR, RowLayout<T, TPR, CH, AL>::EPT>::THREADS,
                                  NormCfg<TPR, RowLayout<T, TPR, CH, AL>::EPT>::FWD_PER_SM)
norm_fwd_kernel(const T *x, const T *residual, const float *__restrict__ gamma, const float *__restrict__ beta,
                float eps, int64_t N, int d, int64_t G, T *y, T *sum_out, float *mean_out, float *rstd_out) {
    using L = RowLayout<T, TPR, CH, AL>;
    constexpr int VEC = L::VEC;
    using Cfg = NormCfg<TPR, L::EPT>;
    constexpr bool HOLD = Cfg::HOLD;
    constexpr uint32_t arrays = ADD ? 2 : 1;
    constexpr int DEPTH = fwd_depth<TPR, L::EPT>(arrays, CH), THREADS = Cfg::THREADS;
    constexpr uint32_t STEP = THREADS * 16;  // between a thread's slots
    extern __shared__ uint4 ring[];          // [DEPTH][arrays][CH][THREADS]
    __shared__ float red[2][1][32];
    pdl_trigger();
    const int t = threadIdx.x % TPR;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * (THREADS / TPR) + threadIdx.x / TPR;
    pdl_wait();
    if (g >= N) return;
    const L lay(d, AL ? 0 : static_cast<int>((g * d) % VEC), t);
    const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16;
    const int64_t total = N * d;
    const float inv_d = 1.0f / static_cast<float>(d);
    auto fetch = [&](int64_t row, int stage) {
        if (row < N) {
            const uint32_t s = slot0 + stage * arrays * CH * STEP;
            lay.fetch(x + row * d, total - row * d, s, STEP);
            if constexpr (ADD) lay.fetch(residual + row * d, total - row * d, s + CH * STEP, STEP);
        }
        copy_commit();
    };
#pragma unroll
    for (int q = 0; q < DEPTH; ++q) fetch(g + q * G, q);
    float ga[HOLD ? CH : 1][VEC], be[HOLD ? CH : 1][VEC];
    if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            lay.columns(gamma, 1.0f, c, ga[c]);
            lay.columns(beta, 0.0f, c, be[c]);
        }
    }
    int stage = 0;
    for (int64_t row = g; row < N; row += G) {
        const int64_t base = row * d;
        const uint4 *mine = ring + (stage * arrays * CH) * THREADS + threadIdx.x;
        float v[CH][VEC];
        float s[1] = {0.0f};
        copy_wait<DEPTH - 1>();
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 xr = mine[c * THREADS];
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[c][i] = elem<T>(xr, i);
            if constexpr (ADD) {
                const uint4 rr = mine[(CH + c) * THREADS];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[c][i] += elem<T>(rr, i);
                const uint4 h = pack<T>(v[c]);  // the stored sum is what is normalised
                lay.store(sum_out + base, c, h);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[c][i] = elem<T>(h, i);
            }
            lay.inside(v[c], c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += v[c][i];
        }
        group_sum<TPR>(s, red, 0);
        const float mu = s[0] * inv_d;
        fetch(row + DEPTH * G, stage);  // the slots have been read: the sum needed them
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
        s[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[c][i] -= mu;
            lay.inside(v[c], c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(v[c][i], v[c][i], s[0]);
        }
        group_sum<TPR>(s, red, 1);
        const float rstd = 1.0f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float gc[VEC], bc[VEC];
            if constexpr (!HOLD) {
                lay.columns(gamma, 1.0f, c, gc);
                lay.columns(beta, 0.0f, c, bc);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                v[c][i] = fmaf(v[c][i] * rstd, HOLD ? ga[HOLD ? c : 0][i] : gc[i], HOLD ? be[HOLD ? c : 0][i] : bc[i]);
            lay.store(y + base, c, pack<T>(v[c]));
        }
        if (t == 0) {
            if (mean_out != nullptr) mean_out[row] = mu;
            if (rstd_out != nullptr) rstd_out[row] = rstd;
        }
    }
}

// The backward: both row sums in one reduction, and the column sums of the
// group's rows in registers (HOLD) or, past 16 elements a thread, in shared
// memory, each thread its own entries.  At the end the block's groups add their
// columns in order.  part: [grid][2][d], null without column sums.  ADD: with dres.
template <typename T, int TPR, int CH, bool AL, bool ADD>
__global__ void __launch_bounds__(NormCfg<TPR, RowLayout<T, TPR, CH, AL>::EPT>::THREADS)
norm_bwd_kernel(const T *dy, const T *h, const float *__restrict__ gamma, const float *__restrict__ mean,
                const float *__restrict__ rstd, const T *dres, int64_t N, int d, int64_t G, int period, T *dx, float *part) {
    using L = RowLayout<T, TPR, CH, AL>;
    constexpr int VEC = L::VEC;
    using Cfg = NormCfg<TPR, L::EPT>;
    constexpr uint32_t arrays = ADD ? 3 : 2;
    constexpr int DEPTH = bwd_depth<TPR, L::EPT>(arrays, CH), THREADS = Cfg::THREADS, GROUPS = THREADS / TPR;
    constexpr bool HOLD = Cfg::HOLD;
    static_assert(HOLD || GROUPS == 1, "column sums in shared memory belong to one group");
    constexpr uint32_t STEP = THREADS * 16;
    extern __shared__ uint4 ring[];  // [DEPTH][arrays][CH][THREADS], then !HOLD: [2][CH][VEC][THREADS] floats
    __shared__ float red[2][2][32];
    pdl_trigger();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    // block b's groups take the rows b mod P, P apart, so that they share `off`
    const int P = AL ? 1 : static_cast<int>(period);
    const int64_t g = blockIdx.x % P + static_cast<int64_t>(P) * (static_cast<int64_t>(blockIdx.x / P) * GROUPS + grp);
    const L lay(d, AL ? 0 : static_cast<int>((g * d) % VEC), t);
    const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16;
    float *cols = reinterpret_cast<float *>(ring + (HOLD ? 0 : DEPTH * arrays * CH * THREADS));
    const int64_t total = N * d;
    const float inv_d = 1.0f / static_cast<float>(d);
    float ga[HOLD ? CH : 1][VEC], ag[HOLD ? CH : 1][VEC], ab[HOLD ? CH : 1][VEC];
    if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) ag[c][i] = ab[c][i] = 0.0f;
    } else {
        for (int q = 0; q < 2 * CH * VEC; ++q) cols[q * THREADS + threadIdx.x] = 0.0f;
    }
    auto fetch = [&](int64_t row, int stage) {
        if (row < N) {
            const uint32_t s = slot0 + stage * arrays * CH * STEP;
            lay.fetch(dy + row * d, total - row * d, s, STEP);
            lay.fetch(h + row * d, total - row * d, s + CH * STEP, STEP);
            if constexpr (ADD) lay.fetch(dres + row * d, total - row * d, s + 2 * CH * STEP, STEP);
        }
        copy_commit();
    };
    pdl_wait();
#pragma unroll
    for (int q = 0; q < DEPTH; ++q) fetch(g + q * G, q);
    float mu = 0.0f, rs = 0.0f;
    if (g < N) {
        mu = mean[g];
        rs = rstd[g];
    }
    if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < CH; ++c) lay.columns(gamma, 1.0f, c, ga[c]);
    }
    int stage = 0, buf = 0;
    for (int64_t row = g; row < N; row += G) {
        const int64_t base = row * d;
        const uint4 *mine = ring + (stage * arrays * CH) * THREADS + threadIdx.x;
        float xh[CH][VEC], gy[CH][VEC];
        uint4 dr[CH];
        float s[2] = {0.0f, 0.0f};
        copy_wait<DEPTH - 1>();
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 yr = mine[c * THREADS], hr = mine[(CH + c) * THREADS];
            float yv[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                yv[i] = elem<T>(yr, i);
                xh[c][i] = (elem<T>(hr, i) - mu) * rs;
            }
            lay.inside(yv, c);
            lay.inside(xh[c], c);
            if constexpr (ADD) dr[c] = mine[(2 * CH + c) * THREADS];
            float gc[VEC];
            if constexpr (!HOLD) lay.columns(gamma, 1.0f, c, gc);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = yv[i];
                gy[c][i] = v * (HOLD ? ga[HOLD ? c : 0][i] : gc[i]);
                s[0] += gy[c][i];
                s[1] = fmaf(gy[c][i], xh[c][i], s[1]);
                if constexpr (HOLD) {
                    ag[c][i] = fmaf(v, xh[c][i], ag[c][i]);
                    ab[c][i] += v;
                } else {
                    float *p = cols + (c * VEC + i) * THREADS + threadIdx.x;
                    p[0] = fmaf(v, xh[c][i], p[0]);
                    p[CH * VEC * THREADS] += v;
                }
            }
        }
        const float rs_row = rs;
        if (row + G < N) {
            mu = mean[row + G];
            rs = rstd[row + G];
        }
        group_sum<TPR>(s, red, buf);
        buf ^= 1;
        if constexpr (ADD) {
#pragma unroll
            for (int c = 0; c < CH; ++c) asm volatile("" ::"r"(dr[c].x), "r"(dr[c].y), "r"(dr[c].z), "r"(dr[c].w));
        }
        fetch(row + DEPTH * G, stage);  // the slots have been read
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
        const float ma = s[0] * inv_d, mb = s[1] * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                gy[c][i] = rs_row * (gy[c][i] - ma - xh[c][i] * mb);
                if constexpr (ADD) gy[c][i] += elem<T>(dr[c], i);
            }
            lay.store(dx + base, c, pack<T>(gy[c]));
        }
    }
    if (part == nullptr) return;
    float *p0 = part + static_cast<int64_t>(blockIdx.x) * 2 * d, *p1 = p0 + d;
    if constexpr (GROUPS > 1) {
        // every group leaves its sums in shared memory (rows of TPR threads, 4 floats
        // apart in the banks), and the block adds them column by column
        constexpr int Q = CH * VEC, LD = TPR + 4;
        cols = reinterpret_cast<float *>(ring);  // [GROUPS][2 Q][LD]
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float *q = cols + (grp * 2 * Q + c * VEC + i) * LD + t;
                q[0] = ag[c][i];
                q[Q * LD] = ab[c][i];
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * d; e += THREADS) {
            const int at = (e < d ? e : e - d) + lay.off, vec = at / VEC;
            const float *q = cols + ((e < d ? 0 : Q) + vec / TPR * VEC + at % VEC) * LD + vec % TPR;
            float a = 0.0f;
#pragma unroll
            for (int w = 0; w < GROUPS; ++w) a += q[w * 2 * Q * LD];
            p0[e] = a;
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (lay.in(c, i)) {
                    const int e = lay.first(c) + i;
                    p0[e] = HOLD ? ag[HOLD ? c : 0][i] : cols[(c * VEC + i) * THREADS + threadIdx.x];
                    p1[e] = HOLD ? ab[HOLD ? c : 0][i] : cols[(CH * VEC + c * VEC + i) * THREADS + threadIdx.x];
                }
    }
}

constexpr int kNormSms = 148;  // groups are counted for a B200; the bits then do not depend on the device

// Threads a row and elements a thread for rows of d elements (0: too wide for
// registers).  A row that starts inside a vector needs up to VEC - 1 more.
// Few threads a row save reductions and barriers, few elements a thread save
// registers.  Measured on a B200, calls replayed in a graph: backward 8192 x 768
// bf16 12.3 us with 32 x 24 against 15.5 with 128 x 8; forward 8191 x 1001 bf16
// 13.8 us with 64 x 16 against 14.7 with 32 x 32.
struct NormShape {
    int tpr, ept;
};
NormShape norm_shape(int d, int vec) {
    const int need = d + (d % vec != 0 ? vec - 1 : 0);
    if (need <= 256) return {32, 8};
    if (need <= 512) return {32, 16};
    if (need <= 768) return {32, 24};
    if (need <= 1024) return {64, 16};
    if (need <= 2048) return {128, 16};
    if (need <= 4096) return {256, 16};
    if (need <= 8192) return {512, 16};
    if (need <= 16384) return {512, 32};
    return {0, 0};
}

// The forward's shape: many bf16 rows take 32 elements a thread (16384 x 4096
// without a residual 45 against 58 us); few rows do not (64 x 4096 3.9 against
// 3.3 us), nor fp32 rows (8192 x 4096 44.3 against 42.5 us).
NormShape fwd_shape(int64_t N, int d, int vec) {
    NormShape f = norm_shape(d, vec);
    if (vec == 8 && N >= 8 * 148 && f.ept == 16 && f.tpr >= 128) f = {f.tpr / 2, 32};
    return f;
}

// The backward's shape.  Rows of 1025 to 2048 elements that start inside a vector
// would spill registers with 16 elements a thread (1000 x 1337 fp32 11.5 us; 9.8
// with 256 x 8), whole ones do not (32768 x 2048 bf16 83 us; 98 with 256 x 8).
// fp32 rows past 8192 elements would need 288 KB of shared memory for one row and
// the column sums, so they go to the kernels for any width.
NormShape bwd_shape(int d, int vec) {
    const NormShape f = norm_shape(d, vec);
    if (f.tpr == 128 && d % vec != 0) return {256, 8};
    return f.ept > 24 && vec == 4 ? NormShape{0, 0} : f;
}

int64_t row_period(int d, int vec) {
    int a = d, b = vec;
    while (b != 0) {
        const int r = a % b;
        a = b;
        b = r;
    }
    return vec / a;
}

// Blocks of rpb groups for N rows: at most per_sm on each SM, at least min_rows
// rows a group as long as every SM has a block, and a multiple of the row period.
int64_t norm_blocks(int64_t N, int d, int vec, int rpb, int per_sm, int min_rows) {
    const int64_t p = row_period(d, vec);
    const int64_t all = (N + rpb - 1) / rpb;
    int64_t b = static_cast<int64_t>(kNormSms) * per_sm;
    const int64_t few = N / (static_cast<int64_t>(min_rows) * rpb);
    if (b > few) b = few > kNormSms ? few : kNormSms;
    return b >= all ? (all + p - 1) / p * p : b / p * p;
}

constexpr int kBwdMinRows = 2;

// f(tag of TPR, tag of CH, tag of AL) for the shape.
template <int V> struct Int {
    static constexpr int value = V;
};
template <typename T, typename F>
cudaError_t norm_pick(NormShape n, bool al, F f) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    auto with = [&](auto tpr, auto ept) {
        using CH = Int<decltype(ept)::value / VEC>;
        return al ? f(tpr, CH{}, Int<1>{}) : f(tpr, CH{}, Int<0>{});
    };
    if (n.tpr == 32 && n.ept <= 16) return n.ept == 8 ? with(Int<32>{}, Int<8>{}) : with(Int<32>{}, Int<16>{});
    if (n.tpr == 32) return with(Int<32>{}, Int<24>{});
    if (n.tpr == 64) return n.ept == 16 ? with(Int<64>{}, Int<16>{}) : with(Int<64>{}, Int<32>{});
    if (n.tpr == 128) return n.ept == 16 ? with(Int<128>{}, Int<16>{}) : with(Int<128>{}, Int<32>{});
    if (n.tpr == 256 && n.ept == 32) return with(Int<256>{}, Int<32>{});
    if (n.tpr == 256) return n.ept == 8 ? with(Int<256>{}, Int<8>{}) : with(Int<256>{}, Int<16>{});
    return n.ept == 16 ? with(Int<512>{}, Int<16>{}) : with(Int<512>{}, Int<32>{});
}

// The attribute belongs to the current device's context, so it is set on every call.
template <typename K> cudaError_t allow_smem(K kern, size_t bytes) {
    if (bytes <= 40 * 1024) return cudaSuccess;  // with the static arrays, within the default 48 KB
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

constexpr int kMaxChunks = 64;

int64_t col_chunks(int64_t N) {
    int64_t c = (N + 255) / 256;
    return c < 1 ? 1 : c > kMaxChunks ? kMaxChunks : c;
}

// Rows of the backward's partial column sums.
int64_t bwd_part_rows(int64_t N, int d, int vec) {
    const NormShape f = bwd_shape(d, vec);
    if (f.tpr == 0) return col_chunks(N);
    return norm_blocks(N, d, vec, (f.tpr == 32 && f.ept > 16 ? 256 : 512) / f.tpr, 1, kBwdMinRows);
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t N, int d, int dt) {
    const int64_t rows = bwd_part_rows(N, d, dt == 1 ? 8 : 4);
    return align_up(static_cast<size_t>(rows < 1 ? 1 : rows) * 2 * d * sizeof(float), 256);
}

cudaError_t launch_norm(const void *x, const void *residual, int dt, const float *gamma, const float *beta, float eps,
                        int64_t N, int d, void *y, void *sum_out, float *mean, float *rstd, cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        constexpr int VEC = 16 / static_cast<int>(sizeof(T));
        const NormShape f = fwd_shape(N, d, VEC);
        if (f.tpr == 0) {
            const int64_t cap = static_cast<int64_t>(kNormSms) * 8;
            return launch_pdl(norm_rows_kernel<T>, dim3(static_cast<unsigned>(N < cap ? N : cap)), dim3(kRowThreads), 0,
                              s, static_cast<const T *>(x), static_cast<const T *>(residual), gamma, beta, eps, N, d,
                              static_cast<T *>(y), static_cast<T *>(sum_out), mean, rstd);
        }
        return norm_pick<T>(f, d % VEC == 0, [&](auto tpr, auto ch, auto al) {
            constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
            using Cfg = NormCfg<TPR, CH * VEC>;
            constexpr int GROUPS = Cfg::THREADS / TPR;
            if constexpr (CH * VEC == 32 && TPR < 512 && VEC == 4) {
                return cudaErrorInvalidValue;  // fwd_shape never picks it
            } else {
                const int64_t blocks = norm_blocks(N, d, VEC, GROUPS, Cfg::FWD_PER_SM, 1);
                auto with = [&](auto add) {
                    constexpr bool ADD = decltype(add)::value != 0;
                    constexpr size_t smem =
                        static_cast<size_t>(fwd_depth<TPR, CH * VEC>(ADD ? 2 : 1, CH)) * (ADD ? 2 : 1) * CH * Cfg::THREADS * 16;
                    auto kern = norm_fwd_kernel<T, TPR, CH, decltype(al)::value != 0, ADD>;
                    cudaError_t e = allow_smem(kern, smem);
                    if (e != cudaSuccess) return e;
                    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(Cfg::THREADS), smem, s,
                                      static_cast<const T *>(x), static_cast<const T *>(residual), gamma, beta, eps, N, d,
                                      blocks * GROUPS, static_cast<T *>(y), static_cast<T *>(sum_out), mean, rstd);
                };
                return residual != nullptr ? with(Int<1>{}) : with(Int<0>{});
            }
        });
    };
    return dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

cudaError_t launch_norm_bwd(const void *dy, const void *h, int dt, const float *gamma, const float *mean,
                            const float *rstd, const void *dres, int64_t N, int d, void *dx, float *dgamma,
                            float *dbeta, void *ws, cudaStream_t s) {
    if (N == 0) {
        cudaError_t e = cudaSuccess;
        if (dgamma != nullptr) e = cudaMemsetAsync(dgamma, 0, sizeof(float) * static_cast<size_t>(d), s);
        if (e == cudaSuccess && dbeta != nullptr) e = cudaMemsetAsync(dbeta, 0, sizeof(float) * static_cast<size_t>(d), s);
        return e;
    }
    const bool sums = dgamma != nullptr || dbeta != nullptr;
    float *part = sums ? static_cast<float *>(ws) : nullptr;
    const unsigned cols = static_cast<unsigned>((static_cast<int64_t>(d) + 31) / 32);
    const int64_t rows = bwd_part_rows(N, d, dt == 1 ? 8 : 4);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        constexpr int VEC = 16 / static_cast<int>(sizeof(T));
        const NormShape f = bwd_shape(d, VEC);
        cudaError_t e = cudaSuccess;
        if (f.tpr == 0) {
            if (sums) {
                // the column sums first: dx may be the array dy or h
                e = launch_pdl(norm_bwd_cols_kernel<T>, dim3(cols, static_cast<unsigned>(rows)), dim3(256), 0, s,
                               static_cast<const T *>(dy), static_cast<const T *>(h), mean, rstd, N, d,
                               (N + rows - 1) / rows, part);
                if (e != cudaSuccess) return e;
            }
            const int64_t cap = static_cast<int64_t>(kNormSms) * 8;
            return launch_pdl(norm_bwd_rows_kernel<T>, dim3(static_cast<unsigned>(N < cap ? N : cap)), dim3(kRowThreads),
                              0, s, static_cast<const T *>(dy), static_cast<const T *>(h), gamma, mean, rstd,
                              static_cast<const T *>(dres), N, d, static_cast<T *>(dx));
        }
        return norm_pick<T>(f, d % VEC == 0, [&](auto tpr, auto ch, auto al) {
            constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
            using Cfg = NormCfg<TPR, CH * VEC>;
            if constexpr (CH * VEC == 32 && (VEC == 4 || TPR < 512)) {
                return cudaErrorInvalidValue;  // bwd_shape never picks it
            } else {
                constexpr int GROUPS = Cfg::THREADS / TPR;
                auto with = [&](auto add) {
                    constexpr bool ADD = decltype(add)::value != 0;
                    constexpr size_t ring = static_cast<size_t>(bwd_depth<TPR, CH * VEC>(ADD ? 3 : 2, CH)) * (ADD ? 3 : 2) *
                                            CH * Cfg::THREADS * 16;
                    // the column sums lie behind the ring (!HOLD) or, at the end, over it
                    constexpr size_t own = Cfg::HOLD ? 0 : 2 * sizeof(float) * CH * VEC * Cfg::THREADS;
                    constexpr size_t sums = GROUPS > 1 ? sizeof(float) * GROUPS * 2 * CH * VEC * (TPR + 4) : 0;
                    constexpr size_t smem = ring + own > sums ? ring + own : sums;
                    auto kern = norm_bwd_kernel<T, TPR, CH, decltype(al)::value != 0, ADD>;
                    cudaError_t e = allow_smem(kern, smem);
                    if (e != cudaSuccess) return e;
                    return launch_pdl(kern, dim3(static_cast<unsigned>(rows)), dim3(Cfg::THREADS), smem, s,
                                      static_cast<const T *>(dy), static_cast<const T *>(h), gamma, mean, rstd,
                                      static_cast<const T *>(dres), N, d, rows * GROUPS,
                                      static_cast<int>(row_period(d, VEC)), static_cast<T *>(dx), part);
                };
                return dres != nullptr ? with(Int<1>{}) : with(Int<0>{});
            }
        });
    };
    cudaError_t e = dt == 1 ? go(__nv_bfloat16{}) : go(float{});
    if (e != cudaSuccess || !sums) return e;
    return launch_col_reduce(part, rows, d, 2, dgamma, dbeta, s);
}

}  // namespace moe
