// The dense layer beside the experts (a shared expert's or a dense block's
// projections) and its backward pass:
//   z = x W^T + b,  y = round(act(z) + residual),  z_out = round(z)
//   dZ = dy act'(z),  dx = dZ W,  dW = dZ^T x,  db = sum over rows of dZ
// This file holds the CUDA-core products, which take every type, size and
// alignment, and the host-side choice between them and the tensor cores.
#include "common.cuh"
#include "internal.h"
#include "linear.cuh"

namespace moe {

// The dense layer's status word on each device (bounded waits of its kernels).
static __device__ uint32_t g_linear_status;

cudaError_t linear_status_read_clear(uint32_t *word, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_linear_status, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    static const uint32_t zero = 0u;
    e = cudaMemcpyToSymbolAsync(g_linear_status, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

namespace {

// ---------------------------------------------------------------- any size, on CUDA cores
// C[i][j] = sum_k A(i, k) B(j, k) in fp32, 64 x 64 tiles, 4 x 4 per thread.
// A(i, k) = A[i * ai + k * ak], and B alike, so one kernel serves the forward
// (both rows contiguous), dx (B column-strided) and dW (both).
struct SimtArgs {
    const void *A, *B;
    int64_t ai, ak, bj, bk;
    int64_t M, Nn, K;
    LinearEpi epi;
};

template <typename T>
__global__ void __launch_bounds__(256)
linear_simt_kernel(const SimtArgs p) {
    constexpr int BT = 64, BK = 16;
    __shared__ float As[BK][BT + 1], Bs[BK][BT + 1];
    pdl_trigger();
    pdl_wait();
    const T *A = static_cast<const T *>(p.A), *B = static_cast<const T *>(p.B);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * BT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.y) * BT; i0 < p.M; i0 += static_cast<int64_t>(gridDim.y) * BT) {
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
            for (int q = threadIdx.x; q < BT * BK; q += 256) {
                // neighbouring threads along the contiguous axis
                const int ai = (p.ak == 1) ? q / BK : q % BT, akk = (p.ak == 1) ? q % BK : q / BT;
                const int bj = (p.bk == 1) ? q / BK : q % BT, bkk = (p.bk == 1) ? q % BK : q / BT;
                As[akk][ai] = (i0 + ai < p.M && k0 + akk < p.K) ? to_f32<T>(A[(i0 + ai) * p.ai + (k0 + akk) * p.ak]) : 0.0f;
                Bs[bkk][bj] = (j0 + bj < p.Nn && k0 + bkk < p.K) ? to_f32<T>(B[(j0 + bj) * p.bj + (k0 + bkk) * p.bk]) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < BK; ++k) {
                float a[4], b[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    a[u] = As[k][ty + 16 * u];
                    b[u] = Bs[k][tx + 16 * u];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(a[u], b[v], acc[u][v]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
                if (i < p.M && j < p.Nn) linear_store<T>(p.epi, i, j, p.Nn, acc[u][v]);
            }
    }
}

template <typename T>
cudaError_t launch_simt(const SimtArgs &p, cudaStream_t s) {
    const int64_t gy = (p.M + 63) / 64;
    return launch_pdl(linear_simt_kernel<T>,
                      dim3(static_cast<unsigned>((p.Nn + 63) / 64), static_cast<unsigned>(gy < 32768 ? gy : 32768)),
                      dim3(256), 0, s, p);
}

// ---------------------------------------------------------------- dZ and db
// dZ = dy act'(z), rounded to the storage type, and the column sums of the
// unrounded dZ over a chunk of rows.  A block takes 32 columns, its 8 warps
// every eighth row of the chunk.
template <typename T>
__global__ void __launch_bounds__(256)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, int act, int64_t M, int n, int64_t chunk_rows,
                 T *dz, float *part) {
    __shared__ float red[8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * chunk_rows;
    const int64_t r1 = r0 + chunk_rows < M ? r0 + chunk_rows : M;
    float a = 0.0f;
    if (col < n)
        for (int64_t r = r0 + warp; r < r1; r += 8) {
            float v = to_f32<T>(dy[r * n + col]);
            if (act != kActNone) v = act_backward(v, to_f32<T>(z[r * n + col]), act);
            a += v;
            if (dz != nullptr) dz[r * n + col] = from_f32<T>(v);
        }
    if (part == nullptr) return;
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < n) {
        for (int w = 1; w < 8; ++w) a += red[w][lane];
        part[static_cast<int64_t>(blockIdx.y) * n + col] = a;
    }
}

__global__ void __launch_bounds__(256)
linear_db_kernel(const float *part, int64_t groups, int n, float *db) {
    __shared__ float red[8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (col < n)
        for (int64_t g = warp; g < groups; g += 8) a += part[g * n + col];
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < n) {
        for (int w = 1; w < 8; ++w) a += red[w][lane];
        db[col] = a;
    }
}

int64_t row_chunks(int64_t M) {
    int64_t c = (M + 255) / 256;
    return c < 1 ? 1 : c > 64 ? 64 : c;
}

}  // namespace

size_t linear_ws_bytes(int64_t, int, int, int) { return 0; }

cudaError_t launch_linear(const LinearArgs &a, void *, uint64_t, int, cudaStream_t s) {
    if (a.M == 0) return cudaSuccess;
    SimtArgs p{a.x, a.W, a.d_in, 1, a.d_in, 1, a.M, a.d_out, a.d_in, {a.b, a.act, a.residual, a.y, a.z_out}};
    return a.dt == 1 ? launch_simt<__nv_bfloat16>(p, s) : launch_simt<float>(p, s);
}

namespace {

// Byte offsets inside the backward workspace: dZ of the storage type, and the
// row chunks' partial sums of db.
struct BwdScratch {
    size_t dz, part, total;
};

BwdScratch bwd_scratch(int64_t M, int d_out, int dt, int act) {
    BwdScratch L{};
    size_t o = 0;
    L.dz = o;
    if (act != kActNone) o += align_up(static_cast<size_t>(M) * d_out * (dt == 1 ? 2 : 4), 256);
    L.part = o;
    o += align_up(static_cast<size_t>(row_chunks(M)) * d_out * sizeof(float), 256);
    L.total = o;
    return L;
}

}  // namespace

size_t linear_bwd_ws_bytes(int64_t M, int, int d_out, int dt, int act) { return bwd_scratch(M, d_out, dt, act).total; }

cudaError_t launch_linear_bwd(const LinearBwdArgs &a, void *ws, uint64_t, int, cudaStream_t s) {
    const size_t es = a.dt == 1 ? 2 : 4;
    cudaError_t e = cudaSuccess;
    if (a.M == 0) {
        if (a.dW != nullptr) e = cudaMemsetAsync(a.dW, 0, es * static_cast<size_t>(a.d_in) * a.d_out, s);
        if (e == cudaSuccess && a.db != nullptr) e = cudaMemsetAsync(a.db, 0, sizeof(float) * static_cast<size_t>(a.d_out), s);
        return e;
    }
    const BwdScratch L = bwd_scratch(a.M, a.d_out, a.dt, a.act);
    uint8_t *w = static_cast<uint8_t *>(ws);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        cudaError_t e = cudaSuccess;
        const bool need_dz = a.act != kActNone && (a.dx != nullptr || a.dW != nullptr);
        T *dzw = need_dz ? reinterpret_cast<T *>(w + L.dz) : nullptr;
        float *part = a.db != nullptr ? reinterpret_cast<float *>(w + L.part) : nullptr;
        const unsigned cols = static_cast<unsigned>((static_cast<int64_t>(a.d_out) + 31) / 32);
        const int64_t chunks = row_chunks(a.M);
        if (dzw != nullptr || part != nullptr) {
            e = launch_pdl(linear_dz_kernel<T>, dim3(cols, static_cast<unsigned>(chunks)), dim3(256), 0, s,
                           static_cast<const T *>(a.dy), static_cast<const T *>(a.z), a.act, a.M, a.d_out,
                           (a.M + chunks - 1) / chunks, dzw, part);
            if (e != cudaSuccess) return e;
        }
        if (part != nullptr) {
            e = launch_pdl(linear_db_kernel, dim3(cols), dim3(256), 0, s, part, chunks, a.d_out, a.db);
            if (e != cudaSuccess) return e;
        }
        const void *dz = a.act == kActNone ? a.dy : static_cast<const void *>(dzw);
        if (a.dx != nullptr) {
            SimtArgs p{dz, a.W, a.d_out, 1, 1, a.d_in, a.M, a.d_in, a.d_out, {nullptr, kActNone, nullptr, a.dx, nullptr}};
            if ((e = launch_simt<T>(p, s)) != cudaSuccess) return e;
        }
        if (a.dW != nullptr) {
            SimtArgs p{dz, a.x, 1, a.d_out, 1, a.d_in, a.d_out, a.d_in, a.M, {nullptr, kActNone, nullptr, a.dW, nullptr}};
            if ((e = launch_simt<T>(p, s)) != cudaSuccess) return e;
        }
        return e;
    };
    return a.dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace moe
