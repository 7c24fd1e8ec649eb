// The dense layer beside the experts (a shared expert's or a dense block's
// projections) and its backward pass:
//   z = x W^T + b,  y = round(act(z) + residual),  z_out = round(z)
//   dZ = dy act'(z),  dx = dZ W,  dW = dZ^T x,  db = sum over rows of dZ
// This file holds the CUDA-core products, which take every type, size and
// alignment, and the host-side choice between them and the tensor cores.
#include "common.cuh"
#include "internal.h"
#include "linear.cuh"
#include "linear_tc.h"

namespace moe {

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

// ---------------------------------------------------------------- operands for the tensor cores
// v = p0 + p1 + p2 in bf16 parts (each the rest rounded to bf16; the rests are
// exact in fp32).  A value above bf16's largest, 3.39e38, has no such parts.
__device__ __forceinline__ void bf16_parts(float v, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(v);
    v -= __bfloat162float(p[0]);
    p[1] = __float2bfloat16_rn(v);
    v -= __bfloat162float(p[1]);
    p[2] = __float2bfloat16_rn(v);
}

// Eight neighbouring elements of a row: 16-byte loads when the rows are whole
// vectors (vec), else one by one; zeros past the row's end.
template <typename T> struct Eight {
    static constexpr int W = sizeof(T) == 4 ? 2 : 1;
    uint4 raw[W];
    __device__ __forceinline__ void load(const T *row, int c, int cols, bool vec) {
        if (vec) {
#pragma unroll
            for (int w = 0; w < W; ++w)
                raw[w] = *reinterpret_cast<const uint4 *>(row + c + w * (16 / static_cast<int>(sizeof(T))));
        } else {
            T *e = reinterpret_cast<T *>(raw);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? row[c + i] : from_f32<T>(0.0f);
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(reinterpret_cast<const T *>(raw)[i]); }
};

// Writes eight elements of an operand, a vector of each part; `plane` elements
// from one part to the next (fp32).
template <typename T>
__device__ __forceinline__ void put_operand8(__nv_bfloat16 *out, int64_t at, int64_t plane, const float (&v)[8]) {
    constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    uint4 raw[PARTS];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (PARTS == 3) {
            __nv_bfloat16 p[3];
            bf16_parts(v[i], p);
#pragma unroll
            for (int k = 0; k < 3; ++k) reinterpret_cast<__nv_bfloat16 *>(&raw[k])[i] = p[k];
        } else {
            reinterpret_cast<__nv_bfloat16 *>(&raw[0])[i] = __float2bfloat16_rn(v[i]);
        }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) *reinterpret_cast<uint4 *>(out + at + k * plane) = raw[k];
}

// An array as an operand: rows padded with zeros to ld (a multiple of 8), fp32
// values in parts.  One thread per eight elements; I: index type that holds them all.
template <typename T, typename I>
__global__ void __launch_bounds__(256)
linear_pack_kernel(const T *__restrict__ in, int64_t rows, int cols, int ld, __nv_bfloat16 *out) {
    pdl_trigger();
    pdl_wait();
    const bool vec = cols % 8 == 0;
    const I per_row = static_cast<I>(ld / 8), total = static_cast<I>(rows) * per_row;
    for (I i = static_cast<I>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<I>(gridDim.x) * 256) {
        const I r = i / per_row;
        const int c = static_cast<int>(i - r * per_row) * 8;
        Eight<T> in8;
        in8.load(in + static_cast<int64_t>(r) * cols, c, cols, vec);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = in8[k];
        put_operand8<T>(out, static_cast<int64_t>(i) * 8, rows * ld, v);
    }
}

// ---------------------------------------------------------------- dZ and db
// dZ = dy act'(z), rounded to the storage type and laid out as an operand, and
// the column sums of the unrounded dZ over a chunk of rows.  A block takes 256
// columns, eight to a lane, its 8 warps every eighth row of the chunk, ROWS at a
// time.  dz and part nullable.  O: bf16 for an operand (fp32 in parts), T for
// the CUDA-core products.
template <typename T, typename O>
__global__ void __launch_bounds__(256, 2)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, int act, int64_t M, int n, int ld,
                 int64_t chunk_rows, O *dz, float *part) {
    constexpr int ROWS = sizeof(T) == 4 ? 2 : 4;  // rows a lane has in flight
    __shared__ float red[8][8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + lane * 8;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * chunk_rows;
    const int64_t r1 = r0 + chunk_rows < M ? r0 + chunk_rows : M;
    const bool vec = n % 8 == 0;
    float a[8] = {};
    if (c < ld) {
        for (int64_t r = r0 + warp; r < r1; r += 8 * ROWS) {
            Eight<T> v8[ROWS], z8[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const int64_t q = r + 8 * k;
                if (q < r1) {
                    v8[k].load(dy + q * n, c, n, vec);
                    if (act != kActNone) z8[k].load(z + q * n, c, n, vec);
                }
            }
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const int64_t q = r + 8 * k;
                if (q >= r1) break;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v8[k][i];
                if (act == kActGelu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = act_backward(v[i], z8[k][i], kActGelu);
                } else if (act == kActRelu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = act_backward(v[i], z8[k][i], kActRelu);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] += v[i];
                if (dz != nullptr) {
                    if (sizeof(O) == 4 || (sizeof(T) == 2 && ld % 8 != 0)) {  // plain rows for the CUDA cores
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (c + i < n) dz[q * ld + c + i] = from_f32<O>(v[i]);
                    } else {
                        put_operand8<T>(reinterpret_cast<__nv_bfloat16 *>(dz), q * ld + c, M * ld, v);
                    }
                }
            }
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][i][lane] = a[i];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;  // this thread's column to finish
    if (col < n) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][threadIdx.x & 7][threadIdx.x >> 3];
        part[static_cast<int64_t>(blockIdx.y) * n + col] = s;
    }
}

// db = the chunks' sums added: 32 columns per block, each of 32 warps every 32nd
// chunk, then a tree over the warps.
__global__ void __launch_bounds__(1024)
linear_db_kernel(const float *part, int64_t groups, int n, float *db) {
    __shared__ float red[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (col < n) {
#pragma unroll 4
        for (int64_t g = warp; g < groups; g += 32) a += part[g * n + col];
    }
    red[warp][lane] = a;
    __syncthreads();
    a = red[lane][warp];  // warp w now sums column w
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0 && blockIdx.x * 32 + warp < n) db[blockIdx.x * 32 + warp] = a;
}

// Chunks of rows of the dZ pass: about four blocks an SM, at least 32 rows each.
int64_t row_chunks(int64_t M, int n) {
    const int64_t tiles = (static_cast<int64_t>(n) + 255) / 256;
    int64_t c = 592 / tiles;
    if (c > (M + 31) / 32) c = (M + 31) / 32;
    return c < 1 ? 1 : c;
}

}  // namespace

namespace {

int pad8(int n) { return (n + 7) / 8 * 8; }

// bf16 rows of a multiple of 8 elements are operands as they are.
bool needs_pack(int dt, int cols) { return dt == 0 || cols % 8 != 0; }

size_t operand_bytes(int64_t rows, int cols, int dt) {
    return align_up(static_cast<size_t>(rows) * pad8(cols) * 2 * (dt == 0 ? 3 : 1), 256);
}

// `in` as an operand at `out` (scratch) if it is not one already.
template <typename T>
cudaError_t pack(const void *&in, int64_t rows, int cols, void *out, cudaStream_t s) {
    if (!needs_pack(sizeof(T) == 2 ? 1 : 0, cols)) return cudaSuccess;
    const int64_t n = rows * (pad8(cols) / 8), blocks = (n + 255) / 256;
    const bool small = n + 256 * 2368 < UINT32_MAX;
    cudaError_t e = launch_pdl(small ? linear_pack_kernel<T, uint32_t> : linear_pack_kernel<T, int64_t>,
                               dim3(static_cast<unsigned>(blocks < 2368 ? blocks : 2368)), dim3(256), 0, s,
                               static_cast<const T *>(in), rows, cols, pad8(cols), static_cast<__nv_bfloat16 *>(out));
    in = out;
    return e;
}

// Products too small for the tensor-core kernels' setup run on CUDA cores.
bool use_simt(int64_t M, int d_in, int d_out) { return M * d_in * static_cast<int64_t>(d_out) <= (1 << 18); }

struct FwdScratch {
    size_t x, W, total;
};
FwdScratch fwd_scratch(int64_t M, int d_in, int d_out, int dt) {
    FwdScratch L{};
    if (M == 0 || use_simt(M, d_in, d_out) || !needs_pack(dt, d_in)) return L;
    L.W = operand_bytes(M, d_in, dt);
    L.total = L.W + operand_bytes(d_out, d_in, dt);
    return L;
}

// Byte offsets inside the backward workspace: dZ, x and W as operands, and the
// row chunks' partial sums of db.
struct BwdScratch {
    size_t dz, x, W, part, total;
};
BwdScratch bwd_scratch(int64_t M, int d_in, int d_out, int dt, int act) {
    BwdScratch L{};
    size_t o = 0;
    const bool simt = use_simt(M, d_in, d_out);
    L.dz = o;
    if (simt) {
        if (act != kActNone) o += align_up(static_cast<size_t>(M) * d_out * 4, 256);
    } else if (act != kActNone || needs_pack(dt, d_out)) {
        o += operand_bytes(M, d_out, dt);
    }
    L.x = o;
    if (!simt && needs_pack(dt, d_in)) o += operand_bytes(M, d_in, dt);
    L.W = o;
    if (!simt && needs_pack(dt, d_in)) o += operand_bytes(d_out, d_in, dt);
    L.part = o;
    o += align_up(static_cast<size_t>(row_chunks(M, d_out)) * d_out * sizeof(float), 256);
    L.total = o;
    return L;
}

}  // namespace

size_t linear_ws_bytes(int64_t M, int d_in, int d_out, int dt) { return fwd_scratch(M, d_in, d_out, dt).total; }

cudaError_t launch_linear(const LinearArgs &a, void *ws, uint64_t timeout_ns, int num_sms, cudaStream_t s) {
    if (a.M == 0) return cudaSuccess;
    const LinearEpi epi{a.b, a.act, a.residual, a.y, a.z_out};
    auto go = [&](auto tag) {
        using T = decltype(tag);
        if (use_simt(a.M, a.d_in, a.d_out)) {
            SimtArgs p{a.x, a.W, a.d_in, 1, a.d_in, 1, a.M, a.d_out, a.d_in, epi};
            return launch_simt<T>(p, s);
        }
        const FwdScratch L = fwd_scratch(a.M, a.d_in, a.d_out, a.dt);
        uint8_t *w = static_cast<uint8_t *>(ws);
        const void *x = a.x, *W = a.W;
        cudaError_t e = pack<T>(x, a.M, a.d_in, w + L.x, s);
        if (e == cudaSuccess) e = pack<T>(W, a.d_out, a.d_in, w + L.W, s);
        if (e != cudaSuccess) return e;
        const TcProduct t{W, x, a.M, a.d_out, a.d_in, false, false, epi};
        return launch_tc_products(&t, 1, sizeof(T) == 4, true, timeout_ns, num_sms, s);
    };
    return a.dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

size_t linear_bwd_ws_bytes(int64_t M, int d_in, int d_out, int dt, int act) {
    return bwd_scratch(M, d_in, d_out, dt, act).total;
}

cudaError_t launch_linear_bwd(const LinearBwdArgs &a, void *ws, uint64_t timeout_ns, int num_sms, cudaStream_t s) {
    const size_t es = a.dt == 1 ? 2 : 4;
    if (a.M == 0) {
        cudaError_t e = cudaSuccess;
        if (a.dW != nullptr) e = cudaMemsetAsync(a.dW, 0, es * static_cast<size_t>(a.d_in) * a.d_out, s);
        if (e == cudaSuccess && a.db != nullptr) e = cudaMemsetAsync(a.db, 0, sizeof(float) * static_cast<size_t>(a.d_out), s);
        return e;
    }
    const BwdScratch L = bwd_scratch(a.M, a.d_in, a.d_out, a.dt, a.act);
    uint8_t *w = static_cast<uint8_t *>(ws);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        cudaError_t e = cudaSuccess;
        const bool simt = use_simt(a.M, a.d_in, a.d_out);
        const bool products = a.dx != nullptr || a.dW != nullptr;
        const bool make_dz = products && (a.act != kActNone || (!simt && needs_pack(a.dt, a.d_out)));
        float *part = a.db != nullptr ? reinterpret_cast<float *>(w + L.part) : nullptr;
        const int64_t chunks = row_chunks(a.M, a.d_out);
        const void *dz = make_dz ? static_cast<const void *>(w + L.dz) : a.dy;
        if (make_dz || part != nullptr) {
            // on CUDA cores dZ stays in the storage type; otherwise it is laid out as an operand
            const int ld = simt ? a.d_out : pad8(a.d_out);
            const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(ld) + 255) / 256), static_cast<unsigned>(chunks));
            if (simt)
                e = launch_pdl(linear_dz_kernel<T, T>, grid, dim3(256), 0, s, static_cast<const T *>(a.dy),
                               static_cast<const T *>(a.z), a.act, a.M, a.d_out, ld, (a.M + chunks - 1) / chunks,
                               make_dz ? reinterpret_cast<T *>(w + L.dz) : nullptr, part);
            else
                e = launch_pdl(linear_dz_kernel<T, __nv_bfloat16>, grid, dim3(256), 0, s, static_cast<const T *>(a.dy),
                               static_cast<const T *>(a.z), a.act, a.M, a.d_out, ld, (a.M + chunks - 1) / chunks,
                               make_dz ? reinterpret_cast<__nv_bfloat16 *>(w + L.dz) : nullptr, part);
            if (e != cudaSuccess) return e;
        }
        if (part != nullptr) {
            e = launch_pdl(linear_db_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(a.d_out) + 31) / 32)),
                           dim3(1024), 0, s, part, chunks, a.d_out, a.db);
            if (e != cudaSuccess) return e;
        }
        if (!products) return e;
        if (simt) {
            if (a.dx != nullptr) {
                SimtArgs p{dz, a.W, a.d_out, 1, 1, a.d_in, a.M, a.d_in, a.d_out, {nullptr, kActNone, nullptr, a.dx, nullptr}};
                if ((e = launch_simt<T>(p, s)) != cudaSuccess) return e;
            }
            if (a.dW != nullptr) {
                SimtArgs p{dz, a.x, 1, a.d_out, 1, a.d_in, a.d_out, a.d_in, a.M, {nullptr, kActNone, nullptr, a.dW, nullptr}};
                if ((e = launch_simt<T>(p, s)) != cudaSuccess) return e;
            }
            return e;
        }
        const void *x = a.x, *W = a.W;
        if (a.dW != nullptr) e = pack<T>(x, a.M, a.d_in, w + L.x, s);
        if (e == cudaSuccess && a.dx != nullptr) e = pack<T>(W, a.d_out, a.d_in, w + L.W, s);
        if (e != cudaSuccess) return e;
        TcProduct t[2];
        int n = 0;
        if (a.dW != nullptr)
            t[n++] = TcProduct{x, dz, a.d_out, a.d_in, static_cast<int>(a.M), true, true, {nullptr, kActNone, nullptr, a.dW, nullptr}};
        if (a.dx != nullptr)
            t[n++] = TcProduct{W, dz, a.M, a.d_in, a.d_out, true, false, {nullptr, kActNone, nullptr, a.dx, nullptr}};
        return launch_tc_products(t, n, sizeof(T) == 4, false, timeout_ns, num_sms, s);
    };
    return a.dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace moe
