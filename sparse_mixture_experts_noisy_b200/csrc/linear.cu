// The dense layer beside the experts (a shared expert's or a dense block's
// projections) and its backward pass:
//   z = x W^T + b,  y = round(act(z) + residual),  z_out = round(z)
//   dZ = dy act'(z),  dx = dZ W,  dW = dZ^T x,  db = sum over rows of dZ
// This file holds the passes around the products (operands for the tensor cores,
// dZ, db) and the host-side choice between the products' kernels.
#include "colsum.cuh"
#include "common.cuh"
#include "internal.h"
#include "linear.cuh"
#include "linear_tc.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- operands for the tensor cores
// v = p0 + p1 + p2 in bf16 parts, each the rest rounded to bf16 (the rests are
// exact in fp32).  The sum is v for |v| >= 2^-110; below, the last part ends at
// bf16's smallest step and the sum is off by 2^-134 at most.  p0 stays at bf16's
// largest, 3.39e38, for the finite values above it.  An infinite v has no parts:
// they come out as infinite and NaN, and so its products as NaN.
__device__ __forceinline__ void bf16_parts(float v, __nv_bfloat16 (&p)[3]) {
    constexpr float kMost = 3.38953139e38f;  // bf16 0x7f7f
    p[0] = __float2bfloat16_rn(fminf(fmaxf(v, -kMost), kMost));
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

// One or two arrays of the same width as operands: rows padded with zeros to ld
// (a multiple of 8), fp32 values in parts.  One thread per eight elements; I:
// index type that holds them all.
template <typename T, typename I>
__global__ void __launch_bounds__(256)
linear_pack_kernel(const T *__restrict__ in0, int64_t rows0, __nv_bfloat16 *out0, const T *__restrict__ in1,
                   int64_t rows1, __nv_bfloat16 *out1, int cols, int ld) {
    pdl_trigger();
    pdl_wait();
    const bool vec = cols % 8 == 0;
    const I per_row = static_cast<I>(ld / 8), total = static_cast<I>(rows0 + rows1) * per_row;
    for (I i = static_cast<I>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<I>(gridDim.x) * 256) {
        const I r = i / per_row;
        const int c = static_cast<int>(i - r * per_row) * 8;
        const bool second = static_cast<int64_t>(r) >= rows0;
        const int64_t row = static_cast<int64_t>(r) - (second ? rows0 : 0), rows = second ? rows1 : rows0;
        Eight<T> e;
        e.load((second ? in1 : in0) + row * cols, c, cols, vec);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = e[k];
        put_operand8<T>(second ? out1 : out0, row * ld + c, rows * ld, v);
    }
}

// ---------------------------------------------------------------- dZ and db
// dZ = dy act'(z), rounded to the storage type and laid out as an operand, and
// the column sums of the unrounded dZ over a chunk of rows.  The rounding is what
// the tensor cores take in bf16: dx and dW then have an error of 0.0024 of their
// norm, 0.0017 with dZ in fp32 (32768 x 2048 -> 1408), and the experts' backward
// rounds its dZ the same way.  In fp32 all bits of dZ go on, as three parts.
// A block takes 256 columns, eight to a lane, its 8 warps every eighth row of the
// chunk, ROWS at a time.  operand (rows of ld, fp32 in parts), plain (rows of n in
// the storage type, for the CUDA-core products) and part are nullable.
template <typename T>
__global__ void __launch_bounds__(256, 2)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, int act, int64_t M, int n, int ld,
                 int64_t chunk_rows, __nv_bfloat16 *operand, T *plain, float *part) {
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
                if (operand != nullptr) put_operand8<T>(operand, q * ld + c, M * ld, v);
                if (plain != nullptr) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i < n) plain[q * n + c + i] = from_f32<T>(v[i]);
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

// Arrays of the same width as operands in scratch, in one launch; in1 nullable.
template <typename T>
cudaError_t pack(const void *&in0, int64_t rows0, void *out0, const void *&in1, int64_t rows1, void *out1, int cols,
                 cudaStream_t s) {
    const int64_t n = (rows0 + rows1) * (pad8(cols) / 8), blocks = (n + 255) / 256;
    const bool small = n + 256 * 2368 < UINT32_MAX;
    cudaError_t e = launch_pdl(small ? linear_pack_kernel<T, uint32_t> : linear_pack_kernel<T, int64_t>,
                               dim3(static_cast<unsigned>(blocks < 2368 ? blocks : 2368)), dim3(256), 0, s,
                               static_cast<const T *>(in0), rows0, static_cast<__nv_bfloat16 *>(out0),
                               static_cast<const T *>(in1), rows1, static_cast<__nv_bfloat16 *>(out1), cols, pad8(cols));
    if (rows0 > 0) in0 = out0;
    if (rows1 > 0) in1 = out1;
    return e;
}

// A few tokens: the CUDA-core kernels, unless W is an operand as it is, which
// streams as fast through the tensor cores.  For fp32 they save a copy of W in
// parts, 2.5 times its bytes: 16 x 4096 -> 4096 40.6 us with W from HBM and 30.0
// with W in the L2 cache; 17 tokens, through the tensor cores, 43.1 and 42.9.
// Padding a bf16 W costs less: 16 x 2281 -> 8176 39 and 23 us, 4 tokens 15 and 22;
// while W is small the saved launch counts more (16 x 301 -> 705 3.8 and 7.0 us).
bool use_skinny(int64_t M, int dt, int cols, int other) {
    if (!needs_pack(dt, cols) || M > kSkinnyRows) return false;
    return dt == 0 || M <= 4 || static_cast<int64_t>(cols) * other <= (1 << 20);
}
// The forward of a small fp32 W with 16-byte rows stays ahead for longer: 48 x 300
// -> 700 7.7 us, 9.3 through the tensor cores; with rows of 301 10.7 and 9.3, bf16
// rows of 301 9.4 and 6.7, and dx in a backward of 300 x 700 24.6 and 18.2.
bool use_skinny_fwd(int64_t M, int dt, int d_in, int d_out) {
    return use_skinny(M, dt, d_in, d_out) ||
           (dt == 0 && d_in % 4 == 0 && M <= 4 * kSkinnyRows && static_cast<int64_t>(d_in) * d_out <= (1 << 18));
}
// dW has no weights to copy, and its CUDA-core kernel is bound by arithmetic past
// a few tokens: bf16 9200 x 11200 from 6 tokens 76 us, from 16 at 4096 x 14336
// 121 us, where the tensor cores take about 35: kSkinnyDwRows.

struct FwdScratch {
    size_t x, W, total;
};
FwdScratch fwd_scratch(int64_t M, int d_in, int d_out, int dt) {
    FwdScratch L{};
    if (M == 0 || !needs_pack(dt, d_in) || use_skinny_fwd(M, dt, d_in, d_out)) return L;
    L.W = operand_bytes(M, d_in, dt);
    L.total = L.W + operand_bytes(d_out, d_in, dt);
    return L;
}

// Kernels of a backward call's products, and the forms of dZ they read that have
// to be written: plain rows (CUDA cores) and an operand (tensor cores).  bf16 rows
// of a multiple of 8 elements are both.
struct BwdWays {
    bool dx_skinny, dw_skinny;
    bool plain, operand;
};
BwdWays bwd_ways(int64_t M, int d_in, int d_out, int dt, int act) {
    BwdWays w{};
    w.dw_skinny = M <= kSkinnyDwRows;
    // few columns and a long sum leave that kernel a few CTAs with many rows each
    // (backward of 9 x 272 -> 5696 fp32 45 us; 27 with dx on the tensor cores)
    const int vec = dt == 1 ? 8 : 4, tiles = (d_in - 1) / (d_in % vec == 0 ? 32 * vec : 32) + 1;
    w.dx_skinny = (use_skinny(M, dt, d_in, d_out) || use_skinny(M, dt, d_out, d_in)) && (tiles >= 16 || d_out <= 4096);
    const bool tc = !w.dw_skinny || !w.dx_skinny, same = !needs_pack(dt, d_out);
    w.operand = tc && (act != kActNone || !same);
    w.plain = (w.dw_skinny || w.dx_skinny) && act != kActNone && !(w.operand && same);
    return w;
}

// Byte offsets inside the backward workspace: dZ in both forms, x and W as
// operands, and the row chunks' partial sums of db.
struct BwdScratch {
    size_t operand, plain, x, W, part, total;
};
BwdScratch bwd_scratch(int64_t M, int d_in, int d_out, int dt, int act) {
    const BwdWays w = bwd_ways(M, d_in, d_out, dt, act);
    BwdScratch L{};
    size_t o = 0;
    L.operand = o;
    if (w.operand) o += operand_bytes(M, d_out, dt);
    L.plain = o;
    if (w.plain) o += align_up(static_cast<size_t>(M) * d_out * (dt == 1 ? 2 : 4), 256);
    L.x = o;
    if (!w.dw_skinny && needs_pack(dt, d_in)) o += operand_bytes(M, d_in, dt);
    L.W = o;
    if (!w.dx_skinny && needs_pack(dt, d_in)) o += operand_bytes(d_out, d_in, dt);
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
        if (use_skinny_fwd(a.M, a.dt, a.d_in, a.d_out))
            return launch_skinny_fwd<T>(static_cast<const T *>(a.x), static_cast<const T *>(a.W), a.M, a.d_in, a.d_out,
                                        epi, s);
        const void *x = a.x, *W = a.W;
        if (needs_pack(a.dt, a.d_in)) {
            const FwdScratch L = fwd_scratch(a.M, a.d_in, a.d_out, a.dt);
            uint8_t *w = static_cast<uint8_t *>(ws);
            cudaError_t e = pack<T>(x, a.M, w + L.x, W, a.d_out, w + L.W, a.d_in, s);
            if (e != cudaSuccess) return e;
        }
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
    const BwdWays ways = bwd_ways(a.M, a.d_in, a.d_out, a.dt, a.act);
    const BwdScratch L = bwd_scratch(a.M, a.d_in, a.d_out, a.dt, a.act);
    uint8_t *w = static_cast<uint8_t *>(ws);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        cudaError_t e = cudaSuccess;
        const bool products = a.dx != nullptr || a.dW != nullptr;
        const int ld = pad8(a.d_out);
        const int64_t chunks = row_chunks(a.M, a.d_out);
        __nv_bfloat16 *operand = products && ways.operand ? reinterpret_cast<__nv_bfloat16 *>(w + L.operand) : nullptr;
        T *plain = products && ways.plain ? reinterpret_cast<T *>(w + L.plain) : nullptr;
        float *part = a.db != nullptr ? reinterpret_cast<float *>(w + L.part) : nullptr;
        // what the products read: dy itself where no dZ of that form is written
        const void *dz_operand = operand != nullptr ? static_cast<const void *>(operand) : a.dy;
        const T *dz_plain = plain != nullptr ? plain
                            : (operand != nullptr && a.act != kActNone) ? reinterpret_cast<const T *>(operand)
                                                                        : static_cast<const T *>(a.dy);
        if (operand != nullptr || plain != nullptr || part != nullptr) {
            const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(ld) + 255) / 256), static_cast<unsigned>(chunks));
            e = launch_pdl(linear_dz_kernel<T>, grid, dim3(256), 0, s, static_cast<const T *>(a.dy),
                           static_cast<const T *>(a.z), a.act, a.M, a.d_out, ld, (a.M + chunks - 1) / chunks, operand,
                           plain, chunks == 1 ? a.db : part);
            if (e != cudaSuccess) return e;
        }
        if (part != nullptr && chunks > 1) {
            e = launch_col_reduce(part, chunks, a.d_out, 1, a.db, nullptr, s);
            if (e != cudaSuccess) return e;
        }
        if (!products) return e;
        const bool tc_dw = a.dW != nullptr && !ways.dw_skinny, tc_dx = a.dx != nullptr && !ways.dx_skinny;
        const void *x = a.x, *W = a.W;
        if (needs_pack(a.dt, a.d_in) && (tc_dw || tc_dx)) {
            e = pack<T>(x, tc_dw ? a.M : 0, w + L.x, W, tc_dx ? a.d_out : 0, w + L.W, a.d_in, s);
            if (e != cudaSuccess) return e;
        }
        TcProduct t[2];
        int n = 0;
        if (!ways.dw_skinny)
            t[n++] = TcProduct{x, dz_operand, a.d_out, a.d_in, static_cast<int>(a.M), true, true, {nullptr, kActNone, nullptr, a.dW, nullptr}};
        if (!ways.dx_skinny)
            t[n++] = TcProduct{W, dz_operand, a.M, a.d_in, a.d_out, true, false, {nullptr, kActNone, nullptr, a.dx, nullptr}};
        if (n > 0) {
            e = launch_tc_products(t, n, sizeof(T) == 4, false, timeout_ns, num_sms, s);
            if (e != cudaSuccess) return e;
        }
        if (a.dx != nullptr && ways.dx_skinny) {
            e = launch_skinny_dx<T>(dz_plain, static_cast<const T *>(a.W), a.M, a.d_in, a.d_out,
                                    static_cast<T *>(a.dx), s);
            if (e != cudaSuccess) return e;
        }
        if (a.dW != nullptr && ways.dw_skinny)
            e = launch_skinny_dw<T>(dz_plain, static_cast<const T *>(a.x), a.M, a.d_in, a.d_out,
                                    static_cast<T *>(a.dW), s);
        return e;
    };
    return a.dt == 1 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace moe
