// The dense layer's products for a few tokens, on CUDA cores: each weight is read
// once (or written once, for dW) with 16-byte accesses and meets up to 16 tokens
// in registers, and no copy of W in another form is needed.  The forward takes more
// tokens of a small W in further blocks, 16 each.  fp32 accumulation in fp32
// storage too.
//   forward  z[m][n]  = sum_k x[m][k] W[n][k]       rows of W, K split over a block's warps
//   dx       dx[m][i] = sum_o dZ[m][o] W[o][i]      columns of W, o split over warps and a cluster
//   dW       dW[o][i] = sum_m dZ[m][o] x[m][i]      one pass over dW
// One token of 4096 x 4096 fp32 streams W from HBM in 12.0 us, 5.6 TB/s (6.4 us
// where W is in the L2 cache).  With more tokens the forward is bound by its loads
// of x: a warp reads all its tokens' vectors for 4 rows of W, so 16 tokens bring 4
// bytes of x through the L1 cache for each byte of W, and about 250 registers a
// thread leave an SM one block to hide them.  4 tokens take 17.5 us, 8 take 28.4
// and 16 take 40.6 (10.4, 18.0 and 30.0 from L2).
// The multiply-adds take less in fp32 (128 weights in a warp's 512 bytes of W, 4 M
// instructions, 16 cycles of an SM at M = 16; the bytes take 22 from HBM), more in
// bf16 (256 weights, 32 cycles).
// VEC: elements of a 16-byte vector, or 1 where rows do not start on 16 bytes.
#include "common.cuh"
#include "internal.h"
#include "linear.cuh"
#include "linear_tc.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = 8;

// VEC elements as they lie in memory.
template <typename T, int VEC> struct Raw {
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(reinterpret_cast<const T *>(&u)[i]); }
};
template <typename T> struct Raw<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ float operator[](int) const { return to_f32<T>(u); }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        uint4 raw;
        T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(v[i]);
        *reinterpret_cast<uint4 *>(p) = raw;
    }
}

// ---------------------------------------------------------------- forward
// Sums V values of each lane over the warp (V a multiple of 32, or at most 32 and
// a power of two): each step halves the values a lane still carries.  After it
// lane l holds the totals of values l V / 32 + i in v[i] (V >= 32), or of value
// l / (32 / V) in v[0].
template <int V>
__device__ __forceinline__ void fold(float *v, int lane) {
    int n = V;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n /= 2;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
}

// A warp group of KW warps takes R rows of W; its warp w the vectors w, w + KW,
// ... of K.
template <typename T, int VEC, int MT, int R, int KW>
__global__ void __launch_bounds__(kThreads)
skinny_fwd_kernel(const T *__restrict__ x, const T *__restrict__ W, int M, int K, int Nn, const LinearEpi epi) {
    const int m0 = blockIdx.y * MT;  // this block's tokens
    x += static_cast<int64_t>(m0) * K;
    M -= m0;
    constexpr int V = R * MT, GROUPS = kWarps / KW;
    static_assert(V % 32 == 0 || (V < 32 && (V & (V - 1)) == 0), "fold");
    __shared__ float red[kWarps][V];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = warp / KW;
    const int n0 = (blockIdx.x * GROUPS + grp) * R;
    float acc[V] = {};  // [r][m]
    if (n0 < Nn) {
        // rows past W's or x's last read a valid one; their sums are dropped
        const T *wr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) wr[r] = W + static_cast<int64_t>(n0 + r < Nn ? n0 + r : n0) * K;
#pragma unroll 2
        for (int k = (warp % KW * 32 + lane) * VEC; k < K; k += KW * 32 * VEC) {
            Raw<T, VEC> w[R];
#pragma unroll
            for (int r = 0; r < R; ++r) w[r].load(wr[r] + k);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                Raw<T, VEC> a;
                a.load(x + static_cast<int64_t>(m < M ? m : 0) * K + k);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[r * MT + m] = fmaf(a[i], w[r][i], acc[r * MT + m]);
            }
        }
    }
    fold<V>(acc, lane);
    if constexpr (V >= 32) {
#pragma unroll
        for (int i = 0; i < V / 32; ++i) red[warp][lane * (V / 32) + i] = acc[i];
    } else {
        if (lane % (32 / V) == 0) red[warp][lane / (32 / V)] = acc[0];
    }
    __syncthreads();
    for (int q = threadIdx.x; q < GROUPS * V; q += kThreads) {
        const int g = q / V, v = q % V, m = v % MT, n = (blockIdx.x * GROUPS + g) * R + v / MT;
        if (m < M && n < Nn) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) sum += red[g * KW + w][v];
            linear_store<T>(epi, m0 + m, n, Nn, sum);
        }
    }
}

// ---------------------------------------------------------------- dx
// A cluster of S blocks takes 32 VEC columns; block r the rows o = r, r + S, ...
// in chunks that its 8 warps share.
template <typename T, int VEC, int MT>
__global__ void __launch_bounds__(kThreads)
skinny_dx_kernel(const T *__restrict__ dz, const T *__restrict__ W, int M, int Ni, int No, int S, T *dx) {
    constexpr int COLS = 32 * VEC, CHUNK = 128, FLY = 8;  // rows of W a chunk; a lane's loads in flight
    extern __shared__ float smem[];                       // [kWarps][MT][COLS]
    __shared__ __align__(16) float g[CHUNK][MT];          // dZ of the chunk
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int i0 = blockIdx.x / S * COLS, col = i0 + lane * VEC;
    const bool live = col < Ni;
    float acc[MT][VEC] = {};
    for (int base = rank * CHUNK; base < No; base += S * CHUNK) {
        // the chunk's first rows are on their way while its dZ is staged
        Raw<T, VEC> w[FLY];
        auto fetch = [&](int first) {
#pragma unroll
            for (int u = 0; u < FLY; ++u) {
                const int o = base + warp + 8 * (first + u);
                if (live) w[u].load(W + static_cast<int64_t>(o < No ? o : base) * Ni + col);
            }
        };
        fetch(0);
        __syncthreads();
        for (int q = threadIdx.x; q < CHUNK * MT; q += kThreads) {
            const int m = q / CHUNK, o = q % CHUNK;
            g[o][m] = (m < M && base + o < No) ? to_f32<T>(dz[static_cast<int64_t>(m) * No + base + o]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int f = 0; f < CHUNK / kWarps; f += FLY) {
            if (f > 0) fetch(f);
            if (live) {
#pragma unroll
                for (int u = 0; u < FLY; ++u) {
                    const int o = warp + 8 * (f + u);
                    if (base + o < No) {  // a row past the last would bring its own NaN
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) acc[m][i] = fmaf(g[o][m], w[u][i], acc[m][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < VEC; ++i) smem[(warp * MT + m) * COLS + i * 32 + lane] = acc[m][i];
    __syncthreads();
    // the block's sums in smem[0 .. MT COLS), then the cluster's parts in rank order
    for (int q = threadIdx.x; q < MT * COLS; q += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += smem[w * MT * COLS + q];
        smem[q] = v;
    }
    __syncthreads();
    if (S > 1) cluster_sync();
    for (int q = rank * kThreads + threadIdx.x; q < M * COLS; q += S * kThreads) {
        float v = 0.0f;
        if (S > 1) {
            float u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                u[c] = 0.0f;
                if (c < S)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(u[c])
                                 : "r"(map_to_cta(smem_u32(smem + q), c))
                                 : "memory");
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) v += u[c];
        } else {
            v = smem[q];
        }
        const int m = q / COLS, i = i0 + (q % 32) * VEC + (q % COLS) / 32;
        if (i < Ni) dx[static_cast<int64_t>(m) * Ni + i] = from_f32<T>(v);
    }
    if (S > 1) cluster_sync();  // no block leaves while another reads its sums
}

// ---------------------------------------------------------------- dW
// A block takes 32 VEC columns and 64 rows of dW: x of the columns in registers,
// dZ of the rows in shared memory, each warp every eighth row.
template <typename T, int VEC, int MT>
__global__ void __launch_bounds__(kThreads)
skinny_dw_kernel(const T *__restrict__ dz, const T *__restrict__ x, int M, int Ni, int No, T *dW) {
    constexpr int ROWS = 64;
    __shared__ __align__(16) float g[ROWS][MT];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = (blockIdx.x * 32 + lane) * VEC;
    float a[MT][VEC];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[m][i] = 0.0f;
        if (m < M && col < Ni) {
            Raw<T, VEC> raw;
            raw.load(x + static_cast<int64_t>(m) * Ni + col);
#pragma unroll
            for (int i = 0; i < VEC; ++i) a[m][i] = raw[i];
        }
    }
    for (int64_t o0 = static_cast<int64_t>(blockIdx.y) * ROWS; o0 < No; o0 += static_cast<int64_t>(gridDim.y) * ROWS) {
        __syncthreads();
        for (int q = threadIdx.x; q < ROWS * MT; q += kThreads) {
            const int m = q / ROWS, o = q % ROWS;
            g[o][m] = (m < M && o0 + o < No) ? to_f32<T>(dz[static_cast<int64_t>(m) * No + o0 + o]) : 0.0f;
        }
        __syncthreads();
        if (col < Ni) {
#pragma unroll 2
            for (int o = warp; o < ROWS; o += kWarps) {
                if (o0 + o >= No) break;
                float v[VEC] = {};
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = fmaf(g[o][m], a[m][i], v[i]);
                store_vec<T, VEC>(dW + (o0 + o) * Ni + col, v);
            }
        }
    }
}

template <int V> struct Int {
    static constexpr int value = V;
};

// f(tag of VEC, tag of MT) for rows of `cols` elements.
template <typename T, int MOST, typename F> cudaError_t skinny_pick(int cols, int64_t M, F f) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    auto with = [&](auto vec) {
        if (M <= 1) return f(vec, Int<1>{});
        if constexpr (MOST > 4) {
            if (M > 8) return f(vec, Int<MOST>{});
            if (M > 4) return f(vec, Int<8>{});
        }
        return f(vec, Int<4>{});
    };
    return cols % VEC == 0 ? with(Int<VEC>{}) : with(Int<1>{});
}

}  // namespace

template <typename T>
cudaError_t launch_skinny_fwd(const T *x, const T *W, int64_t M, int K, int Nn, const LinearEpi &epi, cudaStream_t s) {
    return skinny_pick<T, kSkinnyRows>(K, M, [&](auto vec, auto mt) {
        // rows a warp group: enough to share x, few enough that the SMs have blocks.  A
        // group is a warp where a row gives it work for four vectors a lane.
        constexpr int V = decltype(vec)::value, MT = decltype(mt)::value;
        auto go = [&](auto r, auto kw) {
            constexpr int R = decltype(r)::value, KW = decltype(kw)::value, rows = R * (kWarps / KW);
            const dim3 grid(static_cast<unsigned>((Nn + rows - 1) / rows), static_cast<unsigned>((M + MT - 1) / MT));
            return launch_pdl(skinny_fwd_kernel<T, V, MT, R, KW>, grid, dim3(kThreads), 0, s, x, W,
                              static_cast<int>(M), K, Nn, epi);
        };
        constexpr int R = MT > 1 ? 4 : 2;
        return K >= 8 * 32 * V || Nn < 148 * kWarps ? go(Int<R>{}, Int<kWarps>{}) : go(Int<R>{}, Int<1>{});
    });
}

template <typename T>
cudaError_t launch_skinny_dx(const T *dz, const T *W, int64_t M, int Ni, int No, T *dx, cudaStream_t s) {
    return skinny_pick<T, kSkinnyRows>(Ni, M, [&](auto vec, auto mt) {
        constexpr int V = decltype(vec)::value, MT = decltype(mt)::value;
        constexpr int smem = kWarps * MT * 32 * V * static_cast<int>(sizeof(float));
        auto kern = skinny_dx_kernel<T, V, MT>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int tiles = (Ni + 32 * V - 1) / (32 * V);
        int S = (No + 127) / 128;  // a chunk of rows each at least
        if (S > 8) S = 8;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = S;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = S > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, kern, dz, W, static_cast<int>(M), Ni, No, S, dx);
    });
}

template <typename T>
cudaError_t launch_skinny_dw(const T *dz, const T *x, int64_t M, int Ni, int No, T *dW, cudaStream_t s) {
    return skinny_pick<T, kSkinnyDwRows>(Ni, M, [&](auto vec, auto mt) {
        constexpr int V = decltype(vec)::value, MT = decltype(mt)::value;
        const int64_t gy = (static_cast<int64_t>(No) + 63) / 64;
        return launch_pdl(skinny_dw_kernel<T, V, MT>,
                          dim3(static_cast<unsigned>((Ni + 32 * V - 1) / (32 * V)), static_cast<unsigned>(gy < 65535 ? gy : 65535)),
                          dim3(kThreads), 0, s, dz, x, static_cast<int>(M), Ni, No, dW);
    });
}

template cudaError_t launch_skinny_fwd<float>(const float *, const float *, int64_t, int, int, const LinearEpi &, cudaStream_t);
template cudaError_t launch_skinny_fwd<__nv_bfloat16>(const __nv_bfloat16 *, const __nv_bfloat16 *, int64_t, int, int,
                                                      const LinearEpi &, cudaStream_t);
template cudaError_t launch_skinny_dx<float>(const float *, const float *, int64_t, int, int, float *, cudaStream_t);
template cudaError_t launch_skinny_dx<__nv_bfloat16>(const __nv_bfloat16 *, const __nv_bfloat16 *, int64_t, int, int,
                                                     __nv_bfloat16 *, cudaStream_t);
template cudaError_t launch_skinny_dw<float>(const float *, const float *, int64_t, int, int, float *, cudaStream_t);
template cudaError_t launch_skinny_dw<__nv_bfloat16>(const __nv_bfloat16 *, const __nv_bfloat16 *, int64_t, int, int,
                                                     __nv_bfloat16 *, cudaStream_t);

}  // namespace moe
