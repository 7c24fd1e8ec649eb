// The dense layer's products on the fifth-generation tensor cores.
//
//   D[m][n] = sum_k Q(m, k) P(n, k)
// with n the contiguous index of the output row.  P is the MMA's A operand and Q
// its B operand, so a lane of tensor memory holds one n and a column one m: a
// warp stores 32 neighbouring elements of an output row whatever its width and
// alignment, and the bias is one value per lane.
//   forward   D = y  [M][d_out]     P = W  [d_out][d_in]          Q = x  [M][d_in]       k = d_in
//   dx        D = dx [M][d_in]      P = W  [k = d_out][d_in] (MN) Q = dZ [M][d_out]      k = d_out
//   dW        D = dW [d_out][d_in]  P = x  [k = M][d_in]     (MN) Q = dZ [k = M][d_out] (MN)
// "(MN)": the operand is stored with k as its rows; the MMA reads such a tile
// MN-major, so nothing is transposed in memory.  TMA fills what lies outside an
// array with zeros, so no size has to be a multiple of a tile.
//
// fp32 storage runs on the bf16 tensor cores: each value is split into three
// bf16 parts, v = v0 + v1 + v2 (8 significant bits each), stored as three
// planes, and the six products of parts p, q with p + q <= 2 are summed; the
// three that are left out are below 2^-24 of the product.  Each product of two
// parts is exact in fp32.  A K block's three planes of both operands are loaded
// together and serve all six products.  The tensor core truncates when it adds
// to its accumulator, an error that grows with the number of additions, so K is
// cut into pieces of kPieceKb blocks: each starts from zero and is added to the
// others in registers.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "linear.cuh"
#include "linear_tc.h"
#include "tmap.h"

namespace moe {

// The dense layer's status word on each device (bounded waits of its kernels).
static __device__ uint32_t g_linear_status;

cudaError_t linear_status_address(uint32_t **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_linear_status);
}

cudaError_t linear_status_read_clear(uint32_t *word, cudaStream_t s) {
    uint32_t *at = nullptr;
    cudaError_t e = linear_status_address(&at);
    return e != cudaSuccess ? e : status_read_clear(at, word, s);
}

namespace {

constexpr int kBK = 64;        // K elements per stage: 128 bytes, one swizzle row
// K blocks per piece of an fp32 product.  2-norm of the error over the result's at
// 4000 x 4096 x 4096, and the time of 4096^3: 1 block 1.7e-7 and 729 us (the
// epilogue warps cannot keep up), 2 blocks 6.0e-7 and 580, 4 blocks 1.5e-6 and 575;
// an fp32 product on CUDA cores has 1.1e-6.
constexpr int kPieceKb = 2;
constexpr int kTerms = 6;      // products of parts

// Plane of P and of Q for term t: (0,2) (2,0) (1,1) (0,1) (1,0) (0,0).
__device__ __forceinline__ int term_p(int t) { return t == 1 ? 2 : (t == 2 || t == 4) ? 1 : 0; }
__device__ __forceinline__ int term_q(int t) { return t == 0 ? 2 : (t == 2 || t == 3) ? 1 : 0; }

struct ProdArgs {
    int64_t M;       // rows of D
    int Nn, kb;      // columns of D, K blocks
    int p_mn, q_mn;  // operand stored with k as its rows
    int tm;          // pairs: rows of D in a tile
    LinearEpi epi;
};

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > timeout_ns) return false;
    return true;
}

// One lane of a converged warp.  The TMA and MMA warps run their loops whole and
// let this lane issue: the loop's state then stays in uniform registers.  With
// the loop inside `if (lane == 0)`, and operand layouts tested per K block, a
// stage cost the issuing thread about 400 ns, more than its MMAs.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p;
}

// The issuing instructions, executed by the lanes with `one` set.  As predicated
// instructions in converged code, not under a branch: addresses and descriptors
// are then computed in uniform registers.
__device__ __forceinline__ void expect_tx_if(uint32_t one, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_if(uint32_t one, uint32_t dst, const void *tmap, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_pair_if(uint32_t one, uint32_t dst, const void *tmap, uint32_t bar, int x, int y,
                                             int z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(one)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_if(uint32_t one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
            : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}
__device__ __forceinline__ void commit_both_if(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(bar), "h"(static_cast<uint16_t>(3)), "r"(one)
        : "memory");
}

// mbar_wait_bounded by a whole converged warp, every lane polling.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t *status, uint64_t timeout_ns,
                                          uint32_t where) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, status, timeout_ns, where));
}

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};
// f(operand P is MN-major, operand Q is MN-major) with the layouts as constants.
template <typename F> __device__ __forceinline__ void by_layout(const bool p_mn, const bool q_mn, F f) {
    if (!p_mn) f(No{}, No{});
    else if (!q_mn) f(Yes{}, No{});
    else f(Yes{}, Yes{});
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Stores up to CN accumulated columns (rows m0.. of D, `cols` of them valid) of
// this lane's n.  FULL: bias, activation, residual and z as the epilogue says;
// otherwise the value alone.  Every choice is made once for the CN columns: a
// branch per element made a 256 x 256 tile's epilogue take 20 us.
// Measured and not kept, at 64 x 4096 -> 14336 (dW, 40 us) and 4096 x 256 -> 4096
// (24 us): two elements a lane by a swap between neighbouring lanes, 44 and 27 us;
// the next columns read from tensor memory while these are stored, with the loop
// unrolled for it, 40 and 29 us (more instructions to fetch).
template <typename T, int CN>
__device__ __forceinline__ void put_cols(T *p, const float (&v)[CN], int ld, int cols) {
    if (cols >= CN) {
#pragma unroll
        for (int i = 0; i < CN; ++i) p[static_cast<int64_t>(i) * ld] = from_f32<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < CN; ++i)
            if (i < cols) p[static_cast<int64_t>(i) * ld] = from_f32<T>(v[i]);
    }
}

// The residual's values at CN columns (a valid one in place of those past `cols`).
template <typename T, int CN>
__device__ __forceinline__ void get_residual(T (&res)[CN], const LinearEpi &e, int64_t m0, int n, int ld, int cols) {
    const T *p = static_cast<const T *>(e.residual) + m0 * ld + n;
#pragma unroll
    for (int i = 0; i < CN; ++i) res[i] = p[static_cast<int64_t>(i < cols ? i : 0) * ld];
}

template <typename T, bool FULL, int CN>
__device__ __forceinline__ void finish_cols(const LinearEpi &e, const float *acc, const T (&res)[CN], int64_t m0, int n,
                                            int ld, int cols, float bias) {
    const int64_t at = m0 * ld + n;
    float v[CN];
#pragma unroll
    for (int i = 0; i < CN; ++i) v[i] = acc[i];
    if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < CN; ++i) v[i] += bias;
        if (e.z_out != nullptr) put_cols<T, CN>(static_cast<T *>(e.z_out) + at, v, ld, cols);
        if (e.act == kActGelu) {
#pragma unroll
            for (int i = 0; i < CN; ++i) v[i] = act_value(v[i], kActGelu);
        } else if (e.act == kActRelu) {
#pragma unroll
            for (int i = 0; i < CN; ++i) v[i] = act_value(v[i], kActRelu);
        }
        if (e.residual != nullptr) {
#pragma unroll
            for (int i = 0; i < CN; ++i) v[i] += to_f32<T>(res[i]);
        }
    }
    put_cols<T, CN>(static_cast<T *>(e.out) + at, v, ld, cols);
}

template <typename T, bool FULL, int CN>
__device__ __forceinline__ void store_cols(const LinearEpi &e, const float *acc, int64_t m0, int n, int ld, int cols,
                                           float bias) {
    T res[CN];
    if (FULL && e.residual != nullptr) get_residual<T, CN>(res, e, m0, n, ld, cols);
    finish_cols<T, FULL, CN>(e, acc, res, m0, n, ld, cols, bias);
}

// ---------------------------------------------------------------- CTA pairs
// A pair of CTAs (tcgen05 cta_group::2) computes tiles of 256 n x tm m of D, tm
// 128, 192 or 256: CTA r loads P rows [n0 + 128 r, +128) and Q rows
// [m0 + r tm / 2, + tm / 2) per K block, the leader's MMA reads both, and each
// CTA's tensor memory gets its 128 n of all tm m.  fp32 tiles have 192 m at most,
// of which an epilogue thread adds 96 columns in registers.
// Persistent, one pair per two SMs; two accumulators, so the epilogue of
// one tile (or piece) overlaps the MMAs of the next.  Warp 0: TMA; warp 1: MMA;
// the others: epilogue, in groups of four, each a share of the m.
//
// One launch runs one product or two (dW, then dx).  A unit is a tile of a
// product; the first product's units are dealt in turn, and the second's start
// with the pairs that got one fewer of the first's, as many as fit into the time
// the others still need, before they are dealt to all.
// Epilogue warps come in groups of four, which read all 128 lanes of tensor
// memory; two groups share a tile's rows.  bf16 tiles have two such sets, one for
// each accumulator: a set spends most of a short tile's epilogue on its own chain
// of waits, reads and stores, and the other works meanwhile.  An fp32 thread's
// sums need the registers of one set.
constexpr int pair_groups(bool fp32) { return fp32 ? 2 : 4; }
constexpr int pair_threads(bool fp32) { return 64 + 128 * pair_groups(fp32); }
constexpr int kPairMaxStages = 6;
constexpr int kPairRing = 216 * 1024;
constexpr int pair_max_tm(bool fp32) { return fp32 ? 192 : 256; }
// Bytes of a CTA's Q rows in a plane of a stage: 64-wide boxes when MN-major.
__host__ __device__ constexpr int pair_q_bytes(int tm, bool mn) {
    return (mn ? (tm / 2 + 63) / 64 * 64 : tm / 2) * kBK * 2;
}
constexpr int kGroupM = 8;  // m tiles that share a sweep over n: their Q rows stay in L2

struct PairArgs {
    ProdArgs p[2];
    int units[2];
    int late, early;  // second product: pairs [0, late) start late; the others do `early` units first
    int stages, q_room;  // ring slots; bytes a slot keeps for a plane of Q
    uint64_t timeout_ns;
};

struct PairUnit {
    int prob, n0;
    int64_t m0;
};

__device__ __forceinline__ bool pair_unit(const PairArgs &a, int pair, int npairs, int n1, int i, PairUnit &t) {
    int u;
    if (i < n1) {
        t.prob = 0;
        u = pair + i * npairs;
    } else {
        t.prob = 1;
        i -= n1;
        const int head = a.early * (npairs - a.late);
        if (pair >= a.late && i < a.early) {
            u = (pair - a.late) + i * (npairs - a.late);
        } else {
            u = head + pair + (pair >= a.late ? i - a.early : i) * npairs;
        }
        if (u >= a.units[1]) return false;
    }
    const ProdArgs &p = a.p[t.prob];
    const int mt = static_cast<int>((p.M + p.tm - 1) / p.tm), nt = (p.Nn + 255) / 256;
    const int sweep = kGroupM * nt;
    const int grp = u / sweep, rem = u - grp * sweep;
    const int rows = mt - grp * kGroupM;  // m tiles of the last group
    const int row = rows < kGroupM ? rem % rows : rem % kGroupM, col = rows < kGroupM ? rem / rows : rem / kGroupM;
    t.m0 = static_cast<int64_t>(grp * kGroupM + row) * p.tm;
    t.n0 = col * 256;
    return true;
}

template <typename T, bool FULL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair_threads(sizeof(T) == 4), 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tp0, const __grid_constant__ CUtensorMap tq0,
                   const __grid_constant__ CUtensorMap tp1, const __grid_constant__ CUtensorMap tq1,
                   const __grid_constant__ PairArgs args) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PLANES = SPLIT ? 3 : 1, TERMS = SPLIT ? kTerms : 1;
    constexpr int SETS = pair_groups(SPLIT) / 2, HMAX = pair_max_tm(SPLIT) / 2;
    constexpr uint32_t P_BYTES = 128 * kBK * 2, Q_AT = PLANES * P_BYTES;
    const int stages = args.stages;
    const uint32_t q_room = args.q_room, stage_bytes = PLANES * (P_BYTES + q_room);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t bars[2 * kPairMaxStages + 5];
    __shared__ uint32_t tmem_holder;
    __shared__ uint32_t cta_status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int n1 = pair < args.units[0] ? (args.units[0] - pair + npairs - 1) / npairs : 0;  // units of the first product
    uint32_t *status = &cta_status;
    const uint64_t tmo = args.timeout_ns;
    const uint32_t smem_base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
    const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[kPairMaxStages]);
    const uint32_t tfull0 = smem_u32(&bars[2 * kPairMaxStages]), tempty0 = smem_u32(&bars[2 * kPairMaxStages + 2]);
    const uint32_t drain = smem_u32(&bars[2 * kPairMaxStages + 4]);
    const uint32_t full0_lead = map_to_cta(full0, 0), tempty0_lead = map_to_cta(tempty0, 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(tfull0, 1);
        mbar_init(tfull0 + 8, 1);
        mbar_init(tempty0, 16);  // a set's 8 epilogue warps in each CTA
        mbar_init(tempty0 + 8, 16);
        mbar_init(drain, 1);
        fence_barrier_init();
        cta_status = 0u;
        tma_prefetch_desc(&tp0);
        tma_prefetch_desc(&tq0);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&tmem_holder), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    pdl_trigger();  // behind the allocation: see common.cuh
    const uint32_t tmem_base = tmem_holder;
    pdl_wait();

    if (warp == 0) {
        const uint32_t one = elect_one();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        PairUnit t;
        for (int i = 0; ok && pair_unit(args, pair, npairs, n1, i, t); ++i) {
            const CUtensorMap *tp = t.prob ? &tp1 : &tp0, *tq = t.prob ? &tq1 : &tq0;
            const int nr = t.n0 + static_cast<int>(rank) * 128;
            const int qr = args.p[t.prob].tm / 2, mr = static_cast<int>(t.m0) + static_cast<int>(rank) * qr;
            const int kbs = args.p[t.prob].kb;
            by_layout(args.p[t.prob].p_mn != 0, args.p[t.prob].q_mn != 0, [&](auto pm, auto qm) {
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!wait_warp(empty0 + 8 * stage, phase ^ 1u, status, tmo, 61)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0_lead + 8 * stage;
                    const uint32_t sa = smem_base + stage * stage_bytes;
                    const int kx = kb * kBK;
                    expect_tx_if(leader ? one : 0u, full0 + 8 * stage,
                                 2 * PLANES * (P_BYTES + pair_q_bytes(2 * qr, decltype(qm)::value)));
                    {
#pragma unroll
                        for (int z = 0; z < PLANES; ++z) {
                            const uint32_t a = sa + z * P_BYTES, b = sa + Q_AT + z * q_room;
                            if constexpr (decltype(pm)::value) {
                                load_pair_if(one, a, tp, fb, nr, kx, z);
                                load_pair_if(one, a + 8192u, tp, fb, nr + 64, kx, z);
                            } else {
                                load_pair_if(one, a, tp, fb, kx, nr, z);
                            }
                            if constexpr (decltype(qm)::value) {
                                load_pair_if(one, b, tq, fb, mr, kx, z);
                                if (qr > 64) load_pair_if(one, b + 8192u, tq, fb, mr + 64, kx, z);
                            } else {
                                load_pair_if(one, b, tq, fb, kx, mr, z);
                            }
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            });
        }
        if (!ok && leader && one) {
            // the pair's copies of the stages armed here land before exit
            int st = stage;
            uint32_t ph = phase;
            for (int i = 0; i < stages && i < issued; ++i) {
                if (st == 0) {
                    st = stages - 1;
                    ph ^= 1u;
                } else {
                    --st;
                }
                wait_drain(full0 + 8 * st, ph, tmo);
            }
        }
    } else if (warp == 1) {
        if (leader) {
            const uint32_t one = elect_one();
            int stage = 0, local = 0;
            uint32_t phase = 0;
            bool ok = true, any = false;
            PairUnit t;
            for (int i = 0; ok && pair_unit(args, pair, npairs, n1, i, t); ++i) {
                const int kbs = args.p[t.prob].kb;
                by_layout(args.p[t.prob].p_mn != 0, args.p[t.prob].q_mn != 0, [&](auto pm, auto qm) {
                    constexpr bool PM = decltype(pm)::value, QM = decltype(qm)::value;
                    const uint32_t idesc = idesc_bf16_f32(256, args.p[t.prob].tm) | (PM ? kIdescAMajorMN : 0u) |
                                           (QM ? kIdescBMajorMN : 0u);
                    // K-major: the next 16 of K are 32 bytes on in the swizzled row;
                    // MN-major: 16 rows of 128 bytes on
                    constexpr uint32_t astep = PM ? 128u : 2u, bstep = QM ? 128u : 2u;
                    const int piece = SPLIT ? kPieceKb : kbs;
                    for (int k0 = 0; k0 < kbs && ok; k0 += piece) {
                        const int n = k0 + piece < kbs ? piece : kbs - k0;
                        const int acc = local & 1;
                        if (!wait_warp(tempty0 + 8 * acc, ((local >> 1) & 1) ^ 1u, status, tmo, 62)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
                        for (int k = 0; k < n; ++k) {
                            if (!wait_warp(full0 + 8 * stage, phase, status, tmo, 63)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            {
                                const uint32_t sa = smem_base + stage * stage_bytes;
                                const uint64_t ad = PM ? smem_desc_mn_sw128(sa, 8192u, 1024u) : smem_desc_sw128(sa);
                                const uint64_t bd = QM ? smem_desc_mn_sw128(sa + Q_AT, 8192u, 1024u)
                                                       : smem_desc_sw128(sa + Q_AT);
#pragma unroll
                                for (int x = 0; x < TERMS; ++x) {
                                    const uint64_t ax = ad + (SPLIT ? term_p(x) * (P_BYTES >> 4) : 0);
                                    const uint64_t bx = bd + (SPLIT ? term_q(x) * (q_room >> 4) : 0);
#pragma unroll
                                    for (int kk = 0; kk < kBK / 16; ++kk)
                                        mma_if<true>(one, d_tmem, ax + astep * kk, bx + bstep * kk, idesc,
                                                       (k > 0 || x > 0 || kk > 0) ? 1u : 0u);
                                }
                                commit_both_if(one, empty0 + 8 * stage);
                            }
                            __syncwarp();
                            any = true;
                            if (++stage == stages) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                        if (!ok) break;
                        commit_both_if(one, tfull0 + 8 * acc);
                        __syncwarp();
                        ++local;
                    }
                });
            }
            if (!ok && any && one) {
                umma_commit_pair(drain);
                wait_drain(drain, 0, tmo);
            }
        }
    } else {
        const int q = warp & 3, half = ((warp - 2) >> 2) & 1, set = (warp - 2) >> 3;
        int local = set;  // pieces before this one, over all sets: the accumulators' turn
        bool ok = true;
        PairUnit t;
        for (int i = set; ok && pair_unit(args, pair, npairs, n1, i, t); i += SETS) {
            const ProdArgs &p = args.p[t.prob];
            const int n = t.n0 + static_cast<int>(rank) * 128 + q * 32 + lane;
            const int hm = p.tm / 2;  // m of this group
            const int64_t m0 = t.m0 + half * hm;
            const int64_t left = p.M - m0;
            const int rows = left < hm ? static_cast<int>(left > 0 ? left : 0) : hm;
            const float bias = (FULL && p.epi.bias != nullptr && n < p.Nn) ? p.epi.bias[n] : 0.0f;
            // bf16 with a residual: its values are read 16 columns ahead of their use,
            // the first before the tile is done (read in place, a 32-column step took
            // HBM's latency each time)
            const bool add = FULL && !SPLIT && p.epi.residual != nullptr && n < p.Nn && rows > 0;
            T res[16];
            if (add) get_residual<T, 16>(res, p.epi, m0, n, p.Nn, rows);
            float sum[SPLIT ? HMAX : 1];
            const int pieces = SPLIT ? (p.kb + kPieceKb - 1) / kPieceKb : 1;
            for (int pc = 0; pc < pieces; ++pc) {
                const int acc = local & 1;
                if (!mbar_wait_warp(tfull0 + 8 * acc, (local >> 1) & 1, status, tmo, 64)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                       static_cast<uint32_t>(acc * 256 + half * hm);
                if constexpr (SPLIT) {
#pragma unroll
                    for (int c = 0; c < HMAX / 16; ++c) {
                        if (c * 16 >= hm) break;
                        uint32_t r[16];
                        tmem_ld_32x32b_x16(taddr + c * 16, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[c * 16 + j] = pc == 0 ? __uint_as_float(r[j]) : sum[c * 16 + j] + __uint_as_float(r[j]);
                    }
                } else {
                    if constexpr (FULL) {
                        for (int c = 0; c * 16 < rows; ++c) {
                            T next[16];
                            if (add && c * 16 + 16 < rows)
                                get_residual<T, 16>(next, p.epi, m0 + c * 16 + 16, n, p.Nn, rows - c * 16 - 16);
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(taddr + c * 16, r);
                            tmem_wait_ld();
                            if (n < p.Nn)
                                finish_cols<T, true, 16>(p.epi, reinterpret_cast<const float *>(r), res, m0 + c * 16, n,
                                                         p.Nn, rows - c * 16, bias);
#pragma unroll
                            for (int j = 0; j < 16; ++j) res[j] = next[j];
                        }
                    } else {
                        for (int c = 0; c * 32 < rows; ++c) {
                            uint32_t r[32];
                            tmem_ld_32x32b_x32(taddr + c * 32, r);
                            tmem_wait_ld();
                            if (n < p.Nn)
                                store_cols<T, false, 32>(p.epi, reinterpret_cast<const float *>(r), m0 + c * 32, n, p.Nn,
                                                         rows - c * 32, bias);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(tempty0 + 8 * acc);
                    else mbar_arrive_cluster(tempty0_lead + 8 * acc);
                }
                local += SETS;
            }
            if constexpr (SPLIT) {
                if (ok && n < p.Nn) {
#pragma unroll
                    for (int c = 0; c < HMAX / 16; ++c)
                        if (c * 16 < rows)
                            store_cols<T, FULL, 16>(p.epi, sum + c * 16, m0 + c * 16, n, p.Nn, rows - c * 16, bias);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0) publish_status(&g_linear_status, cta_status);
    cluster_sync();  // the pair's MMAs and remote arrivals are done before TMEM goes
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------- one CTA, K split over a cluster
// For products with few tiles.  A cluster of S CTAs computes a 128 (n) x BN (m)
// tile of D, CTA r its share of the K blocks; each leaves its sums in shared
// memory, and after a cluster barrier CTA r adds the S parts of its share of the
// columns in order (through distributed shared memory) and stores them.  Small
// batches stream W this way: BN is the batch rounded up to 16, 32, 64 or 128.
// Two bf16 CTAs fit an SM, so one's start and end overlap the other's copies; an
// fp32 stage (three planes) needs the whole SM.
constexpr int kSplitThreads = 192;
constexpr int split_ctas(bool fp32) { return fp32 ? 1 : 2; }
constexpr int kSplitSmem = 216 * 1024;

// Columns of one accumulator, and of the two that a CTA has.
template <int BN> constexpr int split_acc_cols() { return BN < 32 ? 32 : BN; }
template <int BN> constexpr uint32_t split_tmem_cols() { return 2 * split_acc_cols<BN>(); }
template <int BN> constexpr int split_b_bytes(bool mn) { return (mn && BN < 64 ? 64 : BN) * kBK * 2; }
template <typename T, int BN> constexpr int split_stage_bytes(bool mn) {
    return (sizeof(T) == 4 ? 3 : 1) * (128 * kBK * 2 + split_b_bytes<BN>(mn));
}
// Stages of a ring, and a launch's shared memory: the ring, over which the sums go.
constexpr int kSplitMaxStages = 6;
constexpr int split_stages(bool fp32, int stage_bytes) {
    const int n = (kSplitSmem / split_ctas(fp32) - 1024) / stage_bytes;
    return n > kSplitMaxStages ? kSplitMaxStages : n;
}
template <typename T, int BN> constexpr int split_smem(int stage_bytes) {
    const int ring = split_stages(sizeof(T) == 4, stage_bytes) * stage_bytes;
    return 1024 + (ring > BN * 512 ? ring : BN * 512);
}
// The most that any launch of the kernel asks for.  The limit set on a kernel is
// this one whatever the call needs: it belongs to the kernel, and a call that set
// a smaller one would take it from under another thread's launch.
template <typename T, int BN> constexpr int split_smem_limit() {
    constexpr int k = split_smem<T, BN>(split_stage_bytes<T, BN>(false));
    constexpr int mn = split_smem<T, BN>(split_stage_bytes<T, BN>(true));
    static_assert(tmem_room(split_tmem_cols<BN>(), k < mn ? k : mn), "tensor memory");
    return k > mn ? k : mn;
}

// One product or two (dW and dx, which share a launch); blocks [0, tiles0 S) are
// the first's.
struct SplitArgs {
    ProdArgs p[2];
    int tiles0, S, stages;
    uint64_t timeout_ns;
};

// Adds the cluster's S <= C parts of columns [j0, j0 + mine) of this lane's n, in
// rank order, and stores them: 32 loads in flight (loaded one after the other
// they took 10 us of a 28 us decode product).
template <typename T, int C>
__device__ __forceinline__ void add_parts(const ProdArgs &p, uint32_t at, int S, int j0, int mine, int64_t m0, int n,
                                          float bias) {
    constexpr int J = 32 / C;
    uint32_t peer[C];
#pragma unroll
    for (int c = 0; c < C; ++c) peer[c] = map_to_cta(at, c < S ? c : 0);
    for (int j = 0; j < mine; j += J) {
        float u[J][C], v[J];
#pragma unroll
        for (int i = 0; i < J; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                u[i][c] = 0.0f;
                if (c < S && j + i < mine)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(u[i][c])
                                 : "r"(peer[c] + static_cast<uint32_t>(j0 + j + i) * 512u)
                                 : "memory");
            }
#pragma unroll
        for (int i = 0; i < J; ++i) {
            v[i] = u[i][0];
#pragma unroll
            for (int c = 1; c < C; ++c) v[i] += u[i][c];
        }
        store_cols<T, true, J>(p.epi, v, m0 + j0 + j, n, p.Nn, mine - j, bias);
    }
}

template <typename T, int BN>
__global__ void __launch_bounds__(kSplitThreads, split_ctas(sizeof(T) == 4))
linear_split_kernel(const __grid_constant__ CUtensorMap tp0, const __grid_constant__ CUtensorMap tq0,
                    const __grid_constant__ CUtensorMap tp1, const __grid_constant__ CUtensorMap tq1,
                    const __grid_constant__ SplitArgs args) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PLANES = SPLIT ? 3 : 1, TERMS = SPLIT ? kTerms : 1;
    constexpr int COLS = split_acc_cols<BN>();
    constexpr uint32_t TMEM_COLS = split_tmem_cols<BN>();
    constexpr uint32_t A_BYTES = 128 * kBK * 2;
    constexpr int kMaxStages = kSplitMaxStages;
    const int S = args.S, stages = args.stages;
    const uint64_t tmo = args.timeout_ns;
    int tile = static_cast<int>(blockIdx.x / static_cast<unsigned>(S));
    const bool second = tile >= args.tiles0;
    if (second) tile -= args.tiles0;
    const ProdArgs &p = args.p[second ? 1 : 0];
    const CUtensorMap *tp = second ? &tp1 : &tp0, *tq = second ? &tq1 : &tq0;
    const uint32_t b_bytes = split_b_bytes<BN>(p.q_mn != 0);
    const uint32_t stage_bytes = PLANES * (A_BYTES + b_bytes);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t tmem_holder;
    __shared__ uint32_t cta_status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    uint32_t *status = &cta_status;
    const uint32_t smem_base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
    const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[kMaxStages]);
    const uint32_t tfull0 = smem_u32(&bars[2 * kMaxStages]), tempty0 = smem_u32(&bars[2 * kMaxStages + 2]);
    const uint32_t drain = smem_u32(&bars[2 * kMaxStages + 4]);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(tfull0, 1);
        mbar_init(tfull0 + 8, 1);
        mbar_init(tempty0, 4);
        mbar_init(tempty0 + 8, 4);
        mbar_init(drain, 1);
        fence_barrier_init();
        cta_status = 0u;
        tma_prefetch_desc(tp);
        tma_prefetch_desc(tq);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_holder), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // behind the allocation: see common.cuh
    const uint32_t tmem_base = tmem_holder;
    pdl_wait();

    const int nt = (p.Nn + 127) / 128;
    const int n0 = tile % nt * 128;
    const int64_t m0 = static_cast<int64_t>(tile / nt) * BN;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / S);
    const int piece = SPLIT ? kPieceKb : kb1 - kb0;

    float sum[BN];
    bool good = true;
    if (kb0 >= kb1) {  // no share of a short K
#pragma unroll
        for (int j = 0; j < BN; ++j) sum[j] = 0.0f;
    }
    if (warp == 0) {
        const uint32_t one = elect_one();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        by_layout(p.p_mn != 0, p.q_mn != 0, [&](auto pm, auto qm) {
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_warp(empty0 + 8 * stage, phase ^ 1u, status, tmo, 71)) {
                    ok = false;
                    break;
                }
                {
                    const uint32_t fb = full0 + 8 * stage, sa = smem_base + stage * stage_bytes;
                    expect_tx_if(one, fb, stage_bytes);
                    const int kx = kb * kBK, mr = static_cast<int>(m0);
#pragma unroll
                    for (int z = 0; z < PLANES; ++z) {
                        const uint32_t a = sa + z * A_BYTES, b = sa + PLANES * A_BYTES + z * b_bytes;
                        if constexpr (decltype(pm)::value) {
                            load_if(one, a, tp, fb, n0, kx, z);
                            load_if(one, a + 8192u, tp, fb, n0 + 64, kx, z);
                        } else {
                            load_if(one, a, tp, fb, kx, n0, z);
                        }
                        if constexpr (decltype(qm)::value) {
                            load_if(one, b, tq, fb, mr, kx, z);
                            if constexpr (BN == 128) load_if(one, b + 8192u, tq, fb, mr + 64, kx, z);
                        } else {
                            load_if(one, b, tq, fb, kx, mr, z);
                        }
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        });
        if (!ok && one) {
            int st = stage;
            uint32_t ph = phase;
            for (int i = 0; i < stages && i < issued; ++i) {
                if (st == 0) {
                    st = stages - 1;
                    ph ^= 1u;
                } else {
                    --st;
                }
                wait_drain(full0 + 8 * st, ph, tmo);
            }
        }
    } else if (warp == 1) {
        const uint32_t one = elect_one();
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true, any = false;
        by_layout(p.p_mn != 0, p.q_mn != 0, [&](auto pm, auto qm) {
            constexpr bool PM = decltype(pm)::value, QM = decltype(qm)::value;
            constexpr uint32_t idesc = idesc_bf16_f32(128, BN) | (PM ? kIdescAMajorMN : 0u) | (QM ? kIdescBMajorMN : 0u);
            constexpr uint32_t astep = PM ? 128u : 2u, bstep = QM ? 128u : 2u;
            for (int k0 = kb0; k0 < kb1 && ok; k0 += piece, ++local) {
                const int n = k0 + piece < kb1 ? piece : kb1 - k0;
                const int acc = local & 1;
                if (!wait_warp(tempty0 + 8 * acc, ((local >> 1) & 1) ^ 1u, status, tmo, 72)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * COLS);
                for (int k = 0; k < n; ++k) {
                    if (!wait_warp(full0 + 8 * stage, phase, status, tmo, 73)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    {
                        const uint32_t sa = smem_base + stage * stage_bytes;
                        const uint32_t sb = sa + PLANES * A_BYTES;
                        const uint64_t ad = PM ? smem_desc_mn_sw128(sa, 8192u, 1024u) : smem_desc_sw128(sa);
                        const uint64_t bd = QM ? smem_desc_mn_sw128(sb, 8192u, 1024u) : smem_desc_sw128(sb);
#pragma unroll
                        for (int x = 0; x < TERMS; ++x) {
                            const uint64_t ax = ad + (SPLIT ? term_p(x) * (A_BYTES >> 4) : 0);
                            const uint64_t bx = bd + (SPLIT ? term_q(x) * (b_bytes >> 4) : 0);
#pragma unroll
                            for (int kk = 0; kk < kBK / 16; ++kk)
                                mma_if<false>(one, d_tmem, ax + astep * kk, bx + bstep * kk, idesc,
                                          (k > 0 || x > 0 || kk > 0) ? 1u : 0u);
                        }
                        commit_if(one, empty0 + 8 * stage);
                    }
                    __syncwarp();
                    any = true;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                commit_if(ok ? one : 0u, tfull0 + 8 * acc);
                __syncwarp();
            }
        });
        if (!ok && any && one) {
            umma_commit(drain);
            wait_drain(drain, 0, tmo);
        }
    } else {
        const int q = warp & 3;
        int local = 0;
        for (int k0 = kb0; k0 < kb1; k0 += piece, ++local) {
            const int acc = local & 1;
            if (!mbar_wait_warp(tfull0 + 8 * acc, (local >> 1) & 1, status, tmo, 74)) {
                good = false;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * COLS);
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c * 16, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    sum[c * 16 + j] = local == 0 ? __uint_as_float(r[j]) : sum[c * 16 + j] + __uint_as_float(r[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
        }
        if (S > 1 && good) {
            // the ring is idle: every copy has landed and every MMA has read it
            float *part = reinterpret_cast<float *>(dyn_smem + (smem_base - smem_u32(dyn_smem)));
#pragma unroll
            for (int j = 0; j < BN; ++j) part[j * 128 + q * 32 + lane] = sum[j];
        }
    }
    const int64_t left = p.M - m0;
    const int rows = left < BN ? static_cast<int>(left) : BN;
    const int lane_n = (warp & 3) * 32 + lane, n = n0 + lane_n;
    if (S > 1) {
        __syncwarp();
        __syncthreads();
        cluster_sync();
        if (warp >= 2 && n < p.Nn) {
            const float bias = p.epi.bias != nullptr ? p.epi.bias[n] : 0.0f;
            const int share = (rows + S - 1) / S, j0 = rank * share;
            const int mine = rows - j0 < share ? rows - j0 : share;
            if (S <= 2) add_parts<T, 2>(p, smem_base + static_cast<uint32_t>(lane_n) * 4u, S, j0, mine, m0, n, bias);
            else if (S <= 4) add_parts<T, 4>(p, smem_base + static_cast<uint32_t>(lane_n) * 4u, S, j0, mine, m0, n, bias);
            else add_parts<T, 8>(p, smem_base + static_cast<uint32_t>(lane_n) * 4u, S, j0, mine, m0, n, bias);
        }
    } else if (warp >= 2 && good && n < p.Nn) {
        const float bias = p.epi.bias != nullptr ? p.epi.bias[n] : 0.0f;
#pragma unroll
        for (int c = 0; c < BN / 16; ++c)
            if (c * 16 < rows) store_cols<T, true, 16>(p.epi, sum + c * 16, m0 + c * 16, n, p.Nn, rows - c * 16, bias);
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0) publish_status(&g_linear_status, cta_status);
    if (S > 1) cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

ProdArgs prod_args(const TcProduct &t) {
    return ProdArgs{t.M, t.Nn, (t.K + kBK - 1) / kBK, t.p_mn ? 1 : 0, t.q_mn ? 1 : 0, 0, t.epi};
}

// Limit of a wait: the base, and for the epilogue's wait on a whole tile about ten
// times what the tile's K blocks take.
uint64_t wait_limit(uint64_t base, const TcProduct *t, int count, bool fp32) {
    int kb = 0;
    for (int i = 0; i < count; ++i)
        if ((t[i].K + kBK - 1) / kBK > kb) kb = (t[i].K + kBK - 1) / kBK;
    return base + static_cast<uint64_t>(kb) * (fp32 ? 20000u : 5000u);
}

// Tensor maps of both operands: `planes` planes of [k][row] or [row][k], each
// row `ld` elements (a multiple of 8).
bool operand_map(CUtensorMap *m, const void *base, int planes, int64_t rows, int K, bool mn, int box) {
    const int64_t inner = mn ? (rows + 7) / 8 * 8 : (static_cast<int64_t>(K) + 7) / 8 * 8;
    const int64_t outer = mn ? K : rows;
    return make_tmap_bf16_3d(m, base, planes, static_cast<int>(outer), static_cast<int>(inner), mn ? 64 : box);
}

int pair_units(const TcProduct &t, int tm) {
    return static_cast<int>((t.M + tm - 1) / tm) * ((t.Nn + 255) / 256);
}

// Time of one K block of a tile of tm rows, in cycles.  The MMAs of a bf16 tile
// take 2 tm; the rest was measured (2048 x 12288 x 1280 in one round of 256, one
// of 192, two of 128: 68, 53 and 81 us).  fp32 tiles: six products, 1.14 us at
// 128 rows and 1.61 at 192.
int tile_cycles(int tm, bool fp32) {
    if (fp32) return tm == 128 ? 2170 : 3060;
    return tm == 128 ? 303 : tm == 192 ? 399 : 512;
}

// How a launch deals its units: see PairArgs.
struct PairPlan {
    int tm[2], units[2];
    int late, early;
    int64_t cycles;
};

// The tile heights (and, with two products, the early units) that finish first.
// At 2048 x 1280, 40 tiles of 256 rows leave half the pairs without work and 80
// of 128 take two rounds; 55 of 192 take one.
PairPlan pair_plan(const TcProduct *t, int count, bool fp32, int pairs) {
    PairPlan best{};
    best.cycles = INT64_MAX;
    for (int tm0 = pair_max_tm(fp32); tm0 >= 128; tm0 -= 64) {
        const int n0 = pair_units(t[0], tm0);
        const int64_t u0 = static_cast<int64_t>((t[0].K + kBK - 1) / kBK) * tile_cycles(tm0, fp32);
        const int late = n0 % pairs;
        const int64_t low = n0 / pairs * u0, high = low + (late != 0 ? u0 : 0);
        if (count == 1) {
            if (high < best.cycles) best = PairPlan{{tm0, 0}, {n0, 0}, 0, 0, high};
            continue;
        }
        for (int tm1 = pair_max_tm(fp32); tm1 >= 128; tm1 -= 64) {
            const int n1 = pair_units(t[1], tm1);
            const int64_t u1 = static_cast<int64_t>((t[1].K + kBK - 1) / kBK) * tile_cycles(tm1, fp32);
            const int first = late != 0 ? static_cast<int>(u0 / u1) : 0;
            for (int early = first; early <= first + (late != 0 ? 1 : 0); ++early) {
                const int64_t head = static_cast<int64_t>(early) * (pairs - late);
                int64_t end = high;
                if (n1 <= head) {
                    const int64_t done = low + (n1 + pairs - late - 1) / (pairs - late) * u1;
                    if (done > end) end = done;
                } else {
                    if (low + early * u1 > end) end = low + early * u1;
                    end += (n1 - head + pairs - 1) / pairs * u1;
                }
                if (end < best.cycles) best = PairPlan{{tm0, tm1}, {n0, n1}, late, early, end};
            }
        }
    }
    return best;
}

template <typename T, bool FULL>
cudaError_t launch_pair(const TcProduct *t, int count, uint64_t timeout_ns, int num_sms, cudaStream_t s) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PLANES = SPLIT ? 3 : 1;
    auto kern = linear_pair_kernel<T, FULL>;
    constexpr int smem = kPairRing + 1024;
    static_assert(tmem_room(512, smem), "tensor memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // pairs that fit the device at once, asked for once per device
    static std::atomic<int> fit[64];
    int dev = 0, pairs = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev < 64) pairs = fit[dev].load(std::memory_order_relaxed);
    if (pairs == 0) {
        pairs = num_sms / 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * pairs);
        cfg.blockDim = dim3(pair_threads(SPLIT));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        int max_clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&max_clusters, kern, &cfg) == cudaSuccess && max_clusters > 0 &&
            max_clusters < pairs)
            pairs = max_clusters;
        (void)cudaGetLastError();
        if (dev < 64) fit[dev].store(pairs, std::memory_order_relaxed);
    }
    CUtensorMap mp[2], mq[2];
    PairArgs a{};
    if (pairs > pair_units(t[0], 128) + (count == 2 ? pair_units(t[1], 128) : 0))
        pairs = pair_units(t[0], 128) + (count == 2 ? pair_units(t[1], 128) : 0);
    const PairPlan plan = pair_plan(t, count, SPLIT, pairs);
    a.late = plan.late;
    a.early = plan.early;
    for (int i = 0; i < count; ++i) {
        a.p[i] = prod_args(t[i]);
        a.p[i].tm = plan.tm[i];
        a.units[i] = plan.units[i];
        const int q = pair_q_bytes(a.p[i].tm, t[i].q_mn);
        if (q > a.q_room) a.q_room = q;
        if (!operand_map(&mp[i], t[i].P, PLANES, t[i].Nn, t[i].K, t[i].p_mn, 128) ||
            !operand_map(&mq[i], t[i].Q, PLANES, t[i].M, t[i].K, t[i].q_mn, a.p[i].tm / 2))
            return cudaErrorInvalidValue;
    }
    if (count == 1) {
        mp[1] = mp[0];
        mq[1] = mq[0];
    }
    a.stages = kPairRing / (PLANES * (128 * kBK * 2 + a.q_room));
    if (a.stages > kPairMaxStages) a.stages = kPairMaxStages;
    a.timeout_ns = wait_limit(timeout_ns, t, count, SPLIT);
    return launch_pdl(kern, dim3(2 * pairs), dim3(pair_threads(SPLIT)), smem, s, mp[0], mq[0], mp[1], mq[1], a);
}

int64_t split_tiles(const TcProduct &t, int bn) {
    return static_cast<int64_t>((t.Nn + 127) / 128) * ((t.M + bn - 1) / bn);
}

template <typename T, int BN>
cudaError_t launch_split(const TcProduct *t, int count, int S, uint64_t timeout_ns, cudaStream_t s) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PLANES = SPLIT ? 3 : 1;
    CUtensorMap mp[2], mq[2];
    SplitArgs a{};
    int stage_bytes = 0;
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i) {
        if (!operand_map(&mp[i], t[i].P, PLANES, t[i].Nn, t[i].K, t[i].p_mn, 128) ||
            !operand_map(&mq[i], t[i].Q, PLANES, t[i].M, t[i].K, t[i].q_mn, BN))
            return cudaErrorInvalidValue;
        a.p[i] = prod_args(t[i]);
        const int b = split_stage_bytes<T, BN>(t[i].q_mn);
        if (b > stage_bytes) stage_bytes = b;
        tiles += split_tiles(t[i], BN);
        if (i == 0) a.tiles0 = static_cast<int>(tiles);
    }
    if (count == 1) {
        mp[1] = mp[0];
        mq[1] = mq[0];
    }
    if (tiles * S > INT32_MAX) return cudaErrorInvalidValue;
    a.S = S;
    a.stages = split_stages(SPLIT, stage_bytes);
    a.timeout_ns = wait_limit(timeout_ns, t, count, SPLIT);
    const int smem = split_smem<T, BN>(stage_bytes);
    auto kern = linear_split_kernel<T, BN>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, split_smem_limit<T, BN>());
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
    cfg.blockDim = dim3(kSplitThreads);
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
    return cudaLaunchKernelEx(&cfg, kern, mp[0], mq[0], mp[1], mq[1], a);
}

// Whether a product has tiles enough to run on CTA pairs.
bool use_pairs(const TcProduct &t, bool fp32, int num_sms) {
    const PairPlan p = pair_plan(&t, 1, fp32, num_sms / 2);
    return p.units[0] * 2 >= num_sms / 2;
}

// One or two products on the split kernel.  BN is the batch rounded up; with
// many rows it shrinks from 128 as long as not every SM has a CTA.  S: two K
// blocks a CTA at least.
template <typename T>
cudaError_t run_split(const TcProduct *t, int count, uint64_t timeout_ns, int num_sms, cudaStream_t s) {
    int64_t rows = 0;
    int kb = 0;
    for (int i = 0; i < count; ++i) {
        if (t[i].M > rows) rows = t[i].M;
        if ((t[i].K + kBK - 1) / kBK > kb) kb = (t[i].K + kBK - 1) / kBK;
    }
    const int max_split = kb / 2 > 8 ? 8 : kb / 2 < 1 ? 1 : kb / 2;
    auto tiles = [&](int bn) {
        int64_t n = 0;
        for (int i = 0; i < count; ++i) n += split_tiles(t[i], bn);
        return n;
    };
    int bn = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    while (bn > 32 && tiles(bn) * max_split < num_sms) bn /= 2;
    int S = static_cast<int>(split_ctas(sizeof(T) == 4) * num_sms / tiles(bn));
    if (S > max_split) S = max_split;
    if (S < 1) S = 1;
    // planned for both, so that a gradient's bits do not depend on what else is wanted
    if (t[0].epi.out == nullptr) {
        ++t;
        --count;
    }
    if (count == 2 && t[1].epi.out == nullptr) --count;
    if (count == 0 || t[0].epi.out == nullptr) return cudaSuccess;
    switch (bn) {
    case 16: return launch_split<T, 16>(t, count, S, timeout_ns, s);
    case 32: return launch_split<T, 32>(t, count, S, timeout_ns, s);
    case 64: return launch_split<T, 64>(t, count, S, timeout_ns, s);
    default: return launch_split<T, 128>(t, count, S, timeout_ns, s);
    }
}

}  // namespace

cudaError_t launch_tc_products(const TcProduct *t, int count, bool fp32, bool full, uint64_t timeout_ns, int num_sms,
                               cudaStream_t s) {
    // products of one kind share a launch; on the split kernel only if their K are
    // alike, since they share the number of splits (backward of 11 x 192 -> 4432 fp32
    // 48 us in one launch, 27 in two)
    const bool first = use_pairs(t[0], fp32, num_sms);
    const bool alike = count == 1 || first || (t[0].K <= 4 * static_cast<int64_t>(t[1].K) + 512 &&
                                               t[1].K <= 4 * static_cast<int64_t>(t[0].K) + 512);
    if (count == 2 && (use_pairs(t[1], fp32, num_sms) != first || !alike)) {
        cudaError_t e = launch_tc_products(t, 1, fp32, full, timeout_ns, num_sms, s);
        return e != cudaSuccess ? e : launch_tc_products(t + 1, 1, fp32, full, timeout_ns, num_sms, s);
    }
    if (!first)
        return fp32 ? run_split<float>(t, count, timeout_ns, num_sms, s)
                    : run_split<__nv_bfloat16>(t, count, timeout_ns, num_sms, s);
    // a tile's height does not change a sum's order, so a product alone is planned alone
    if (t[0].epi.out == nullptr) {
        ++t;
        --count;
    }
    if (count == 2 && t[1].epi.out == nullptr) --count;
    if (count == 0 || t[0].epi.out == nullptr) return cudaSuccess;
    if (fp32)
        return full ? launch_pair<float, true>(t, count, timeout_ns, num_sms, s)
                    : launch_pair<float, false>(t, count, timeout_ns, num_sms, s);
    return full ? launch_pair<__nv_bfloat16, true>(t, count, timeout_ns, num_sms, s)
                : launch_pair<__nv_bfloat16, false>(t, count, timeout_ns, num_sms, s);
}

}  // namespace moe
