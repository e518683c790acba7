// Block-FP8 products of many weights at once: each expert's rows, gathered by
// index or in place, times that expert's weights, with bias, activation or gate
// in the epilogue.
//   z[p, j] = sum over k-blocks b of sa[r, b] sw[e, j / 128, b] S(r, e, j, b),
//   S = sum over the 128 k of block b of dec(a[r, k]) dec(w[e, j, k]),
// for the positions p of expert e, with r = rows[p] or p.
//
// One CTA per SM works through tiles of 128 positions x BN columns, an expert's
// row tiles next to each other for each of its weight panels, so that a panel
// is read from HBM once. A tile that reaches past an expert's last row computes
// rows that are not stored. Per k-block of 128:
//   warp 0      TMA: the tile's activation rows, by index four rows at a time
//               (tile::gather4, one instruction per lane) or in boxes of 32
//               rows; only as many rows as the tile has;
//   warp 1      TMA: BN weight rows in two boxes (gated: the first half from
//               the gate's rows, the second from the other half's);
//   warp 2      tcgen05.mma.kind::f8f6f4 (M 128, N BN, K 32) into a ring of
//               TMEM partials;
//   warps 4-11  promotion: acc += partial * fl(sa * sw) in f32 registers, one
//               row and BN / 2 columns per thread (gated: BN / 4 of each half,
//               so that a thread holds both factors of its results).
// The scales are f32 and differ per k-block, so each k-block's partial has to
// leave TMEM; warps whose 32 rows all lie past the tile's last row skip that.
#include "bq.h"
#include "bq_device.cuh"
#include "bq_epi.cuh"
#include "bq_internal.h"
#include "bq_tc.cuh"

namespace bq {
namespace {

constexpr int XM = 128, XK = 128, X_NT = 384;
constexpr int X_TABLE = 256;                 // entries of the tile table
constexpr int REGX_LAUNCH = 168, REGX_CTL = 56, REGX_ACC = 224;
static_assert(128 * REGX_CTL + 256 * REGX_ACC <= X_NT * REGX_LAUNCH, "register split");

template <int BN>
struct PlanX {
    static constexpr uint32_t A_BYTES = XM * XK, W_BYTES = BN * XK;
    static constexpr int S = (int)(196608 / (A_BYTES + W_BYTES));   // ring stages
    static constexpr int NB = 512 / BN < 4 ? 512 / BN : 4;          // TMEM partials
    static constexpr uint32_t TMEM = (uint32_t)(NB * BN);
    static constexpr uint32_t OFF_A = 0, OFF_W = S * A_BYTES;
    static constexpr uint32_t OFF_STAGE = OFF_W + S * W_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_STAGE + 8 * EPI_WARP_BYTES;
    static constexpr int B_FULL_A = 0, B_FULL_W = B_FULL_A + S, B_EMPTY = B_FULL_W + S, B_TFULL = B_EMPTY + S,
                         B_TEMPTY = B_TFULL + NB, B_DONE = B_TEMPTY + NB, N_BAR = B_DONE + 1;
    static constexpr uint32_t OFF_MISC = OFF_BAR + N_BAR * 8;        // [0] TMEM base, [1] abort flag, [2] tiles, [4..11] scan
    static constexpr uint32_t OFF_TABLE = OFF_MISC + 48;
    static constexpr uint32_t SMEM = OFF_TABLE + X_TABLE * 4 + 1024; // room to align the base to 1024
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(W_BYTES % 2048 == 0, "both weight boxes start on 1024-byte boundaries");
};

struct ExpertArgs {
    int64_t a_rows, k, n, p;      // p: rows of c
    int nkb, n_experts, ntiles;
    int per_entry;                // experts per table entry
    int nsw;                      // ceil(n / 128)
    const int32_t *rows, *offsets;
    const float *sa, *sw;
    EpiArgs epi;
};

// First position of expert e, within [0, p]. Without offsets one expert has
// every position.
__device__ __forceinline__ int64_t first_of(const ExpertArgs& g, int e) {
    if (!g.offsets) return e == 0 ? 0 : g.p;
    const int64_t o = __ldg(g.offsets + e);
    return o < 0 ? 0 : (o > g.p ? g.p : o);
}
__device__ __forceinline__ int row_tiles(const ExpertArgs& g, int e) {
    const int64_t r = first_of(g, e + 1) - first_of(g, e);
    return r > 0 ? (int)((r + XM - 1) / XM) : 0;
}

struct Tile {
    int e, nt, rows;
    int64_t p0;
};
// Tile u: table[i] holds the row tiles before expert i * per_entry.
__device__ __forceinline__ Tile tile_at(const ExpertArgs& g, const volatile int* table, int64_t u) {
    const int q = (int)(u / g.ntiles);             // row tiles before, had each one panel after another
    int lo = 0, hi = (g.n_experts + g.per_entry - 1) / g.per_entry - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] <= q) lo = mid; else hi = mid - 1;
    }
    int before = table[lo], e = lo * g.per_entry, mine = row_tiles(g, e);
    while (before + mine <= q && e + 1 < g.n_experts) {
        before += mine;
        mine = row_tiles(g, ++e);
    }
    const int64_t v = u - (int64_t)before * g.ntiles;
    Tile t;
    t.e = e;
    t.nt = mine > 0 ? (int)(v / mine) : 0;
    const int mt = mine > 0 ? (int)(v - (int64_t)t.nt * mine) : 0;
    t.p0 = first_of(g, e) + (int64_t)mt * XM;
    const int64_t left = first_of(g, e + 1) - t.p0;
    t.rows = left < XM ? (int)left : XM;
    return t;
}

// Four rows by index (128 bytes of each, in the 128-byte swizzle).
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* tm, int x, int4 r, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                 :: "r"(dst), "l"((uint64_t)tm), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_regs_ready16(uint32_t (&r)[16]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
template <int N, int AT, int M>
__device__ __forceinline__ void add_scaled(F2 (&acc)[M], const uint32_t (&r)[N], F2 cf) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        acc[AT + i] = f2_fma(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), cf, acc[AT + i]);
}
// One k-block of promotion: two runs of SW columns at t0 and t1, each with its
// own scale.
template <int SW>
__device__ __forceinline__ void promote_runs(F2 (&acc)[SW], uint32_t t0, uint32_t t1, F2 c0, F2 c1) {
    if constexpr (SW == 16) {
        uint32_t r0[16], r1[16];
        tmem_ld16(t0, r0);
        tmem_ld16(t1, r1);
        tmem_ld_wait();
        tmem_regs_ready16(r0);
        tmem_regs_ready16(r1);
        add_scaled<16, 0>(acc, r0, c0);
        add_scaled<16, 8>(acc, r1, c1);
    } else if constexpr (SW == 32) {
        uint32_t r0[32], r1[32];
        tmem_ld32(t0, r0);
        tmem_ld32(t1, r1);
        tmem_ld_wait();
        tmem_regs_ready(r0);
        tmem_regs_ready(r1);
        add_scaled<32, 0>(acc, r0, c0);
        add_scaled<32, 16>(acc, r1, c1);
    } else {
        uint32_t r0[32], r1[32];
        tmem_ld32(t0, r0);
        tmem_ld32(t0 + 32, r1);
        tmem_ld_wait();
        tmem_regs_ready(r0);
        tmem_regs_ready(r1);
        add_scaled<32, 0>(acc, r0, c0);
        add_scaled<32, 16>(acc, r1, c0);
        tmem_ld32(t1, r0);
        tmem_ld32(t1 + 32, r1);
        tmem_ld_wait();
        tmem_regs_ready(r0);
        tmem_regs_ready(r1);
        add_scaled<32, 32>(acc, r0, c1);
        add_scaled<32, 48>(acc, r1, c1);
    }
}

template <int BN, bool GATED>
__global__ void __launch_bounds__(X_NT, 1) k_fp8_experts(const __grid_constant__ CUtensorMap tm_a,
                                                         const __grid_constant__ CUtensorMap tm_w,
                                                         const __grid_constant__ ExpertArgs g) {
    using P = PlanX<BN>;
    constexpr int S = P::S, NB = P::NB, SW = BN / 4;
    constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(XM >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = sm_addr(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* sb = smem_raw + (base - raw_base);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sb + P::OFF_MISC);
    volatile uint32_t* abort_flag = misc + 1;
    const uint32_t abort_addr = base + P::OFF_MISC + 4;
    volatile int* table = reinterpret_cast<volatile int*>(sb + P::OFF_TABLE);
    auto bar = [&](int i) -> uint32_t { return base + P::OFF_BAR + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            bar_init(bar(P::B_FULL_A + i), 1);
            bar_init(bar(P::B_FULL_W + i), 1);
            bar_init(bar(P::B_EMPTY + i), 1);
        }
        for (int i = 0; i < NB; ++i) { bar_init(bar(P::B_TFULL + i), 1); bar_init(bar(P::B_TEMPTY + i), 8); }
        bar_init(bar(P::B_DONE), 1);
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 && lane == 0) { prefetch_map(&tm_a); prefetch_map(&tm_w); }
    if (warp == 9) tmem_alloc(base + P::OFF_MISC, P::TMEM < 32 ? 32 : P::TMEM);
    // Row tiles before each table entry (exclusive sums over warps 0-7).
    int mine = 0, incl = 0;
    if (warp < 8) {
        for (int i = 0; i < g.per_entry; ++i) {
            const int e = threadIdx.x * g.per_entry + i;
            if (e < g.n_experts) mine += row_tiles(g, e);
        }
        incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) misc[4 + warp] = (uint32_t)incl;
    }
    __syncthreads();
    if (warp < 8) {
        int pre = 0;
        for (int w = 0; w < warp; ++w) pre += (int)misc[4 + w];
        table[threadIdx.x] = pre + incl - mine;
        if (threadIdx.x == 255) misc[2] = (uint32_t)(pre + incl);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int64_t tiles = (int64_t)misc[2] * g.ntiles;
    const int nkb = g.nkb;

    if (warp < 4) {
        set_max_regs_dec<REGX_CTL>();
        if (warp == 0) {
            // Activation rows.
            int i = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
                const Tile t = tile_at(g, table, u);
                int loads;
                uint32_t bytes;
                int4 r = make_int4(0, 0, 0, 0);
                if (g.rows) {
                    loads = (t.rows + 3) >> 2;
                    bytes = (uint32_t)loads * 512u;
                    if (lane < loads) {
                        const int last = t.rows - 1, j = 4 * lane;
                        r.x = __ldg(g.rows + t.p0 + j);
                        r.y = __ldg(g.rows + t.p0 + min(j + 1, last));
                        r.z = __ldg(g.rows + t.p0 + min(j + 2, last));
                        r.w = __ldg(g.rows + t.p0 + min(j + 3, last));
                    }
                } else {
                    loads = (t.rows + 31) >> 5;
                    bytes = (uint32_t)loads * 4096u;
                }
                for (int kb = 0; kb < nkb; ++kb) {
                    const int s = i % S;
                    ok = bar_wait<1, false>(bar(P::B_EMPTY + s), ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag, abort_addr);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const uint32_t fb = bar(P::B_FULL_A + s);
                    if (lane == 0) bar_expect_tx(fb, bytes);
                    __syncwarp();
                    const uint32_t dst = base + P::OFF_A + (uint32_t)s * P::A_BYTES;
                    if (lane < loads) {
                        if (g.rows) tma_gather4(dst + (uint32_t)lane * 512u, &tm_a, kb * XK, r, fb);
                        else tma_2d(dst + (uint32_t)lane * 4096u, &tm_a, kb * XK, (int)(t.p0 + 32 * lane), fb);
                    }
                    ++i;
                }
            }
            for (int j = max(0, i - S); j < i; ++j) bar_drain(bar(P::B_FULL_A + j % S), (uint32_t)(j / S) & 1u);
        } else if (warp == 1 && lane == 0) {
            // Weight rows.
            int i = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
                const Tile t = tile_at(g, table, u);
                const int64_t w0 = (int64_t)t.e * g.n + (int64_t)t.nt * (GATED ? BN / 2 : BN);
                const int y0 = (int)w0, y1 = (int)(w0 + (GATED ? g.n / 2 : BN / 2));
                for (int kb = 0; kb < nkb; ++kb) {
                    const int s = i % S;
                    if (!(ok = bar_wait<1, false>(bar(P::B_EMPTY + s), ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag, abort_addr))) break;
                    const uint32_t fb = bar(P::B_FULL_W + s);
                    bar_expect_tx(fb, P::W_BYTES);
                    const uint32_t dst = base + P::OFF_W + (uint32_t)s * P::W_BYTES;
                    tma_2d(dst, &tm_w, kb * XK, y0, fb);
                    tma_2d(dst + P::W_BYTES / 2, &tm_w, kb * XK, y1, fb);
                    ++i;
                }
            }
            for (int j = max(0, i - S); j < i; ++j) bar_drain(bar(P::B_FULL_W + j % S), (uint32_t)(j / S) & 1u);
        } else if (warp == 2 && lane == 0) {
            // MMA issue.
            int i = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
                for (int kb = 0; kb < nkb; ++kb) {
                    const int buf = i % NB, s = i % S;
                    if (!(ok = bar_wait<1, false>(bar(P::B_TEMPTY + buf), ((uint32_t)(i / NB) & 1u) ^ 1u, abort_flag, abort_addr))) break;
                    if (!(ok = bar_wait<1, false>(bar(P::B_FULL_A + s), (uint32_t)(i / S) & 1u, abort_flag, abort_addr))) break;
                    if (!(ok = bar_wait<1, false>(bar(P::B_FULL_W + s), (uint32_t)(i / S) & 1u, abort_flag, abort_addr))) break;
                    tc_fence_after();
                    const uint64_t da = desc_k_sw128(base + P::OFF_A + (uint32_t)s * P::A_BYTES);
                    const uint64_t dw = desc_k_sw128(base + P::OFF_W + (uint32_t)s * P::W_BYTES);
#pragma unroll
                    for (int k4 = 0; k4 < XK / 32; ++k4)
                        mma_f8(tmem + (uint32_t)(buf * BN), da + (uint64_t)(2 * k4), dw + (uint64_t)(2 * k4), IDESC, k4 > 0 ? 1u : 0u);
                    mma_commit(bar(P::B_TFULL + buf));
                    mma_commit(bar(P::B_EMPTY + s));
                    ++i;
                }
            }
            mma_commit(bar(P::B_DONE));
            bar_drain(bar(P::B_DONE), 0u);
        }
    } else {
        // ---------------------------------------------------- promotion
        set_max_regs_inc<REGX_ACC>();
        const int q = warp & 3, h = (warp - 4) >> 2;
        float* stage = reinterpret_cast<float*>(sb + P::OFF_STAGE + (uint32_t)(warp - 4) * EPI_WARP_BYTES);
        // This thread's two runs of SW columns of the tile.
        const int run0 = GATED ? h * SW : h * 2 * SW, run1 = GATED ? BN / 2 + h * SW : run0 + SW;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        int i = 0;
        bool ok = true;
        F2 acc[SW];
        for (int64_t u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
            const Tile t = tile_at(g, table, u);
            const int mine_rows = min(32, t.rows - 32 * q);      // this warp's rows
            const bool busy = mine_rows > 0;
            const int64_t col = (int64_t)t.nt * (GATED ? BN / 2 : BN) + run0;   // first column of z (gate)
            int64_t ar = -1;
            if (lane < mine_rows) {
                const int64_t p = t.p0 + 32 * q + lane;
                ar = g.rows ? (int64_t)__ldg(g.rows + p) : p;
                if (ar >= g.a_rows) ar = -1;
            }
            const bool row_in = ar >= 0;
            const float* sap = g.sa + (row_in ? ar * nkb : 0);
            const bool col_in = col < g.n;
            const float* swp = g.sw + ((int64_t)t.e * g.nsw + (col_in ? col / 128 : 0)) * nkb;
            const float* sup = GATED ? g.sw + ((int64_t)t.e * g.nsw + (g.n / 2 + col) / 128) * nkb : swp;
            const bool use = row_in && col_in;
#pragma unroll
            for (int j = 0; j < SW; ++j) acc[j] = 0ull;
            // Scales two blocks ahead.
            float a0 = use ? __ldg(sap) : 0.0f, w0 = use ? __ldg(swp) : 0.0f, v0 = GATED && use ? __ldg(sup) : 0.0f;
            const bool two = use && nkb > 1;
            float a1 = two ? __ldg(sap + 1) : 0.0f, w1 = two ? __ldg(swp + 1) : 0.0f, v1 = GATED && two ? __ldg(sup + 1) : 0.0f;
            for (int kb = 0; kb < nkb; ++kb) {
                const bool more = use && kb + 2 < nkb;
                const float a2 = more ? __ldg(sap + kb + 2) : 0.0f, w2 = more ? __ldg(swp + kb + 2) : 0.0f;
                const float v2 = GATED && more ? __ldg(sup + kb + 2) : 0.0f;
                const int buf = i % NB;
                ok = bar_wait<1, false>(bar(P::B_TFULL + buf), (uint32_t)(i / NB) & 1u, abort_flag, abort_addr);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;      // the warp goes on, or stops, as one
                tc_fence_after();
                if (busy) {
                    const F2 c0 = f2_bcast(__fmul_rn(a0, w0)), c1 = GATED ? f2_bcast(__fmul_rn(a0, v0)) : c0;
                    const uint32_t tb = lane_base + (uint32_t)(buf * BN);
                    promote_runs<SW>(acc, tb + (uint32_t)run0, tb + (uint32_t)run1, c0, c1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(P::B_TEMPTY + buf));
                ++i;
                a0 = a1; a1 = a2;
                w0 = w1; w1 = w2;
                v0 = v1; v1 = v2;
            }
            if (!ok) break;
            if (busy) {
                // 32 staged columns at a time: of both runs (gated), or consecutive ones.
#pragma unroll
                for (int c = 0; c < SW / 16; ++c) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        f2_split(acc[GATED ? 8 * c + j : 16 * c + j], v[2 * j], v[2 * j + 1]);
                        f2_split(acc[GATED ? SW / 2 + 8 * c + j : 16 * c + 8 + j], v[16 + 2 * j], v[16 + 2 * j + 1]);
                    }
                    const int64_t at = col + (GATED ? 16 : 32) * c;
                    epi_chunk<GATED>(g.epi, stage, lane, t.p0 + 32 * q, mine_rows, at, (int64_t)t.e * g.n + at, v);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM < 32 ? 32 : P::TMEM);
    }
}

template <int BN, bool GATED>
cudaError_t launch_experts(const uint8_t* a, const uint8_t* w, const ExpertArgs& ga, int64_t most_tiles, cudaStream_t st) {
    using P = PlanX<BN>;
    static int ready[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    auto kern = k_fp8_experts<BN, GATED>;
    cudaError_t e;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
        if (fa.numRegs != REGX_LAUNCH) return cudaErrorNotSupported;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::SMEM)) != cudaSuccess) return e;
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    ExpertArgs g = ga;
    const int64_t width = GATED ? BN / 2 : BN;
    g.ntiles = (int)((g.epi.n_out + width - 1) / width);
    CUtensorMap ta, tw;
    if ((e = encode_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, (uint64_t)g.k, (uint64_t)g.a_rows, (uint64_t)g.k, XK,
                        g.rows ? 1 : 32)) != cudaSuccess)
        return e;
    if ((e = encode_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)g.k, (uint64_t)(g.n * g.n_experts), (uint64_t)g.k,
                        XK, BN / 2)) != cudaSuccess)
        return e;
    int64_t grid = sm_count();
    if (grid > most_tiles * g.ntiles) grid = most_tiles * g.ntiles;
    kern<<<(unsigned)grid, X_NT, P::SMEM, st>>>(ta, tw, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t experts_error_take(unsigned int* flag) { return take_gemm_error(flag); }

cudaError_t fp8_experts(const uint8_t* a, const float* sa, int64_t a_rows, int64_t k, const int32_t* rows,
                        const int32_t* offsets, int n_experts, int64_t p, const uint8_t* w, const float* sw, int64_t n,
                        const void* bias, int bias_t, int act, int gated, const void* residual, void* c, int c_t, void* pre,
                        cudaStream_t st) {
    ExpertArgs g = {};
    g.a_rows = a_rows; g.k = k; g.n = n; g.p = p;
    g.nkb = (int)(k / XK);
    g.n_experts = n_experts;
    g.per_entry = (n_experts + X_TABLE - 1) / X_TABLE;
    g.nsw = (int)((n + 127) / 128);
    g.rows = rows; g.offsets = offsets; g.sa = sa; g.sw = sw;
    g.epi.bias = bias; g.epi.bias_t = bias_t;
    g.epi.residual = residual; g.epi.c = c; g.epi.pre = pre; g.epi.c_t = c_t;
    g.epi.n = n; g.epi.n_out = gated ? n / 2 : n;
    g.epi.act = act;
    g.epi.vec = g.epi.n_out % 4 == 0;
    // Row tiles at most: one started per expert that can have a row, and the full ones.
    const int64_t most = (p < n_experts ? p : n_experts) + p / XM;
    return gated ? launch_experts<256, true>(a, w, g, most, st) : launch_experts<256, false>(a, w, g, most, st);
}

}  // namespace bq

static bool float_out(bq_dtype t) { return t == BQ_F32 || t == BQ_F16 || t == BQ_BF16; }

extern "C" bq_status bq_fp8_grouped_gemm(const uint8_t* a_e4m3, const float* a_scale, int64_t a_rows, int64_t k,
                                         const int32_t* rows, const int32_t* offsets, int32_t n_experts, int64_t c_rows,
                                         const uint8_t* w_e4m3, const float* w_scale, int64_t n, const void* bias,
                                         bq_dtype bias_dtype, bq_act act, int32_t gated, void* c, bq_dtype c_dtype,
                                         void* stream) {
    if (!float_out(c_dtype) || (bias && !float_out(bias_dtype))) return BQ_ERR_UNSUPPORTED;
    if (act < BQ_ACT_NONE || act > BQ_ACT_SILU) return BQ_ERR_UNSUPPORTED;
    const int64_t most = (1ll << 31) - 256;          // room for a tile's coordinates past the end
    if (a_rows < 0 || c_rows < 0 || n < 0 || k <= 0 || k % 128 != 0) return BQ_ERR_INVALID_ARG;
    if (a_rows >= most || c_rows >= most || k >= most || n >= most) return BQ_ERR_INVALID_ARG;
    if (n_experts < 1 || n_experts > 1024 || n * n_experts >= most) return BQ_ERR_INVALID_ARG;
    if (gated && n % 256 != 0) return BQ_ERR_INVALID_ARG;
    if (c_rows == 0 || n == 0) return BQ_OK;
    if (!offsets || !w_e4m3 || !w_scale || !c) return BQ_ERR_INVALID_ARG;
    if (!a_e4m3 || !a_scale || a_rows == 0) return BQ_ERR_INVALID_ARG;
    if (((uintptr_t)a_e4m3 & 15u) || ((uintptr_t)w_e4m3 & 15u) || ((uintptr_t)c & 15u)) return BQ_ERR_MISALIGNED;
    if (((uintptr_t)a_scale & 3u) || ((uintptr_t)w_scale & 3u) || ((uintptr_t)rows & 3u) || ((uintptr_t)offsets & 3u) ||
        ((uintptr_t)bias & (bias_dtype == BQ_F32 ? 3u : 1u)))
        return BQ_ERR_MISALIGNED;
    const cudaError_t e = bq::fp8_experts(a_e4m3, a_scale, a_rows, k, rows, offsets, n_experts, c_rows, w_e4m3, w_scale, n,
                                          bias, bias_dtype, act, gated != 0, nullptr, c, c_dtype, nullptr, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported) return BQ_ERR_UNSUPPORTED;
    return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
}

extern "C" bq_status bq_fp8_block_gemm_epilogue(const uint8_t* a_e4m3, const float* a_scale, int64_t m, int64_t k,
                                                const uint8_t* w_e4m3, const float* w_scale, int64_t n, const void* bias,
                                                bq_dtype bias_dtype, bq_act act, const void* residual, void* c,
                                                bq_dtype c_dtype, void* pre, void* stream) {
    if (!float_out(c_dtype) || (bias && !float_out(bias_dtype))) return BQ_ERR_UNSUPPORTED;
    if (act < BQ_ACT_NONE || act > BQ_ACT_SILU) return BQ_ERR_UNSUPPORTED;
    const int64_t most = (1ll << 31) - 256;
    if (m < 0 || n < 0 || k <= 0 || k % 128 != 0 || m >= most || n >= most || k >= most) return BQ_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return BQ_OK;
    if (!a_e4m3 || !a_scale || !w_e4m3 || !w_scale || !c) return BQ_ERR_INVALID_ARG;
    if (((uintptr_t)a_e4m3 & 15u) || ((uintptr_t)w_e4m3 & 15u) || ((uintptr_t)c & 15u) || ((uintptr_t)residual & 15u) ||
        ((uintptr_t)pre & 15u))
        return BQ_ERR_MISALIGNED;
    if (((uintptr_t)a_scale & 3u) || ((uintptr_t)w_scale & 3u) || ((uintptr_t)bias & (bias_dtype == BQ_F32 ? 3u : 1u)))
        return BQ_ERR_MISALIGNED;
    const cudaError_t e = bq::fp8_experts(a_e4m3, a_scale, m, k, nullptr, nullptr, 1, m, w_e4m3, w_scale, n, bias, bias_dtype,
                                          act, 0, residual, c, c_dtype, pre, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported) return BQ_ERR_UNSUPPORTED;
    return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
}
