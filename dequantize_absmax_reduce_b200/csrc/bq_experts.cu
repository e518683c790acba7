// Block-FP8 products of many weights at once: each expert's rows, gathered by
// index or in place, times that expert's weights, with bias, activation or gate
// in the epilogue.
//   z[p, j] = sum over k-blocks b of sa[r, b] sw[e, j / 128, b] S(r, e, j, b),
//   S = sum over the 128 k of block b of dec(a[r, k]) dec(w[e, j, k]),
// for the positions p of expert e, with r = rows[p] or p.
//
// One CTA per SM works through tiles of XR positions x BN columns, an expert's
// row tiles next to each other for each of its weight panels, so that a panel
// is read from HBM once. A tile that reaches past an expert's last row computes
// rows that are not stored. Per k-block of 128:
//   warps 0, 3  the tile's activation rows: in place by TMA in boxes of 32 rows
//               (warp 0), by index with 16-byte asynchronous copies (both warps:
//               TMA's gather of four rows took 37 ns an instruction, 1.2 us per
//               k-block of 128 rows); only as many rows as the tile has. On the
//               widest tiles warp 3 also copies the block scales;
//   warp 1      TMA: BN weight rows in two boxes (gated: the first half from
//               the gate's rows, the second from the other half's);
//   warp 2      tcgen05.mma.kind::f8f6f4 (M 128, N BN, K 32) into a ring of
//               TMEM partials;
//   warps 4-11  promotion: acc += partial * fl(sa * sw) in f32 registers, one
//               row and BN / 2 columns per thread (gated: BN / 4 of each half,
//               so that a thread holds both factors of its results).
// The scales are f32 and differ per k-block, so each k-block's partial has to
// leave TMEM; warps whose 32 rows all lie past the tile's last row skip that.
//
// What bounds it. Long runs of rows: the promotion's reads of TMEM beside the
// MMA's own (tensor pipe 47-51 % active; 16384 x 4096 x 7168 without extras 463
// us, 2.08 PFLOP/s). Its loop has to keep two loads of 32 columns in flight and
// spill nothing: with one load 750 us, with 100 bytes of spills 670. Few rows:
// the weights' stream from HBM (64 rows on 32 experts of 4096 x 7168: 145 us,
// 5.6 TB/s, 0.86 of the copy rate; call after call, at the power limit, 163).
#include "bq.h"
#include "bq_device.cuh"
#include "bq_epi.cuh"
#include "bq_internal.h"
#include "bq_tc.cuh"

namespace bq {
namespace {

constexpr int XM = 128, XK = 128, X_NT = 384;
constexpr int X_TABLE = 256;                 // entries of the tile table
constexpr int REGX_LAUNCH = 168, REGX_CTL = 88, REGX_ACC = 208;
static_assert(128 * REGX_CTL + 256 * REGX_ACC <= X_NT * REGX_LAUNCH, "register split");

// XR: rows of a tile. The MMA always takes 128; behind a tile of 32 a slot holds
// zeros. Slots of 32 rows, with other slots' bytes behind them, leave the ring a
// fourth stage, but products that nobody reads cost clock at the power limit (64
// rows on 32 experts of 4096 x 7168, call after call at that limit: 173 us against 163).
template <int BN, int XR>
struct PlanX {
    // k-blocks of a ring stage and of a TMEM buffer: each signal between the
    // roles costs the single threads that issue loads and MMAs some 70 clocks, so
    // narrow tiles, whose k-blocks are short, share one between two.
    static constexpr int KS = BN == 256 ? 1 : 2;
    static constexpr uint32_t A_BYTES = XM * XK, W_BYTES = BN * XK; // of a k-block
    // Ring stages. The widest tiles give one up for a ring of scales.
    static constexpr bool SCALES = BN == 256;
    static constexpr int S = (int)((SCALES ? 147456 : 196608) / (KS * (A_BYTES + W_BYTES)));
    static constexpr int NB = 512 / (KS * BN) < 4 ? 512 / (KS * BN) : 4;   // TMEM buffers
    static constexpr uint32_t TMEM = (uint32_t)(NB * KS * BN);
    static constexpr uint32_t OFF_A = 0, OFF_W = S * KS * A_BYTES;
    static constexpr uint32_t OFF_STAGE = OFF_W + S * KS * W_BYTES;
    static constexpr uint32_t OFF_SG = OFF_STAGE + 8 * EpiPlan<BN / 4>::WARP_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_SG + (SCALES ? SG * SG_BYTES : 0);
    static constexpr int B_FULL = 0, B_EMPTY = B_FULL + S, B_TFULL = B_EMPTY + S, B_TEMPTY = B_TFULL + NB,
                         B_DONE = B_TEMPTY + NB, B_SFULL = B_DONE + 1, B_SEMPTY = B_SFULL + (SCALES ? SG : 0),
                         N_BAR = B_SEMPTY + (SCALES ? SG : 0);
    static constexpr uint32_t OFF_MISC = (OFF_BAR + N_BAR * 8 + 15) / 16 * 16;   // [0] TMEM base, [1] abort flag, [2] tiles, [4..11] scan
    static constexpr uint32_t OFF_TABLE = OFF_MISC + 48;
    static constexpr uint32_t SMEM = OFF_TABLE + X_TABLE * 4 + 1024; // room to align the base to 1024
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(W_BYTES % 2048 == 0, "both weight boxes start on 1024-byte boundaries");
    static_assert(TMEM == 512 || TMEM == 256, "a power of two");
};
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

struct ExpertArgs {
    int64_t k, n;
    int a_rows, p;                // p: rows of c
    int nkb, n_experts, ntiles;
    int per_entry;                // experts per table entry
    int nsw;                      // ceil(n / 128)
    const uint8_t* a;
    const int32_t *rows, *offsets;
    const float *sa, *sw;
    EpiArgs epi;
};

// First position of expert e, within [0, p]. Without offsets one expert has
// every position.
__device__ __forceinline__ int first_of(const ExpertArgs& g, int e) {
    if (!g.offsets) return e == 0 ? 0 : g.p;
    return max(0, min(__ldg(g.offsets + e), g.p));
}
template <int XR>
__device__ __forceinline__ int row_tiles(const ExpertArgs& g, int e) {
    const int r = first_of(g, e + 1) - first_of(g, e);
    return r > 0 ? (int)(((unsigned)r + XR - 1) / XR) : 0;
}

struct Tile {
    int e, nt, rows, p0;
};
// Tile u (there are fewer than 2^31): table[i] holds the row tiles before expert
// i * per_entry. An expert's tiles come in bands of 16 row tiles, walked down
// the rows first: the CTAs working at one time share a few weight panels and a
// band of activation rows in L2.
template <int XR>
__device__ __forceinline__ Tile tile_at(const ExpertArgs& g, const volatile int* table, int u) {
    const int q = (int)((unsigned)u / (unsigned)g.ntiles);
    int lo = 0, hi = (g.n_experts - 1) / g.per_entry;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] <= q) lo = mid; else hi = mid - 1;
    }
    int before = table[lo], e = lo * g.per_entry, mine = row_tiles<XR>(g, e);
    while (before + mine <= q && e + 1 < g.n_experts) {
        before += mine;
        mine = row_tiles<XR>(g, ++e);
    }
    const unsigned v = (unsigned)(u - before * g.ntiles), per_band = 16u * (unsigned)g.ntiles;
    const unsigned band = v / per_band, rest = v - band * per_band;
    const unsigned deep = (unsigned)max(1, min(16, mine - 16 * (int)band));
    Tile t;
    t.e = e;
    t.nt = (int)(rest / deep);
    const int first = first_of(g, e), at = (int)(16 * band + rest % deep) * XR;
    t.p0 = first + at;
    t.rows = min(XR, first_of(g, e + 1) - first - at);
    return t;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_cluster_pair(uint32_t cl_addr, F2 x, F2 y) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" :: "r"(cl_addr), "l"(x), "l"(y) : "memory");
}
__device__ __forceinline__ void ld_shared_pair(uint32_t addr, F2& x, F2& y) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(addr) : "memory");
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
    if constexpr (SW == 32) {
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

// SPLIT: the CTAs of a cluster share one tile, each with a run of its k-blocks,
// and the first adds up their sums (in the order of their ranks, through its
// shared memory) and writes the tile: for products of few tiles, which would
// otherwise leave most SMs idle.
// FLAT: c's columns are not a multiple of 8 (see epi_flat).
template <int BN, bool GATED, int XR, bool SPLIT, bool FLAT>
__global__ void __launch_bounds__(X_NT, 1) k_fp8_experts(const __grid_constant__ CUtensorMap tm_a,
                                                         const __grid_constant__ CUtensorMap tm_w,
                                                         const __grid_constant__ ExpertArgs g) {
    using P = PlanX<BN, XR>;
    constexpr int S = P::S, NB = P::NB, KS = P::KS, SW = BN / 4;
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
    // A whole warp waits, and goes on or stops as one.
    auto wait = [&](int b, uint32_t parity) -> bool {
        const bool ok = bar_wait<1, false>(bar(b), parity, abort_flag, abort_addr);
        return __all_sync(0xffffffffu, ok);
    };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            bar_init(bar(P::B_FULL + i), g.rows ? 65 : 2);     // both gathering warps' lanes, or one, and the weights
            bar_init(bar(P::B_EMPTY + i), 1);
        }
        for (int i = 0; i < NB; ++i) { bar_init(bar(P::B_TFULL + i), 1); bar_init(bar(P::B_TEMPTY + i), 8); }
        bar_init(bar(P::B_DONE), 1);
        if (P::SCALES) for (int i = 0; i < SG; ++i) { bar_init(bar(P::B_SFULL + i), 32); bar_init(bar(P::B_SEMPTY + i), 8); }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 && lane == 0) { prefetch_map(&tm_a); prefetch_map(&tm_w); }
    if constexpr (XR < XM) {
        // The tensor core multiplies the rows behind a tile's as well, and at the
        // card's power limit that costs clock. Zeros cost least.
        for (uint32_t i = threadIdx.x * 16u; i < S * KS * P::A_BYTES; i += X_NT * 16u)
            *reinterpret_cast<uint4*>(sb + P::OFF_A + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_shared();
    }
    if (warp == 9) tmem_alloc(base + P::OFF_MISC, P::TMEM);
    // Row tiles before each table entry (exclusive sums over warps 0-7).
    int mine = 0, incl = 0;
    if (warp < 8) {
        for (int i = 0; i < g.per_entry; ++i) {
            const int e = threadIdx.x * g.per_entry + i;
            if (e < g.n_experts) mine += row_tiles<XR>(g, e);
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
    const int tiles = (int)misc[2] * g.ntiles;
    const int nkb = g.nkb;
    const int rank = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
    const int per = (nkb + parts - 1) / parts;
    const int k0 = min(nkb, rank * per), k1 = min(nkb, k0 + per);    // this CTA's k-blocks
    const int u0 = SPLIT ? (int)blockIdx.x / parts : (int)blockIdx.x, ustep = SPLIT ? tiles : (int)gridDim.x;

    if (warp < 4) {
        set_max_regs_dec<REGX_CTL>();
        if (warp == 0 && !g.rows) {
            // Activation rows in place: boxes of 32 rows.
            Ring<S> r;
            bool ok = true;
            for (int u = u0; ok && u < tiles; u += ustep) {
                const Tile t = tile_at<XR>(g, table, u);
                const int loads = (t.rows + 31) >> 5;
                for (int kb = k0; kb < k1; kb += KS) {
                    if (!(ok = wait(P::B_EMPTY + r.slot, r.round ^ 1u))) break;
                    const uint32_t fb = bar(P::B_FULL + r.slot);
                    const int ks = min(KS, k1 - kb);
                    if (elect_one()) {
                        bar_expect_tx(fb, (uint32_t)(ks * loads) * 4096u);
                        for (int h = 0; h < ks; ++h)
                            for (int j = 0; j < loads; ++j)
                                tma_2d(base + P::OFF_A + (uint32_t)(r.slot * KS + h) * P::A_BYTES + (uint32_t)j * 4096u, &tm_a,
                                       (kb + h) * XK, t.p0 + 32 * j, fb);
                    }
                    __syncwarp();
                    r.next();
                }
            }
        } else if (warp == 0 || (warp == 3 && (g.rows || P::SCALES))) {
            // Activation rows by index: warps 0 and 3 take every other four rows.
            // A lane copies the same 16 bytes of a row's 128 for up to 16 rows, into
            // the 128-byte swizzle that the MMA reads (its row modulo 8 is fixed).
            // The copies arrive on the stage's barrier by themselves; the issuing
            // thread of the MMAs then orders them before the tensor core's reads.
            const int part = warp == 3 ? 1 : 0, rl = 4 * part + (lane >> 3), chunk = lane & 7;
            const uint32_t dst0 = base + P::OFF_A + (uint32_t)rl * 128u + (uint32_t)((chunk ^ rl) << 4);
            const uint8_t* src0 = g.a + 16 * chunk;
            const uint32_t row16 = (uint32_t)(g.k >> 4);         // 16-byte units of a row
            // Warp 3 of the widest tiles copies the block scales as well.
            Ring<S> r;
            [[maybe_unused]] Ring<SG> rs;
            [[maybe_unused]] const bool vec = (nkb & 3) == 0 && (((uintptr_t)g.sa | (uintptr_t)g.sw) & 15u) == 0;
            bool ok = true;
            for (int u = u0; ok && u < tiles; u += ustep) {
                const Tile t = tile_at<XR>(g, table, u);
                // In 16-byte units. A row outside the activations reads the first one
                // (its sums are replaced by zeros in the epilogue).
                uint32_t at[XR / 8];
#pragma unroll
                for (int j = 0; j < XR / 8; ++j) {
                    const int row = 8 * j + rl;
                    const int v = g.rows && row < t.rows ? __ldg(g.rows + t.p0 + row) : -1;
                    at[j] = v >= 0 && v < g.a_rows ? (uint32_t)v * row16 : 0u;
                }
                const int loads = (t.rows + 7 - 4 * part) >> 3;  // of this warp: four rows each
                [[maybe_unused]] int srow[4];                    // activation rows of the tile's rows lane, lane + 32, ..
                [[maybe_unused]] const float* swp = nullptr;
                if constexpr (P::SCALES) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at_row = min(lane + 32 * j, t.rows - 1) + t.p0;
                        const int v = g.rows ? __ldg(g.rows + at_row) : at_row;
                        srow[j] = v >= 0 && v < g.a_rows ? v : 0;
                    }
                    // Sets of weight scales: of the two column halves (one past n: unused), or of gate and other half.
                    const int64_t tile = GATED ? (int64_t)t.nt + (lane & 1) * (g.n / 256) : min(2 * t.nt + (lane & 1), g.nsw - 1);
                    swp = g.sw + ((int64_t)t.e * g.nsw + tile) * nkb;
                }
                for (int kb = k0; kb < k1; kb += KS) {
                    if constexpr (P::SCALES) {
                        if (warp == 3 && (kb & 3) == 0) {
                            if (!(ok = wait(P::B_SEMPTY + rs.slot, rs.round ^ 1u))) break;
                            const uint32_t to = base + P::OFF_SG + (uint32_t)rs.slot * SG_BYTES;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                copy_scales4(to + 16u * (uint32_t)(lane + 32 * j), g.sa + (int64_t)srow[j] * nkb, kb, k1, vec);
                            if (lane < 2) copy_scales4(to + 16u * (uint32_t)(128 + lane), swp, kb, k1, vec);
                            copy_arrive(bar(P::B_SFULL + rs.slot));
                            rs.next();
                        }
                        if (!g.rows) continue;
                    }
                    if (!(ok = wait(P::B_EMPTY + r.slot, r.round ^ 1u))) break;
#pragma unroll
                    for (int h = 0; h < KS; ++h) {
                        if (kb + h >= k1) break;
                        const uint32_t dst = dst0 + (uint32_t)(r.slot * KS + h) * P::A_BYTES;
                        const uint8_t* src = src0 + (kb + h) * XK;
#pragma unroll
                        for (int j = 0; j < XR / 8; ++j)
                            if (j < loads) copy16(dst + (uint32_t)j * 1024u, src + 16 * (uint64_t)at[j]);
                    }
                    copy_arrive(bar(P::B_FULL + r.slot));
                    r.next();
                }
            }
            copy_wait_all();                                     // none in flight when the block ends
        } else if (warp == 1) {
            // Weight rows.
            Ring<S> r;
            bool ok = true;
            for (int u = u0; ok && u < tiles; u += ustep) {
                const Tile t = tile_at<XR>(g, table, u);
                const int64_t w0 = (int64_t)t.e * g.n + (int64_t)t.nt * (GATED ? BN / 2 : BN);
                const int y0 = (int)w0, y1 = (int)(w0 + (GATED ? g.n / 2 : BN / 2));
                for (int kb = k0; kb < k1; kb += KS) {
                    if (!(ok = wait(P::B_EMPTY + r.slot, r.round ^ 1u))) break;
                    const uint32_t fb = bar(P::B_FULL + r.slot);
                    const int ks = min(KS, k1 - kb);
                    if (elect_one()) {
                        bar_expect_tx(fb, (uint32_t)ks * P::W_BYTES);
#pragma unroll
                        for (int h = 0; h < KS; ++h) {
                            if (h >= ks) break;
                            const uint32_t dst = base + P::OFF_W + (uint32_t)(r.slot * KS + h) * P::W_BYTES;
                            tma_2d(dst, &tm_w, (kb + h) * XK, y0, fb);
                            tma_2d(dst + P::W_BYTES / 2, &tm_w, (kb + h) * XK, y1, fb);
                        }
                    }
                    __syncwarp();
                    r.next();
                }
            }
        } else if (warp == 2) {
            // MMA issue.
            Ring<S> r;
            Ring<NB> b;
            bool ok = true;
            for (int u = u0; ok && u < tiles; u += ustep) {
                for (int kb = k0; kb < k1; kb += KS) {
                    if (!(ok = wait(P::B_TEMPTY + b.slot, b.round ^ 1u))) break;
                    if (!(ok = wait(P::B_FULL + r.slot, r.round))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (g.rows) fence_async_shared();
                        const uint64_t da = desc_k_sw128(base + P::OFF_A + (uint32_t)(r.slot * KS) * P::A_BYTES);
                        const uint64_t dw = desc_k_sw128(base + P::OFF_W + (uint32_t)(r.slot * KS) * P::W_BYTES);
#pragma unroll
                        for (int h = 0; h < KS; ++h) {
                            if (kb + h >= k1) break;
#pragma unroll
                            for (int k4 = 0; k4 < XK / 32; ++k4)
                                mma_f8(tmem + (uint32_t)((b.slot * KS + h) * BN), da + (uint64_t)(h * (P::A_BYTES >> 4) + 2 * k4),
                                       dw + (uint64_t)(h * (P::W_BYTES >> 4) + 2 * k4), IDESC, k4 > 0 ? 1u : 0u);
                        }
                        mma_commit(bar(P::B_TFULL + b.slot));
                        mma_commit(bar(P::B_EMPTY + r.slot));
                    }
                    __syncwarp();
                    r.next();
                    b.next();
                }
            }
            if (elect_one()) mma_commit(bar(P::B_DONE));
            __syncwarp();
            bar_drain(bar(P::B_DONE), 0u);
        }
        if constexpr (SPLIT) {                                   // as the promotion warps below
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ---------------------------------------------------- promotion
        set_max_regs_inc<REGX_ACC>();
        constexpr int G = 4;                                     // k-blocks whose scales are loaded together
        // Rows of scales, and this CTA's run of k-blocks, start on 16-byte boundaries.
        [[maybe_unused]] const bool vec_scales = ((nkb | k0) & 3) == 0 && (((uintptr_t)g.sa | (uintptr_t)g.sw) & 15u) == 0;
        const int q = warp & 3, h = (warp - 4) >> 2;
        float* stage = reinterpret_cast<float*>(sb + P::OFF_STAGE + (uint32_t)(warp - 4) * EpiPlan<SW>::WARP_BYTES);
        // This thread's two runs of SW columns of the tile.
        const int run0 = GATED ? h * SW : h * 2 * SW, run1 = GATED ? BN / 2 + h * SW : run0 + SW;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        Ring<NB> b;
        [[maybe_unused]] Ring<SG> rs;
        bool ok = true;
        [[maybe_unused]] bool joined = false;
        F2 acc[SW];
        for (int u = u0; ok && u < tiles; u += ustep) {
            const Tile t = tile_at<XR>(g, table, u);
            const int mine_rows = min(32, t.rows - 32 * q);      // this warp's rows
            const bool busy = mine_rows > 0;
            const int64_t col = (int64_t)t.nt * (GATED ? BN / 2 : BN) + run0;   // first column of z (gate)
            int ar = -1;
            if (lane < mine_rows) {
                ar = t.p0 + 32 * q + lane;
                if (g.rows) ar = __ldg(g.rows + ar);
                if (ar >= g.a_rows) ar = -1;
            }
            const bool row_in = ar >= 0, use = row_in && col < g.n;
            if constexpr (!GATED) {
                // The biases into the first level cache, where the epilogue finds them
                // (1999 rows, 32 experts, n 7168, k 2048: 120.5 -> 116 us).
                const int es = g.epi.bias_t == BQ_F32 ? 4 : 2, at = lane * (128 / es);
                if (busy && g.epi.bias && at < 2 * SW && col + at < g.n)
                    asm volatile("prefetch.global.L1 [%0];"
                                 :: "l"(reinterpret_cast<const char*>(g.epi.bias) + ((int64_t)t.e * g.n + col + at) * es));
            }
            const float* sap = g.sa + (int64_t)max(ar, 0) * nkb;
            const float* swp = g.sw + ((int64_t)t.e * g.nsw + (use ? col / 128 : 0)) * nkb;
            const int up = GATED ? (int)(g.n / 256) * nkb : 0;   // from a gate's scales to the other half's
#pragma unroll
            for (int j = 0; j < SW; ++j) acc[j] = 0ull;
            if constexpr (P::SCALES) {
                // (Not unrolled: the unrolled loop moved its sums about.)
#pragma unroll 1
                for (int kb = k0; kb < k1; ++kb) {
                    const int j = kb & 3;
                    if (j == 0 && !(ok = wait(P::B_SFULL + rs.slot, rs.round))) break;
                    const uint32_t at = base + P::OFF_SG + (uint32_t)rs.slot * SG_BYTES + 4u * (uint32_t)j;
                    const float sa = ld_shared1(at + 16u * (uint32_t)(32 * q + lane));
                    const F2 c0 = f2_bcast(__fmul_rn(sa, ld_shared1(at + 16u * (uint32_t)(128 + (GATED ? 0 : h)))));
                    const F2 c1 = GATED ? f2_bcast(__fmul_rn(sa, ld_shared1(at + 16u * 129u))) : c0;
                    if (!(ok = wait(P::B_TFULL + b.slot, b.round))) break;
                    tc_fence_after();
                    if (busy) {
                        const uint32_t tb = lane_base + (uint32_t)(b.slot * BN);
                        promote_runs<SW>(acc, tb + (uint32_t)run0, tb + (uint32_t)run1, c0, c1);
                    }
                    tc_fence_before();
                    __syncwarp();
                    const bool last = j == 3 || kb + 1 == k1;
                    if (lane == 0) {
                        bar_arrive(bar(P::B_TEMPTY + b.slot));
                        if (last) bar_arrive(bar(P::B_SEMPTY + rs.slot));
                    }
                    b.next();
                    if (last) rs.next();
                }
            } else {
                // The loads of the next group's scales are in flight while this one is added up.
                Scales4 ca = load_scales4(sap, k0, k1, use, vec_scales), cw = load_scales4(swp, k0, k1, use, vec_scales);
                Scales4 cv = load_scales4(swp + up, k0, k1, GATED && use, vec_scales);
                for (int kb0 = k0; kb0 < k1; kb0 += G) {
                    const Scales4 na = load_scales4(sap, kb0 + G, k1, use, vec_scales);
                    const Scales4 nw = load_scales4(swp, kb0 + G, k1, use, vec_scales);
                    const Scales4 nv = load_scales4(swp + up, kb0 + G, k1, GATED && use, vec_scales);
#pragma unroll
                    for (int j = 0; j < G; j += KS) {
                        if (!ok || kb0 + j >= k1) break;
                        if (!(ok = wait(P::B_TFULL + b.slot, b.round))) break;
                        tc_fence_after();
                        if (busy) {
#pragma unroll
                            for (int i = 0; i < KS; ++i) {
                                if (kb0 + j + i >= k1) break;
                                const F2 c0 = f2_bcast(__fmul_rn(ca.v[j + i], cw.v[j + i]));
                                const F2 c1 = GATED ? f2_bcast(__fmul_rn(ca.v[j + i], cv.v[j + i])) : c0;
                                const uint32_t tb = lane_base + (uint32_t)((b.slot * KS + i) * BN);
                                promote_runs<SW>(acc, tb + (uint32_t)run0, tb + (uint32_t)run1, c0, c1);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(bar(P::B_TEMPTY + b.slot));
                        b.next();
                    }
                    if (!ok) break;
                    ca = na;
                    cw = nw;
                    cv = nv;
                }
            }
            if (!ok) break;
            if constexpr (SPLIT) {
                // Every CTA's ring is empty after the first barrier; the others' sums
                // lie in the first's after the second.
                __syncwarp();
                cluster_sync();
                const uint32_t at = base + (uint32_t)(threadIdx.x - 128) * 16u;
                constexpr uint32_t STEP = 256 * 16, PART = STEP * (SW / 2);
                if (rank > 0 && lane < mine_rows) {              // rows that exist
                    const uint32_t dst = map_rank(at, 0u) + (uint32_t)(rank - 1) * PART;
#pragma unroll
                    for (int j = 0; j < SW / 2; ++j) st_cluster_pair(dst + (uint32_t)j * STEP, acc[2 * j], acc[2 * j + 1]);
                }
                cluster_sync();
                joined = true;
                if (rank > 0) break;
                for (int r = 0; r < parts - 1 && lane < mine_rows; ++r) {
#pragma unroll
                    for (int j = 0; j < SW / 2; ++j) {
                        F2 x, y;
                        ld_shared_pair(at + (uint32_t)r * PART + (uint32_t)j * STEP, x, y);
                        acc[2 * j] = f2_add(acc[2 * j], x);
                        acc[2 * j + 1] = f2_add(acc[2 * j + 1], y);
                    }
                }
            }
            if (busy)
                epi_tile<SW, GATED, FLAT>(g.epi, stage, lane, t.p0 + 32 * q, mine_rows, col, (int64_t)t.e * g.n + col, row_in, acc);
        }
        if constexpr (SPLIT) {
            if (!joined) {                                       // gave up: the others still wait for this CTA
                __syncwarp();
                cluster_sync();
                cluster_sync();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM);
    }
    // A role that gave up can leave TMA copies into the ring behind (every stage
    // loaded is consumed otherwise): keep the shared memory until they have landed.
    if (threadIdx.x == 0 && *abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// `split`: CTAs of a cluster that share a tile (SPLIT kernels).
template <int BN, bool GATED, int XR, bool SPLIT, bool FLAT>
cudaError_t launch_experts(const uint8_t* w, const ExpertArgs& ga, cudaStream_t st, int split = 1) {
    using P = PlanX<BN, XR>;
    static int ready[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    auto kern = k_fp8_experts<BN, GATED, XR, SPLIT, FLAT>;
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
    // Row tiles at most: one started per expert that can have a row, and the full ones.
    const int64_t most_tiles = g.offsets ? min(g.p, g.n_experts) + g.p / XR : (g.p + XR - 1) / XR;
    if (most_tiles * g.ntiles >= (1ll << 31)) return cudaErrorNotSupported;
    CUtensorMap ta, tw;
    if ((e = encode_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a, (uint64_t)g.k, (uint64_t)g.a_rows, (uint64_t)g.k, XK,
                        32)) != cudaSuccess)
        return e;
    if ((e = encode_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)g.k, (uint64_t)(g.n * g.n_experts), (uint64_t)g.k,
                        XK, BN / 2)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    const int64_t work = most_tiles * g.ntiles;
    cfg.gridDim = dim3((unsigned)(SPLIT ? work * split : min(work, (int64_t)sm_count())));
    cfg.blockDim = dim3(X_NT);
    cfg.dynamicSmemBytes = P::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, ta, tw, g);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Tile shapes, by whether rows are gathered, how many an expert has on average and
// how many tiles there are. Times on B200 in us, launches of a CUDA graph call
// after call; 32 experts, n 4096 k 7168 gated ("up") or n 7168 k 2048 ("down"):
//   rows gathered, up to 16 an expert: tiles of 32 rows x 128 columns (up, 64 rows:
//   151 against 207 with 128 rows and 158 with 256 columns; 256: 161, 208, 163; 512:
//   174, 209, 167; one expert, 128 rows: 21, 35, 34);
//   rows gathered, more of them: 256 columns (up, 768 rows: 173 against 190 with 32
//   rows and 210 with 128 x 128; 16384: 597 against 952; 8 experts of 2048 x 2048, 512
//   rows: 16.2 against 15.8). The 128 columns' two k-blocks a stage wait for their
//   gather;
//   rows in place: 256 columns from 16 rows an expert on (down, 512 rows: 103 against
//   110 with 128 columns, 4096: 137 against 149; up, 512: 166 either way, 4096: 212
//   against 234), with tiles enough to fill the card twice (8 experts of 2048 x 1024,
//   512 rows: 13.3 against 10.3), else 128 (down, 64 rows: 93 against 97, and 100 with
//   tiles of 32 rows; up, 64: 150, 154, 150).
//   Widths that are no multiple of 8 stay on 128 columns, whose promotion leaves
//   room for their epilogue.
template <bool GATED>
cudaError_t launch_by_shape(const uint8_t* w, const ExpertArgs& g, cudaStream_t st) {
    const int64_t p = g.p, e = g.n_experts;
    const bool few = g.rows && p <= 16 * e;
    if constexpr (!GATED) {
        if (g.n % 8 != 0)
            return few ? launch_experts<128, false, 32, false, true>(w, g, st) : launch_experts<128, false, 128, false, true>(w, g, st);
    }
    if (few) return launch_experts<128, GATED, 32, false, false>(w, g, st);
    const int64_t row_tiles = max(p / XM, min(p, e));            // about
    if (g.rows || (p >= 16 * e && row_tiles * ((g.n + 255) / 256) >= 2 * sm_count()))
        return launch_experts<256, GATED, 128, false, false>(w, g, st);
    return launch_experts<128, GATED, 128, false, false>(w, g, st);
}

}  // namespace

cudaError_t experts_error_take(unsigned int* flag) { return take_gemm_error(flag); }

static ExpertArgs make_args(const uint8_t* a, const float* sa, int64_t a_rows, int64_t k, const int32_t* rows,
                            const int32_t* offsets, int n_experts, int64_t p, const float* sw, int64_t n) {
    ExpertArgs g = {};
    g.a_rows = (int)a_rows; g.k = k; g.n = n; g.p = (int)p;
    g.nkb = (int)(k / XK);
    g.n_experts = n_experts;
    g.per_entry = (n_experts + X_TABLE - 1) / X_TABLE;
    g.nsw = (int)((n + 127) / 128);
    g.a = a; g.rows = rows; g.offsets = offsets; g.sa = sa; g.sw = sw;
    return g;
}

cudaError_t fp8_experts(const uint8_t* a, const float* sa, int64_t a_rows, int64_t k, const int32_t* rows,
                        const int32_t* offsets, int n_experts, int64_t p, const uint8_t* w, const float* sw, int64_t n,
                        const void* bias, int bias_t, int act, int gated, void* c, int c_t, cudaStream_t st) {
    ExpertArgs g = make_args(a, sa, a_rows, k, rows, offsets, n_experts, p, sw, n);
    g.epi = make_epi(n, gated ? n / 2 : n, bias, bias_t, act, nullptr, c, c_t, nullptr);
    return gated ? launch_by_shape<true>(w, g, st) : launch_by_shape<false>(w, g, st);
}

// The dense product: one expert with every row. Tiles of 256 columns once there
// are more of 128 x 128 than SMs; up to half as many of those as SMs, two or four
// CTAs share a tile's k-blocks.
cudaError_t fp8_dense(const uint8_t* a, const float* sa, int64_t m, int64_t k, const uint8_t* w, const float* sw, int64_t n,
                      const void* bias, int bias_t, int act, const void* residual, void* c, int c_t, void* pre, cudaStream_t st) {
    ExpertArgs g = make_args(a, sa, m, k, nullptr, nullptr, 1, m, sw, n);
    g.epi = make_epi(n, n, bias, bias_t, act, residual, c, c_t, pre);
    const int64_t tiles = ((m + XM - 1) / XM) * ((n + 127) / 128), sms = sm_count();
    const bool flat = n % 8 != 0;
    if (tiles > sms)
        return flat ? launch_experts<128, false, 128, false, true>(w, g, st) : launch_experts<256, false, 128, false, false>(w, g, st);
    const int split = 4 * tiles <= sms && g.nkb >= 8 ? 4 : 2 * tiles <= sms && g.nkb >= 4 ? 2 : 1;
    if (split > 1)
        return flat ? launch_experts<128, false, 128, true, true>(w, g, st, split)
                    : launch_experts<128, false, 128, true, false>(w, g, st, split);
    return flat ? launch_experts<128, false, 128, false, true>(w, g, st) : launch_experts<128, false, 128, false, false>(w, g, st);
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
    if (rows && a_rows * (k / 16) >= (1ll << 32)) return BQ_ERR_INVALID_ARG;
    if (c_rows == 0 || n == 0) return BQ_OK;
    if (!offsets || !w_e4m3 || !w_scale || !c) return BQ_ERR_INVALID_ARG;
    if (!a_e4m3 || !a_scale || a_rows == 0) return BQ_ERR_INVALID_ARG;
    if (((uintptr_t)a_e4m3 & 15u) || ((uintptr_t)w_e4m3 & 15u) || ((uintptr_t)c & 15u)) return BQ_ERR_MISALIGNED;
    if (((uintptr_t)a_scale & 3u) || ((uintptr_t)w_scale & 3u) || ((uintptr_t)rows & 3u) || ((uintptr_t)offsets & 3u) ||
        ((uintptr_t)bias & (bias_dtype == BQ_F32 ? 3u : 1u)))
        return BQ_ERR_MISALIGNED;
    const cudaError_t e = bq::fp8_experts(a_e4m3, a_scale, a_rows, k, rows, offsets, n_experts, c_rows, w_e4m3, w_scale, n,
                                          bias, bias_dtype, act, gated != 0, c, c_dtype, (cudaStream_t)stream);
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
    const cudaError_t e = bq::fp8_dense(a_e4m3, a_scale, m, k, w_e4m3, w_scale, n, bias, bias_dtype, act, residual, c, c_dtype, pre,
                                        (cudaStream_t)stream);
    if (e == cudaErrorNotSupported) return BQ_ERR_UNSUPPORTED;
    return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
}
