// Shared by the block-FP8 products: mbarriers with bounded waits, TMA loads,
// tcgen05 (TMEM, MMA) and tensor maps. Everything has internal linkage: each
// translation unit has its own g_gemm_error.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "bq_device.cuh"

namespace bq {
namespace {

// Set by a bounded wait of this translation unit's kernels that gave up.
__device__ unsigned int g_gemm_error;

// ------------------------------------------------------------ PTX helpers
__device__ __forceinline__ uint32_t sm_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(1000u) : "memory");
    return ok != 0;
}
// The same wait with cluster-scope acquire, for barriers other CTAs of the
// cluster arrive on (their stores to this CTA become visible).
__device__ __forceinline__ bool bar_try_wait_cl(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(1000u) : "memory");
    return ok != 0;
}
// Shared-memory address of the same location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void bar_arrive_remote(uint32_t cl_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cl_addr) : "memory");
}
__device__ __forceinline__ void bar_arrive_remote_relaxed(uint32_t cl_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cl_addr) : "memory");
}
// One arrival on the barrier at `bar` in every CTA of the cluster, lane d of
// the (converged) warp arriving on CTA d, so the arrivals travel in
// parallel. RELEASE: the warp's earlier stores (ordered before by the
// __syncwarp the caller ran) are visible in the cluster before the arrival
// counts; otherwise the arrival only orders what the barrier guards against
// overwriting (reads that have completed).
template <int CL, bool RELEASE>
__device__ __forceinline__ void arrive_all_ranks(uint32_t bar, int lane) {
    if (lane < CL) {
        const uint32_t a = map_rank(bar, (uint32_t)lane);
        if (RELEASE) bar_arrive_remote(a);
        else bar_arrive_remote_relaxed(a);
    }
}
__device__ __forceinline__ void st_cluster_u32(uint32_t cl_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(cl_addr), "r"(v) : "memory");
}
// Bulk copy of `bytes` from this CTA's shared memory to a cluster address
// (another CTA's shared memory); completes transaction bytes on the mbarrier
// at the cluster address `cl_bar` (in the destination CTA).
__device__ __forceinline__ void bulk_to_rank(uint32_t cl_dst, uint32_t src, uint32_t bytes, uint32_t cl_bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(cl_dst), "r"(src), "r"(bytes), "r"(cl_bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Bounded wait (each try suspends for at most about a microsecond); gives up
// early once another role (of any CTA of the cluster) has set the abort
// flag. On giving up by itself it sets the flag in every CTA of the cluster
// and the device error.
// Non-blocking probe of a phase (no suspension): the common case of a
// barrier that has already completed costs one instruction.
template <bool CLUSTER_SCOPE>
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (CLUSTER_SCOPE)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
template <int CL, bool CLUSTER_SCOPE>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         uint32_t abort_addr) {
    if (bar_test<CLUSTER_SCOPE>(bar, parity)) return true;
    for (uint32_t i = 0; i < (1u << 21); ++i) {
        if (CLUSTER_SCOPE ? bar_try_wait_cl(bar, parity) : bar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 15u && *abort_flag) return false;
    }
    if (CL == 1) *abort_flag = 1u;
    else
        for (uint32_t d = 0; d < (uint32_t)CL; ++d) st_cluster_u32(map_rank(abort_addr, d), 1u);
    atomicOr(&g_gemm_error, 1u);
    return false;
}
// Wait used while draining after an abort: bounded, ignores the flag.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 21); ++i)
        if (bar_try_wait(bar, parity)) return;
    atomicOr(&g_gemm_error, 1u);
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"((uint64_t)tm), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* tm) {
    asm volatile("prefetch.tensormap [%0];" :: "l"((uint64_t)tm) : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void set_max_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

// tcgen05 (5th-generation tensor core, accumulators in TMEM).
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, both K-major E4M3, f32 D.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// The mbarrier completes (one arrival) when every tcgen05 operation this
// thread issued before has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
// 32 consecutive f32 columns of this thread's TMEM lane (raw bits). The
// registers hold the values only after tmem_ld_wait and tmem_regs_ready.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// Placed after tcgen05.wait::ld: no use of the loaded registers is moved
// above it (the compiler sees them written here).
__device__ __forceinline__ void tmem_regs_ready(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of a K-major operand with 128-byte rows in
// the 128-byte swizzle (8-row atoms of 1024 bytes): start address, leading
// byte offset 16 (unused by this layout), stride byte offset 1024 between
// 8-row groups, descriptor version 1, layout SWIZZLE_128B.
__device__ __forceinline__ uint64_t desc_k_sw128(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The block scales of four k-blocks from kb on, of [.., kend); zeros past the end
// and unless `use`. One 16-byte load where `vec` says that rows of scales start
// on 16-byte boundaries. Promotion loops load a group ahead: next to a full
// stream of operand tiles a load takes longer than two k-blocks.
struct Scales4 {
    float v[4];
};
__device__ __forceinline__ Scales4 load_scales4(const float* row, int kb, int kend, bool use, bool vec) {
    Scales4 s;
    if (use && vec && kb + 4 <= kend) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(row + kb));
        s.v[0] = f.x; s.v[1] = f.y; s.v[2] = f.z; s.v[3] = f.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s.v[j] = use && kb + j < kend ? __ldg(row + kb + j) : 0.0f;
    }
    return s;
}

// Position in a ring of N slots: the slot, and the parity of its current round.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) { slot = 0; round ^= 1u; }
    }
};
// 16 or 4 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
// This thread's arrival on the barrier, when its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Block scales through shared memory: a ring of groups of four k-blocks, each
// with 16 bytes per row of the tile (128) and per set of weight scales (two).
// A promotion loop whose registers are full of sums must not have loads from
// global memory in flight: the loop that fetched its own scales ran at 980 to
// 1650 clocks a k-block, depending on how the compiler placed the loads.
constexpr int SG = 4;                                  // groups of the ring
constexpr uint32_t SG_BYTES = (128 + 2) * 16;
// Four scales from k-block kb of a row of them; those past kend are left out.
__device__ __forceinline__ void copy_scales4(uint32_t dst, const float* row, int kb, int kend, bool vec) {
    if (vec && kb + 4 <= kend) {
        copy16(dst, row + kb);
    } else {
        for (int j = 0; j < 4 && kb + j < kend; ++j) copy4(dst + 4u * (uint32_t)j, row + kb + j);
    }
}
__device__ __forceinline__ float ld_shared1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

[[maybe_unused]] cudaError_t encode_map(CUtensorMap* tm, CUtensorMapDataType dt, const void* p, uint64_t inner,
                       uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return (PFN_cuTensorMapEncodeTiled_v12000)f;
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t gdim[2] = {inner, outer};
    const cuuint64_t gstride[1] = {row_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estride[2] = {1, 1};
    const CUresult r = encode(tm, dt, 2, const_cast<void*>(p), gdim, gstride, box, estride,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Reads and clears this translation unit's flag.
[[maybe_unused]] cudaError_t take_gemm_error(unsigned int* flag) {
    unsigned int v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_gemm_error, &z, sizeof(z));
    *flag = v;
    return e;
}

}  // namespace
}  // namespace bq
