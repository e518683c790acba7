// Gradient of a product's epilogue c = act(pre) + residual, pre = A W^T + bias:
//   dz = dc * act'(pre) (the gradient of the product, in dc's dtype),
//   dbias[j] = sum over rows of dc * act'(pre), from the unrounded f32 terms.
// (The gradient of the residual is dc itself.) Bound by memory: dc and pre are
// read once and dz is written once. The sum over the rows goes over a fixed
// split of the rows and is joined in a fixed order by a second kernel, so it is
// the same every time.
#include "bq.h"
#include "bq_act.cuh"
#include "bq_cols.cuh"
#include "bq_device.cuh"
#include "bq_internal.h"

namespace bq {
namespace {

constexpr int EB_COLS = 32, EB_ROWS = 8;     // threads of a CTA along a row and down the rows

struct EpiBwdArgs {
    const void *dy, *pre;
    int64_t m, n;
    int64_t rows_per;      // rows of a CTA
    void* dz;
    float* partial;        // [splits, n]
};

// The split of the rows depends on the sizes alone (not on the device).
int64_t epi_splits(int64_t m, int64_t n) {
    const int64_t strips = (n + 255) / 256;
    int64_t s = (1024 + strips - 1) / strips;          // about 1024 CTAs in all
    const int64_t most = (m + 31) / 32;                // at least 32 rows each
    if (s > most) s = most;
    return s < 1 ? 1 : s;
}

// V columns of a thread: 16 bytes where rows start on them, else two or one, with
// as many more rows in flight.
template <class T, int ACT, int V>
__global__ void __launch_bounds__(EB_COLS* EB_ROWS) k_epi_bwd(const EpiBwdArgs a) {
    __shared__ float sum[EB_ROWS][EB_COLS * V + 1];
    constexpr int R = V > 2 ? 2 : 8;             // (16 bytes: four rows leave fewer CTAs, 56 against 53 us at
                                                 // 4096 x 11008 bf16, gelu_tanh; one: 72)
    const int cx = threadIdx.x % EB_COLS, ry = threadIdx.x / EB_COLS;
    const int64_t col = ((int64_t)blockIdx.x * EB_COLS + cx) * V;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows_per, r1 = min(a.m, r0 + a.rows_per);
    const T* dy = reinterpret_cast<const T*>(a.dy);
    const T* pre = reinterpret_cast<const T*>(a.pre);
    T* dz = reinterpret_cast<T*>(a.dz);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (col < a.n) {
        for (int64_t r = r0 + ry; r < r1; r += R * EB_ROWS) {
            // dz may be dy itself: ordinary loads, before the stores below.
            Cols<T, V> gv[R], zv[R];
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (r + q * EB_ROWS >= r1) break;
                const int64_t at = (r + q * EB_ROWS) * a.n + col;
                zv[q].load(pre + at);
                gv[q].load(dy + at);
            }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (r + q * EB_ROWS >= r1) break;
                float g[V], z[V];
                gv[q].get(g);
                zv[q].get(z);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[i] *= act_slope<ACT>(z[i]);
                    acc[i] += g[i];
                }
                gv[q].set(g);
                gv[q].store(dz + (r + q * EB_ROWS) * a.n + col);
            }
        }
    }
    pdl_trigger();
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < V; ++i) sum[ry][cx * V + i] = acc[i];
    __syncthreads();
    for (int c = threadIdx.x; c < EB_COLS * V; c += EB_COLS * EB_ROWS) {
        const int64_t j = (int64_t)blockIdx.x * EB_COLS * V + c;
        if (j < a.n) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < EB_ROWS; ++r) s += sum[r][c];
            a.partial[(int64_t)blockIdx.y * a.n + j] = s;
        }
    }
}

__global__ void __launch_bounds__(128) k_epi_dbias(const float* partial, int64_t splits, int64_t n, float* dbias) {
    pdl_wait();
    const int64_t j = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (j >= n) return;
    float s = 0.0f;
#pragma unroll 4
    for (int64_t i = 0; i < splits; ++i) s += partial[i * n + j];
    dbias[j] = s;
}

template <class T, int ACT>
cudaError_t launch_epi_bwd(EpiBwdArgs a, float* dbias, cudaStream_t st) {
    const int64_t splits = epi_splits(a.m, a.n);
    a.rows_per = (a.m + splits - 1) / splits;
    constexpr int VEC = Traits<T>::VEC;
    const uintptr_t starts = (uintptr_t)a.dy | (uintptr_t)a.pre | (uintptr_t)a.dz;
    const int v = a.n % VEC == 0 && (starts & 15u) == 0 ? VEC : a.n % 2 == 0 && starts % (2 * sizeof(T)) == 0 ? 2 : 1;
    const int64_t wide = EB_COLS * v;
    const dim3 grid((unsigned)((a.n + wide - 1) / wide), (unsigned)splits);
    if (v == VEC) k_epi_bwd<T, ACT, VEC><<<grid, EB_COLS * EB_ROWS, 0, st>>>(a);
    else if (v == 2) k_epi_bwd<T, ACT, 2><<<grid, EB_COLS * EB_ROWS, 0, st>>>(a);
    else k_epi_bwd<T, ACT, 1><<<grid, EB_COLS * EB_ROWS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dbias) return e;
    return launch_pdl(k_epi_dbias, (unsigned)((a.n + 127) / 128), 128, 0, st, (const float*)a.partial, splits, a.n, dbias);
}
template <class T>
cudaError_t by_act(const EpiBwdArgs& a, bq_act act, float* dbias, cudaStream_t st) {
    switch (act) {
        case BQ_ACT_NONE: return launch_epi_bwd<T, BQ_ACT_NONE>(a, dbias, st);
        case BQ_ACT_RELU: return launch_epi_bwd<T, BQ_ACT_RELU>(a, dbias, st);
        case BQ_ACT_GELU: return launch_epi_bwd<T, BQ_ACT_GELU>(a, dbias, st);
        case BQ_ACT_GELU_TANH: return launch_epi_bwd<T, BQ_ACT_GELU_TANH>(a, dbias, st);
        default: return launch_epi_bwd<T, BQ_ACT_SILU>(a, dbias, st);
    }
}

}  // namespace
}  // namespace bq

using namespace bq;

extern "C" size_t bq_gemm_epilogue_backward_workspace_size(int64_t m, int64_t n) {
    if (m <= 0 || n <= 0 || m >= (1ll << 31) || n >= (1ll << 31)) return 0;
    return (size_t)epi_splits(m, n) * (size_t)n * sizeof(float);
}

extern "C" bq_status bq_gemm_epilogue_backward(const void* dy, const void* pre, bq_dtype dtype, int64_t m, int64_t n,
                                               bq_act act, void* dz, float* dbias, void* ws, size_t ws_bytes, void* stream) {
    if (dtype != BQ_F32 && dtype != BQ_F16 && dtype != BQ_BF16) return BQ_ERR_UNSUPPORTED;
    if (act < BQ_ACT_NONE || act > BQ_ACT_SILU) return BQ_ERR_UNSUPPORTED;
    if (m < 0 || n < 0 || m >= (1ll << 31) || n >= (1ll << 31)) return BQ_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (n == 0) return BQ_OK;
    if (((uintptr_t)dbias & 3u) || ((uintptr_t)ws & 3u)) return BQ_ERR_MISALIGNED;
    if (m == 0) {                                   // a sum over no rows
        if (!dbias) return BQ_OK;
        return cudaMemsetAsync(dbias, 0, (size_t)n * sizeof(float), st) == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
    }
    if (!dy || !pre || !dz) return BQ_ERR_INVALID_ARG;
    const uintptr_t mask = dtype == BQ_F32 ? 3u : 1u;
    if (((uintptr_t)dy & mask) || ((uintptr_t)pre & mask) || ((uintptr_t)dz & mask)) return BQ_ERR_MISALIGNED;
    if (dbias && (!ws || ws_bytes < bq_gemm_epilogue_backward_workspace_size(m, n))) return BQ_ERR_INVALID_ARG;
    EpiBwdArgs a{dy, pre, m, n, 0, dz, dbias ? (float*)ws : nullptr};
    const cudaError_t e = dtype == BQ_F32 ? by_act<float>(a, act, dbias, st)
                          : dtype == BQ_F16 ? by_act<__half>(a, act, dbias, st)
                                            : by_act<__nv_bfloat16>(a, act, dbias, st);
    return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
}
