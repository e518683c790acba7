// Expert layers: routing (choice of experts and their weights) with its
// gradient, the expert order of the routed rows, and the sum of the experts'
// rows back into tokens with its gradient.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "bq.h"
#include "bq_device.cuh"
#include "bq_internal.h"

namespace bq {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- routing
// One warp per token. Lane l holds the C consecutive experts from l * C, so
// that the lowest lane with the largest value holds the lowest index of it.
// The order of the choice values decides which experts a token gets, so they
// are computed in f64, where two different logits practically never give
// equal values.
struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t tokens;
    int experts, top_k, n_groups, top_groups, group_top, sigmoid, renorm, vec;
    float scale;
    int32_t* ids;
    float* weights;
};

// The lane's C logits of a row as f32; experts past the end count as -inf.
template <class T, int C>
__device__ __forceinline__ void load_logits(const T* row, int lane, int experts, int vec, float (&x)[C]) {
    const int e0 = lane * C;
    if constexpr (C * sizeof(T) >= 16) {
        if (vec) {
            constexpr int VEC = Traits<T>::VEC;
#pragma unroll
            for (int i = 0; i < C; i += VEC) {
                if (e0 + i < experts) {
                    float v[VEC];
                    load_vec<T>(ld16_nc(row + e0 + i), v);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[i + j] = v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[i + j] = -CUDART_INF_F;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = e0 + i < experts ? ld1<T>(row + e0 + i) : -CUDART_INF_F;
}

template <class T, int C>
__global__ void __launch_bounds__(128) k_moe_route(const RouteArgs a) {
    extern __shared__ double route_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double* vs = route_smem + (size_t)warp * a.experts;
    const int gsize = a.experts / a.n_groups;
    for (int64_t t = (int64_t)blockIdx.x * 4 + warp; t < a.tokens; t += (int64_t)gridDim.x * 4) {
        float x[C];
        load_logits<T, C>(reinterpret_cast<const T*>(a.logits) + t * a.experts, lane, a.experts, a.vec, x);
        bool bad = false;
        double top = -CUDART_INF;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (x[i] != x[i]) { bad = true; x[i] = -CUDART_INF_F; }
            top = fmax(top, (double)x[i]);
        }
        bad = __any_sync(FULL, bad);
        double s[C], v[C];
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < C; ++i) s[i] = 1.0 / (1.0 + exp(-(double)x[i]));
        } else {
            top = warp_max(top);
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                // Equal to the largest, -inf and +inf among them: exp(0).
                s[i] = lane * C + i < a.experts ? exp((double)x[i] == top ? 0.0 : (double)x[i] - top) : 0.0;
                sum += s[i];
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
#pragma unroll
            for (int i = 0; i < C; ++i) s[i] /= sum;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = lane * C + i;
            v[i] = a.bias && e < a.experts ? s[i] + (double)__ldg(a.bias + e) : (double)x[i];
            if (!(x[i] > -CUDART_INF_F) || v[i] != v[i]) v[i] = -CUDART_INF;
        }
        if (a.n_groups > 1) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (lane * C + i < a.experts) vs[lane * C + i] = v[i];
            __syncwarp();
            double gv = -CUDART_INF;
            if (lane < a.n_groups) {
                double b1 = -CUDART_INF, b2 = -CUDART_INF;
                for (int j = 0; j < gsize; ++j) {
                    const double u = vs[lane * gsize + j];
                    if (u > b1) { b2 = b1; b1 = u; } else if (u > b2) b2 = u;
                }
                gv = b1;
                if (a.group_top == 2 && b2 > -CUDART_INF) gv += b2;
            }
            int ahead = 0;
            for (int j = 0; j < a.n_groups; ++j) {
                const double o = __shfl_sync(FULL, gv, j);
                ahead += (o > gv || (o == gv && j < lane)) ? 1 : 0;
            }
            const unsigned kept = __ballot_sync(FULL, lane < a.n_groups && ahead < a.top_groups);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int e = lane * C + i;
                if (e < a.experts && !((kept >> (e / gsize)) & 1u)) v[i] = -CUDART_INF;
            }
        }
        int my_id = -1;
        double my_s = 0.0;
        for (int it = 0; it < a.top_k; ++it) {
            double best = -CUDART_INF, bs = 0.0;
            int bi = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (v[i] > best) { best = v[i]; bs = s[i]; bi = lane * C + i; }
            for (int o = 16; o > 0; o >>= 1) {
                const double ob = __shfl_xor_sync(FULL, best, o), os = __shfl_xor_sync(FULL, bs, o);
                const int oi = __shfl_xor_sync(FULL, bi, o);
                if (ob > best || (ob == best && oi < bi)) { best = ob; bs = os; bi = oi; }
            }
            if (!(best > -CUDART_INF)) break;
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (lane * C + i == bi) v[i] = -CUDART_INF;
            if (lane == it) { my_id = bi; my_s = bs; }
        }
        double w = my_s;
        if (a.renorm) {
            double sum = w;
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
            w = sum > 0.0 ? w / sum : 0.0;
        }
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = my_id;
            a.weights[t * a.top_k + lane] = bad ? CUDART_NAN_F : (float)(w * (double)a.scale);
        }
    }
}

// Gradient of the weights with respect to the logits. With g = dL/dw, s the
// scores of the chosen experts, D their sum (renormalised) or 1:
//   gs_i = scale (g_i - [renorm] sum_j g_j s_j / D) / D,
//   sigmoid:              dl[id_i] += gs_i s_i (1 - s_i), else 0;
//   softmax, renorm:      dl[id_i] += gs_i s_i (the sum over experts is 0);
//   softmax as it is:     dl_j = p_j (gs_j - sum_i gs_i s_i) for every expert.
// Renormalised scores depend on each other's ratios alone, which are taken
// relative to the largest chosen one, so that small scores do not vanish.
struct RouteBwdArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    int64_t tokens;
    int experts, top_k, sigmoid, renorm, vec;
    float scale;
    void* dlogits;
};

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <class T, int C>
__global__ void __launch_bounds__(128) k_moe_route_bwd(const RouteBwdArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = (int64_t)blockIdx.x * 4 + warp; t < a.tokens; t += (int64_t)gridDim.x * 4) {
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.experts;
        int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
        if (id >= a.experts) id = -1;
        const float g = id >= 0 ? a.dweights[t * a.top_k + lane] : 0.0f;
        const float l = id >= 0 ? ld1<T>(row + id) : -CUDART_INF_F;
        const bool dense = !a.sigmoid && !a.renorm;
        float p[C], full[C];
        float contrib, shift = 0.0f;
        if (dense) {
            load_logits<T, C>(row, lane, a.experts, a.vec, p);
            float top = -CUDART_INF_F;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < C; ++i) { bad |= p[i] != p[i]; top = fmaxf(top, p[i]); }
            top = warp_max(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                p[i] = lane * C + i < a.experts ? expf(p[i] == top ? 0.0f : p[i] - top) : 0.0f;
                sum += p[i];
            }
            sum = warp_sum(sum);
            if (__any_sync(FULL, bad)) sum = CUDART_NAN_F;
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < C; ++i) p[i] *= inv;
            const float s = id >= 0 ? expf(l == top ? 0.0f : l - top) * inv : 0.0f;
            contrib = a.scale * g;
            shift = warp_sum(contrib * s);
        } else {
            // Scores up to a common factor, and s (1 - s) / s of the sigmoid.
            const float low = a.sigmoid ? fminf(l, 0.0f) : l;
            float s = 0.0f, tail = 1.0f;
            if (a.renorm) {
                const float top = warp_max(low);
                s = id >= 0 ? expf(low == top ? 0.0f : low - top) : 0.0f;
            } else {
                s = id >= 0 ? expf(low) : 0.0f;
            }
            if (a.sigmoid) {
                const float u = expf(-fabsf(l));           // s = exp(min(l, 0)) / (1 + u)
                s = s / (1.0f + u);
                tail = (l >= 0.0f ? u : 1.0f) / (1.0f + u);   // 1 - s
            }
            float gs;
            if (a.renorm) {
                const float d = warp_sum(s), gm = warp_sum(g * s);
                s = d > 0.0f ? s / d : 0.0f;
                gs = a.scale * (g - (d > 0.0f ? gm / d : 0.0f));
            } else {
                gs = a.scale * g;
            }
            contrib = id >= 0 ? gs * s * tail : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) full[i] = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int at = __shfl_sync(FULL, id, j);
            const float c = __shfl_sync(FULL, contrib, j);
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (lane * C + i == at) full[i] += c;
        }
        if (dense) {
#pragma unroll
            for (int i = 0; i < C; ++i) full[i] = p[i] * (full[i] - shift);
        }
        T* out = reinterpret_cast<T*>(a.dlogits) + t * a.experts + lane * C;
        bool done = false;
        if constexpr (C * sizeof(T) >= 16) {
            if (a.vec) {
                constexpr int VEC = Traits<T>::VEC;
#pragma unroll
                for (int i = 0; i < C; i += VEC)
                    if (lane * C + i < a.experts) {
                        float o[VEC];
#pragma unroll
                        for (int j = 0; j < VEC; ++j) o[j] = full[i + j];
                        st16(out + i, pack_vec<T>(o));
                    }
                done = true;
            }
        }
        if (!done) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (lane * C + i < a.experts) out[i] = to_out<T>(full[i]);
        }
    }
}

// Experts per lane: a power of two, so that every loop over them unrolls.
template <class T, template <class, int> class L, class A>
cudaError_t by_width(const A& a, cudaStream_t st) {
    const int c = (a.experts + 31) / 32;
    if (c <= 1) return L<T, 1>::go(a, st);
    if (c <= 2) return L<T, 2>::go(a, st);
    if (c <= 4) return L<T, 4>::go(a, st);
    if (c <= 8) return L<T, 8>::go(a, st);
    if (c <= 16) return L<T, 16>::go(a, st);
    return L<T, 32>::go(a, st);
}
unsigned warp_grid(int64_t tokens, int per_sm) {
    const int64_t need = (tokens + 3) / 4, most = (int64_t)sm_count() * per_sm;
    return (unsigned)(need < most ? need : most);
}
template <class T, int C>
struct RouteLaunch {
    static cudaError_t go(RouteArgs a, cudaStream_t st) {
        constexpr int VEC = Traits<T>::VEC;
        a.vec = a.experts % VEC == 0 && ((uintptr_t)a.logits & 15u) == 0;
        const size_t smem = a.n_groups > 1 ? 4 * sizeof(double) * (size_t)a.experts : 0;
        k_moe_route<T, C><<<warp_grid(a.tokens, 16), 128, smem, st>>>(a);
        return cudaGetLastError();
    }
};
template <class T, int C>
struct RouteBwdLaunch {
    static cudaError_t go(RouteBwdArgs a, cudaStream_t st) {
        constexpr int VEC = Traits<T>::VEC;
        a.vec = a.experts % VEC == 0 && ((uintptr_t)a.logits & 15u) == 0 && ((uintptr_t)a.dlogits & 15u) == 0;
        k_moe_route_bwd<T, C><<<warp_grid(a.tokens, 16), 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

// ---------------------------------------------------------------- expert order
// A stable counting sort of the pairs (token, slot) by expert in one launch:
// the eight CTAs of a cluster take consecutive runs of the pairs, each warp a
// consecutive run of its CTA's. Pass one counts per warp and expert; prefix
// sums over the warps, over the CTAs (through distributed shared memory) and
// over the experts give every (warp, expert) its first position; pass two
// hands out the positions in the order of the pairs. No atomics: the order
// is the same every time.
constexpr int GROUP_CTAS = 8, GROUP_NT = 1024, GROUP_WARPS = GROUP_NT / 32;

struct GroupArgs {
    const int32_t* ids;
    int64_t pairs;
    int top_k, first, n;
    int32_t *offsets, *rows, *pos;
};

__global__ void __launch_bounds__(GROUP_NT, 1) k_moe_group(const GroupArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ int32_t group_smem[];
    int32_t* table = group_smem;                        // [GROUP_WARPS][n]
    int32_t* mine = table + (size_t)GROUP_WARPS * a.n;  // [n] this CTA's counts
    int32_t* base = mine + a.n;                         // [n] first position of this CTA's run
    __shared__ int32_t warp_tot[GROUP_WARPS];
    __shared__ int32_t total_all;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Pairs of a warp: a multiple of 32, consecutive over (CTA, warp).
    const int64_t per = ((a.pairs + (int64_t)ctas * GROUP_NT - 1) / ((int64_t)ctas * GROUP_NT)) * 32;
    const int64_t lo = min(a.pairs, ((int64_t)rank * GROUP_WARPS + warp) * per), hi = min(a.pairs, lo + per);
    int32_t* tw = table + (size_t)warp * a.n;
    for (int i = lane; i < a.n; i += 32) tw[i] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        int e = i < hi ? a.ids[i] : -1;
        e = e >= a.first && e - a.first < a.n ? e - a.first : -1;
        const unsigned same = __match_any_sync(FULL, e);
        if (e >= 0 && lane == __ffs(same) - 1) tw[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < a.n; e += GROUP_NT) {
        int run = 0;
        for (int w = 0; w < GROUP_WARPS; ++w) {
            const int c = table[(size_t)w * a.n + e];
            table[(size_t)w * a.n + e] = run;
            run += c;
        }
        mine[e] = run;
    }
    cl.sync();
    // Totals of every expert over the cluster, and of the CTAs before this one.
    int total = 0, before = 0;
    if (tid < a.n) {
        for (int r = 0; r < ctas; ++r) {
            const int c = cl.map_shared_rank(mine, r)[tid];
            before += r < rank ? c : 0;
            total += c;
        }
    }
    int incl = total;
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = warp_tot[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, v, o);
            if (lane >= o) v += u;
        }
        warp_tot[lane] = v;
        if (lane == 31) total_all = v;
    }
    __syncthreads();
    const int excl = incl - total + (warp ? warp_tot[warp - 1] : 0);
    if (tid < a.n) {
        base[tid] = excl + before;
        if (rank == 0) {
            a.offsets[tid] = excl;
            if (tid == a.n - 1) a.offsets[a.n] = excl + total;
        }
    }
    cl.sync();                     // no CTA leaves while another reads its counts
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        int e = i < hi ? a.ids[i] : -1;
        e = e >= a.first && e - a.first < a.n ? e - a.first : -1;
        const unsigned same = __match_any_sync(FULL, e);
        int p = -1;
        if (e >= 0) {
            p = base[e] + tw[e] + __popc(same & ((1u << lane) - 1u));
            a.rows[p] = (int32_t)(i / a.top_k);
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) tw[e] += __popc(same);
        __syncwarp();
        if (i < hi) a.pos[i] = p;
    }
    // Rows behind the last expert's.
    for (int64_t i = total_all + (int64_t)rank * GROUP_NT + tid; i < a.pairs; i += (int64_t)ctas * GROUP_NT)
        a.rows[i] = -1;
}

cudaError_t launch_group(const GroupArgs& a, cudaStream_t st) {
    const size_t smem = ((size_t)GROUP_WARPS + 2) * a.n * sizeof(int32_t);
    static int ready[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        const cudaError_t e = cudaFuncSetAttribute(k_moe_group, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (GROUP_WARPS + 2) * 1024 * (int)sizeof(int32_t));
        if (e != cudaSuccess) return e;
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const unsigned ctas = a.pairs > 4 * GROUP_NT ? GROUP_CTAS : 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(GROUP_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_moe_group, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------- combine
// out[t] = residual[t] + sum over slots of weights[t, j] * y[pos[t, j]], in f32
// and rounded once. One pass over memory: a thread owns one 16-byte vector of
// out and loads that vector of every slot's row before it adds them up.
struct CombineArgs {
    const void* y;
    const int32_t* pos;
    const float* weights;
    const void* residual;
    void* out;
    int64_t tokens, y_rows, hidden, per_row;   // per_row: vectors of a row
    int top_k;
};

template <class TY, class TO, int V>
__global__ void __launch_bounds__(256) k_moe_combine(const CombineArgs a) {
    const int64_t total = a.tokens * a.per_row;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        const int64_t t = u / a.per_row, c = (u - t * a.per_row) * V;
        const TY* y = reinterpret_cast<const TY*>(a.y) + c;
        float acc[V];
        const TO* res = reinterpret_cast<const TO*>(a.residual);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t p = __ldg(a.pos + t * a.top_k + j);
            if (p < 0 || p >= a.y_rows) continue;
            const float w = __ldg(a.weights + t * a.top_k + j);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(w, ld1<TY>(y + p * a.hidden + i), acc[i]);
        }
        TO* o = reinterpret_cast<TO*>(a.out) + t * a.hidden + c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (res) acc[i] += (float)res[t * a.hidden + c + i];
            o[i] = to_out<TO>(acc[i]);
        }
    }
}

// dy[pos] = weights * dout and dweights = <dout, y[pos]>: one CTA per token.
struct CombineBwdArgs {
    const void *dout, *y;
    const int32_t* pos;
    const float* weights;
    void* dy;
    float* dweights;
    int64_t tokens, y_rows, hidden;
    int top_k;
};

template <class T>
__global__ void __launch_bounds__(128) k_moe_combine_bwd(const CombineBwdArgs a) {
    __shared__ float part[32][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const T* dout = reinterpret_cast<const T*>(a.dout) + t * a.hidden;
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t p = a.pos[t * a.top_k + j];
            float dot = 0.0f;
            if (p >= 0 && p < a.y_rows) {
                const float w = a.weights[t * a.top_k + j];
                const T* y = reinterpret_cast<const T*>(a.y) + p * a.hidden;
                T* dy = reinterpret_cast<T*>(a.dy) + p * a.hidden;
                for (int64_t c = threadIdx.x; c < a.hidden; c += 128) {
                    const float d = ld1<T>(dout + c);
                    dot = fmaf(d, ld1<T>(y + c), dot);
                    dy[c] = to_out<T>(w * d);
                }
            }
            dot = warp_sum(dot);
            if (lane == 0) part[j][warp] = dot;
        }
        __syncthreads();
        if (threadIdx.x < a.top_k) {
            float s = 0.0f;
            for (int w = 0; w < 4; ++w) s += part[threadIdx.x][w];
            a.dweights[t * a.top_k + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

template <class TY, class TO>
cudaError_t launch_combine(CombineArgs a, cudaStream_t st) {
    a.per_row = a.hidden;
    const int64_t need = (a.tokens * a.per_row + 255) / 256, most = (int64_t)sm_count() * 64;
    k_moe_combine<TY, TO, 1><<<(unsigned)(need < most ? need : most), 256, 0, st>>>(a);
    return cudaGetLastError();
}
template <class TY>
cudaError_t combine_out(const CombineArgs& a, bq_dtype out, cudaStream_t st) {
    if (out == BQ_F32) return launch_combine<TY, float>(a, st);
    if (out == BQ_F16) return launch_combine<TY, __half>(a, st);
    return launch_combine<TY, __nv_bfloat16>(a, st);
}
template <class T>
cudaError_t launch_combine_bwd(const CombineBwdArgs& a, cudaStream_t st) {
    const int64_t most = (int64_t)sm_count() * 16;
    k_moe_combine_bwd<T><<<(unsigned)(a.tokens < most ? a.tokens : most), 128, 0, st>>>(a);
    return cudaGetLastError();
}

bool float_type(bq_dtype t) { return t == BQ_F32 || t == BQ_F16 || t == BQ_BF16; }
uintptr_t type_mask(bq_dtype t) { return t == BQ_F32 ? 3u : 1u; }
bool misaligned(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }
bq_status from(cudaError_t e) {
    return e == cudaSuccess ? BQ_OK : e == cudaErrorNotSupported ? BQ_ERR_UNSUPPORTED : BQ_ERR_CUDA;
}
// Pairs (token, slot) are counted in 32 bits.
bool pairs_fit(int64_t tokens, int32_t top_k) { return tokens <= 0x7fffffffll / top_k; }

}  // namespace
}  // namespace bq

using namespace bq;

extern "C" bq_status bq_moe_route(const void* logits, bq_dtype dtype, int64_t tokens, int32_t experts, const float* bias,
                                  bq_score score, int32_t n_groups, int32_t top_groups, int32_t group_top, int32_t top_k,
                                  int32_t renormalize, float scale, int32_t* ids, float* weights, void* stream) {
    if (!float_type(dtype) || (score != BQ_SCORE_SOFTMAX && score != BQ_SCORE_SIGMOID)) return BQ_ERR_UNSUPPORTED;
    if (tokens < 0 || experts < 1 || experts > 1024 || top_k < 1 || top_k > 32) return BQ_ERR_INVALID_ARG;
    if (n_groups < 1 || n_groups > 32 || experts % n_groups != 0 || top_groups < 1 || top_groups > n_groups)
        return BQ_ERR_INVALID_ARG;
    if (group_top < 1 || group_top > 2 || top_k > top_groups * (experts / n_groups)) return BQ_ERR_INVALID_ARG;
    if (!pairs_fit(tokens, top_k)) return BQ_ERR_INVALID_ARG;
    if (tokens == 0) return BQ_OK;
    if (!logits || !ids || !weights) return BQ_ERR_INVALID_ARG;
    if (misaligned(logits, type_mask(dtype)) || misaligned(bias, 3) || misaligned(ids, 3) || misaligned(weights, 3))
        return BQ_ERR_MISALIGNED;
    RouteArgs a{logits, bias, tokens, experts, top_k, n_groups, top_groups, group_top, score == BQ_SCORE_SIGMOID,
                renormalize != 0, 0, scale, ids, weights};
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == BQ_F32) return from(by_width<float, RouteLaunch>(a, st));
    if (dtype == BQ_F16) return from(by_width<__half, RouteLaunch>(a, st));
    return from(by_width<__nv_bfloat16, RouteLaunch>(a, st));
}

extern "C" bq_status bq_moe_route_backward(const void* logits, bq_dtype dtype, int64_t tokens, int32_t experts,
                                           const int32_t* ids, const float* dweights, bq_score score, int32_t top_k,
                                           int32_t renormalize, float scale, void* dlogits, void* stream) {
    if (!float_type(dtype) || (score != BQ_SCORE_SOFTMAX && score != BQ_SCORE_SIGMOID)) return BQ_ERR_UNSUPPORTED;
    if (tokens < 0 || experts < 1 || experts > 1024 || top_k < 1 || top_k > 32 || !pairs_fit(tokens, top_k))
        return BQ_ERR_INVALID_ARG;
    if (tokens == 0) return BQ_OK;
    if (!logits || !ids || !dweights || !dlogits) return BQ_ERR_INVALID_ARG;
    if (misaligned(logits, type_mask(dtype)) || misaligned(dlogits, type_mask(dtype)) || misaligned(ids, 3) ||
        misaligned(dweights, 3))
        return BQ_ERR_MISALIGNED;
    RouteBwdArgs a{logits, ids, dweights, tokens, experts, top_k, score == BQ_SCORE_SIGMOID, renormalize != 0, 0,
                   scale, dlogits};
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == BQ_F32) return from(by_width<float, RouteBwdLaunch>(a, st));
    if (dtype == BQ_F16) return from(by_width<__half, RouteBwdLaunch>(a, st));
    return from(by_width<__nv_bfloat16, RouteBwdLaunch>(a, st));
}

extern "C" bq_status bq_moe_group(const int32_t* ids, int64_t tokens, int32_t top_k, int32_t first_expert,
                                  int32_t n_experts, int32_t* offsets, int32_t* rows, int32_t* pos, void* stream) {
    if (tokens < 0 || top_k < 1 || !pairs_fit(tokens, top_k) || first_expert < 0 || n_experts < 1 || n_experts > 1024)
        return BQ_ERR_INVALID_ARG;
    if (!offsets || (tokens > 0 && (!ids || !rows || !pos))) return BQ_ERR_INVALID_ARG;
    if (misaligned(ids, 3) || misaligned(offsets, 3) || misaligned(rows, 3) || misaligned(pos, 3)) return BQ_ERR_MISALIGNED;
    GroupArgs a{ids, tokens * top_k, top_k, first_expert, n_experts, offsets, rows, pos};
    return from(launch_group(a, (cudaStream_t)stream));
}

extern "C" bq_status bq_moe_combine(const void* y, bq_dtype y_dtype, int64_t y_rows, int64_t hidden, const int32_t* pos,
                                    const float* weights, int64_t tokens, int32_t top_k, const void* residual, void* out,
                                    bq_dtype out_dtype, void* stream) {
    if (!float_type(y_dtype) || !float_type(out_dtype)) return BQ_ERR_UNSUPPORTED;
    if (y_rows < 0 || hidden < 0 || hidden >= (1ll << 31) || tokens < 0 || top_k < 1 || !pairs_fit(tokens, top_k))
        return BQ_ERR_INVALID_ARG;
    if (tokens == 0 || hidden == 0) return BQ_OK;
    if ((!y && y_rows > 0) || !pos || !weights || !out) return BQ_ERR_INVALID_ARG;
    if (misaligned(y, type_mask(y_dtype)) || misaligned(out, type_mask(out_dtype)) ||
        misaligned(residual, type_mask(out_dtype)) || misaligned(pos, 3) || misaligned(weights, 3))
        return BQ_ERR_MISALIGNED;
    CombineArgs a{y, pos, weights, residual, out, tokens, y_rows, hidden, 0, top_k};
    cudaStream_t st = (cudaStream_t)stream;
    if (y_dtype == BQ_F32) return from(combine_out<float>(a, out_dtype, st));
    if (y_dtype == BQ_F16) return from(combine_out<__half>(a, out_dtype, st));
    return from(combine_out<__nv_bfloat16>(a, out_dtype, st));
}

extern "C" bq_status bq_moe_combine_backward(const void* dout, const void* y, bq_dtype dtype, int64_t y_rows,
                                             int64_t hidden, const int32_t* pos, const float* weights, int64_t tokens,
                                             int32_t top_k, void* dy, float* dweights, void* stream) {
    if (!float_type(dtype)) return BQ_ERR_UNSUPPORTED;
    if (y_rows < 0 || hidden < 0 || hidden >= (1ll << 31) || tokens < 0 || top_k < 1 || top_k > 32 ||
        !pairs_fit(tokens, top_k))
        return BQ_ERR_INVALID_ARG;
    if (tokens == 0) return BQ_OK;
    if ((!dout && hidden > 0) || ((!y || !dy) && y_rows > 0 && hidden > 0) || !pos || !weights || !dweights)
        return BQ_ERR_INVALID_ARG;
    const uintptr_t m = type_mask(dtype);
    if (misaligned(dout, m) || misaligned(y, m) || misaligned(dy, m) || misaligned(pos, 3) || misaligned(weights, 3) ||
        misaligned(dweights, 3))
        return BQ_ERR_MISALIGNED;
    CombineBwdArgs a{dout, y, pos, weights, dy, dweights, tokens, y_rows, hidden, top_k};
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == BQ_F32) return from(launch_combine_bwd<float>(a, st));
    if (dtype == BQ_F16) return from(launch_combine_bwd<__half>(a, st));
    return from(launch_combine_bwd<__nv_bfloat16>(a, st));
}
