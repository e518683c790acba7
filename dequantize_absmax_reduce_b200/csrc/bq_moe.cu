// Expert layers: routing (choice of experts and their weights) with its
// gradient, the expert order of the routed rows, and the sum of the experts'
// rows back into tokens with its gradient.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "bq.h"
#include "bq_act.cuh"
#include "bq_cols.cuh"
#include "bq_device.cuh"
#include "bq_internal.h"

namespace bq {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- routing
// One warp per token. Lane l holds the C consecutive experts from l * C, so
// that the lowest lane with the largest value holds the lowest index of it.
//
// The order of the choice values decides which experts a token gets, and it is
// the order of f64 arithmetic. Where the values are the logits, 32 bits hold them
// exactly. Where they are scores (and biases), scores in f32 are off by less than 28 * 2^-24
// (softmax: an exponential within 2 ulp, its argument's rounding, ten levels of a
// sum of such terms, a reciprocal and a product, on values of at most 1; a sigmoid
// has less) and the sum with the bias by 2^-24 of its size. Values nearer than
// 2^-18 max(1, |v|) to one another, and what the keys' low bits take (sums of two:
// 1.5 * 2^-18 max(1, |v|) each, v the larger member), are looked at again in f64:
// the candidates alone, those too near the last to be told from it among them, or
// the groups' sums. That happens to about one row in a hundred of 256 experts. In
// f64 throughout, 16384 such rows took 65 us; with the near rows chosen anew in
// f64, their wait alone cost 7 us.
//
// A lane sorts its values once, as integers in their order whose lowest bits give
// way to the value's number in the lane (the nearness test allows for that; so do
// logits of 16 bits, which leave them free, and f32 logits that agree in all but
// those bits are looked at again too). A choice is then one redux over the lanes'
// largest, one ballot, and its lane moves up its list.
struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t tokens;
    int experts, top_k, n_groups, top_groups, group_top, sigmoid, renorm, vec;
    int scored;                // choice values: score + bias (0 without one); else the logits
    int group_lanes;           // lanes of a group, a power of two, or 0: groups do not end with lanes
    int sum_lanes;             // half the power of two that holds top_k
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

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
// exp(a - b) for a <= b, without the rounding of the difference, which would cost
// |a - b| half steps: the part lost to it (Knuth's exact sum) comes back to first
// order. 1 where they are equal, infinities among them.
__device__ __forceinline__ float exp_diff(float a, float b) {
    const float d = a - b;
    if (a == b) return 1.0f;
    if (!(d > -150.0f)) return 0.0f;
    const float part = d - a, lost = (a - (d - part)) - (b + part);
    const float e = expf(d);
    return fmaf(e, lost, e);
}
// The same for a share of which a result in T is made: for 16 bits the difference's
// rounding (at most 2^-18 of the share before exp leaves f32's normal numbers) is far
// below half a step.
template <class T>
__device__ __forceinline__ float exp_share(float a, float b) {
    if constexpr (std::is_same<T, float>::value) return exp_diff(a, b);
    else return expf(a == b ? 0.0f : a - b);
}
// Integers in the order of floats; above 0, which stands for "not available".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A row's choice values in f64: the lane's C, from the logits in memory.
template <class T, int C>
__device__ __forceinline__ void exact_values(const RouteArgs& a, const T* row, int lane, double (&v)[C]) {
    double x[C], top = -CUDART_INF, sum = 0.0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = lane * C + i;
        x[i] = e < a.experts ? (double)ld1<T>(row + e) : -CUDART_INF;
        if (x[i] > top) top = x[i];
    }
    if (a.scored && !a.sigmoid) {
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = lane * C + i < a.experts && x[i] == x[i] ? exp(x[i] == top ? 0.0 : x[i] - top) : 0.0;
            sum += v[i];
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = lane * C + i;
        const double s = !a.scored ? x[i] : a.sigmoid ? 1.0 / (1.0 + exp(-x[i])) : v[i] / sum;
        v[i] = a.bias && e < a.experts ? s + (double)__ldg(a.bias + e) : s;
        if (!(x[i] > -CUDART_INF) || v[i] != v[i]) v[i] = -CUDART_INF;
    }
}
// The groups that stay, in f64: bit j of the result for the lane j that stands for
// them (every lane of a group where groups end with lanes, else lane g for group
// g). vs: room for the row's values.
template <class T, int C>
__device__ __noinline__ unsigned exact_groups(const RouteArgs& a, const T* row, int lane, double* vs) {
    double v[C];
    exact_values<T, C>(a, row, lane, v);
    double b1 = -CUDART_INF, b2 = -CUDART_INF;
    auto enter = [&](double u) {
        if (u > b1) { b2 = b1; b1 = u; } else if (u > b2) b2 = u;
    };
    const bool by_lane = a.group_lanes > 0;
    const int every = by_lane ? a.group_lanes : 1, mine = lane / every;
    if (by_lane) {
#pragma unroll
        for (int i = 0; i < C; ++i) enter(v[i]);
        for (int o = 1; o < every; o <<= 1) {
            const double o1 = __shfl_xor_sync(FULL, b1, o), o2 = __shfl_xor_sync(FULL, b2, o);
            enter(o1);
            enter(o2);
        }
    } else {
        const int gsize = a.experts / a.n_groups;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (lane * C + i < a.experts) vs[lane * C + i] = v[i];
        __syncwarp();
        if (lane < a.n_groups)
            for (int j = 0; j < gsize; ++j) enter(vs[lane * gsize + j]);
        __syncwarp();
    }
    double gv = b1;
    if (a.group_top == 2 && b2 > -CUDART_INF) gv += b2;
    int ahead = 0;
    for (int j = 0; j < a.n_groups; ++j) {
        const double o = __shfl_sync(FULL, gv, j * every);
        ahead += (o > gv || (o == gv && j < mine)) ? 1 : 0;
    }
    return __ballot_sync(FULL, mine < a.n_groups && ahead < a.top_groups);
}
// The choice among the warp's candidates (lane j < n holds one, -1 elsewhere), by
// their values in f64: returns the id of rank `lane` below top_k.
template <class T, int C>
__device__ __noinline__ int exact_order(const RouteArgs& a, const T* row, int lane, int id, int n, double* room) {
    double v = -CUDART_INF;
    if (a.scored && !a.sigmoid) {
        double all[C];
        exact_values<T, C>(a, row, lane, all);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (lane * C + i < a.experts) room[lane * C + i] = all[i];
        __syncwarp();
        if (id >= 0) v = room[id];
        __syncwarp();
    } else if (id >= 0) {
        const double x = (double)ld1<T>(row + id);
        v = a.scored ? 1.0 / (1.0 + exp(-x)) + (a.bias ? (double)__ldg(a.bias + id) : 0.0) : x;
    }
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(FULL, v, j);
        const int oi = __shfl_sync(FULL, id, j);
        rank += o > v || (o == v && oi < id) ? 1 : 0;
    }
    int* to = reinterpret_cast<int*>(room);
    if (id >= 0) to[rank] = id;
    __syncwarp();
    const int got = lane < n && lane < a.top_k ? to[lane] : -1;
    __syncwarp();
    return got;
}
// The choice of one row in f64 throughout, where more than 32 values are too near
// one another: returns the id that lane j < top_k holds.
template <class T, int C>
__device__ __noinline__ int route_exact(const RouteArgs& a, const T* row, int lane, unsigned kept) {
    double v[C];
    exact_values<T, C>(a, row, lane, v);
    const int gsize = a.experts / a.n_groups;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = lane * C + i;
        const int bit = a.group_lanes > 0 ? lane : e / gsize;
        if (a.n_groups > 1 && e < a.experts && !((kept >> bit) & 1u)) v[i] = -CUDART_INF;
    }
    int id = -1;
    for (int it = 0; it < a.top_k; ++it) {
        double best = -CUDART_INF;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (v[i] > best) { best = v[i]; bi = lane * C + i; }
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(FULL, best, o);
            const int oi = __shfl_xor_sync(FULL, bi, o);
            if (ob > best || (ob == best && oi < bi)) { best = ob; bi = oi; }
        }
        if (!(best > -CUDART_INF)) break;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (lane * C + i == bi) v[i] = -CUDART_INF;
        if (lane == it) id = bi;
    }
    return id;
}

// Sorts v[0 .. C) downwards (Batcher's odd-even merge sort).
template <int C>
__device__ __forceinline__ void sort_down(uint32_t (&v)[C]) {
#pragma unroll
    for (int p = 1; p < C; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < C; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < C && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                        v[i + j + k] = lo;
                    }
}

// Whether two values (as masked keys, the larger first) may stand in another order in f64.
template <class T, int C, bool SCORED>
__device__ __forceinline__ bool too_near(uint32_t hi, uint32_t lo) {
    if constexpr (SCORED) {
        const float v = key_value(hi);
        // (written so that infinities count as near)
        return !(v - key_value(lo) > (0x1p-18f + C * 0x1p-22f) * fmaxf(1.0f, fabsf(v)));
    } else {
        return std::is_same<T, float>::value && C > 1 && hi == lo;
    }
}

// SCORED: choice values are score + bias (0 without one); else the logits.
// (Up to eight experts a lane seven CTAs share an SM: 24.9 us at 16384 x 256 in
// groups with a bias, sigmoid, and 31.2 softmax; five 24.4 and 32.5, six 26.4 and 33.2.)
template <class T, int C, bool SCORED>
__global__ void __launch_bounds__(128, C <= 8 ? 7 : 2) k_moe_route(const RouteArgs a) {
    extern __shared__ double route_smem[];
    constexpr uint32_t LOW = C - 1;                    // bits that hold a value's number in its lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double* room = route_smem + (size_t)warp * a.experts;
    const int gsize = a.experts / a.n_groups;
    // Biases, and bits of the experts that are in service (a bias of -inf or NaN: never chosen).
    float bias[C];
    uint32_t serve = 0u;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const bool in = lane * C + i < a.experts;
        bias[i] = SCORED && in && a.bias ? __ldg(a.bias + lane * C + i) : 0.0f;
        serve |= in && bias[i] > -CUDART_INF_F ? 1u << i : 0u;
    }
    for (int64_t t = (int64_t)blockIdx.x * 4 + warp; t < a.tokens; t += (int64_t)gridDim.x * 4) {
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.experts;
        float x[C];
        load_logits<T, C>(row, lane, a.experts, a.vec, x);
        // The softmax's largest logit and sum, where scores enter.
        float top = -CUDART_INF_F, inv = 0.0f, p[C];
        if (!a.sigmoid) {
#pragma unroll
            for (int i = 0; i < C; ++i) top = fmaxf(top, x[i]);       // (a NaN is left out)
            top = key_value(__reduce_max_sync(FULL, order_key(top)));
            if (SCORED || !a.renorm) {
                float part[C];
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    p[i] = lane * C + i < a.experts && x[i] == x[i] ? expf(x[i] == top ? 0.0f : x[i] - top) : 0.0f;
                    part[i] = p[i];
                }
#pragma unroll
                for (int w = C / 2; w > 0; w /= 2)
#pragma unroll
                    for (int i = 0; i < w; ++i) part[i] += part[i + w];
                inv = 1.0f / warp_sum(part[0]);
            }
        }
        // Keys; 0: not available. Those of scores are packed at once, so that a
        // group's sum is off by their low bits too; logits are packed below.
        uint32_t key[C], least = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (SCORED) {
                const float v = (a.sigmoid ? logistic(x[i]) : p[i] * inv) + bias[i];
                const uint32_t k = (order_key(v) & ~LOW) | (LOW - i);
                key[i] = x[i] > -CUDART_INF_F && (serve & (1u << i)) ? k : 0u;
            } else {
                // (adding 0 makes one zero of the two)
                key[i] = x[i] > -CUDART_INF_F && (serve & (1u << i)) ? order_key(x[i] + 0.0f) : 0u;
            }
            least = min(least, key[i]);
        }
        bool bad = false;                              // a NaN in the row
        if (__any_sync(FULL, least == 0u)) {
#pragma unroll
            for (int i = 0; i < C; ++i) bad |= x[i] != x[i];
            bad = __any_sync(FULL, bad);
        }
        unsigned groups = FULL;                        // lanes, or groups, that stay
        if (a.n_groups > 1) {
            // A group's two best: of the lanes that hold it, or where groups do not
            // end with lanes through shared memory.
            uint32_t g1 = 0u, g2 = 0u;
            auto enter = [&](uint32_t k) {
                g2 = max(g2, min(k, g1));
                g1 = max(g1, k);
            };
            const bool by_lane = a.group_lanes > 0;
            int mine = lane;                           // this lane's group
            if (by_lane) {
#pragma unroll
                for (int i = 0; i < C; ++i) enter(key[i]);
                for (int o = 1; o < a.group_lanes; o <<= 1) {
                    const uint32_t o1 = __shfl_xor_sync(FULL, g1, o), o2 = __shfl_xor_sync(FULL, g2, o);
                    g2 = max(max(g2, o2), min(g1, o1));
                    g1 = max(g1, o1);
                }
                mine = lane >> (__ffs(a.group_lanes) - 1);
            } else {
                uint32_t* vs = reinterpret_cast<uint32_t*>(room);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < C; ++i)
                    if (lane * C + i < a.experts) vs[lane * C + i] = key[i];
                __syncwarp();
                if (lane < a.n_groups)
                    for (int j = 0; j < gsize; ++j) enter(vs[lane * gsize + j]);
            }
            bool kept = false, near = false;
            if (SCORED || a.group_top == 1) {
                // Values fit f32 (sums of scores: nearly): the best top_groups one by one.
                const bool two = a.group_top == 2 && g2 != 0u;
                const float v1 = g1 ? key_value(g1) : -CUDART_INF_F, v2 = two ? key_value(g2) : 0.0f;
                const float gv = v1 + v2;
                uint32_t gk = g1 ? order_key(gv + 0.0f) : 0u;
                for (int r = 0; r < a.top_groups; ++r) {
                    const uint32_t m = __reduce_max_sync(FULL, gk);
                    if (m == 0u) break;
                    const int w = __shfl_sync(FULL, mine, __ffs(__ballot_sync(FULL, gk == m)) - 1);
                    if (mine == w) { kept = true; gk = 0u; }
                }
                if (SCORED) {
                    // A sum is off by what its members are off, however small it is itself:
                    // near where the lowest that a group that stays may lie is not above the
                    // highest that one left out may. (A key's low bits are up to C steps of 2^-23
                    // of the value; 96 * 2^-24 holds the scores' errors and the roundings.)
                    const float size = fmaxf(fabsf(v1), fabsf(v2));
                    const float err = 0x1.8p-18f * fmaxf(1.0f, size) + C * 0x1p-22f * size;
                    const bool fin = fabsf(v1) + fabsf(v2) < CUDART_INF_F;   // (a packed infinity reads as NaN)
                    const float lo = fin ? gv - err : -CUDART_INF_F, hi = fin ? gv + err : CUDART_INF_F;
                    const uint32_t least_in = __reduce_min_sync(FULL, g1 && kept ? order_key(lo) : FULL);
                    const uint32_t most_out = __reduce_max_sync(FULL, g1 && !kept ? order_key(hi) : 0u);
                    near = most_out >= least_in;
                }
            } else {
                const int every = by_lane ? a.group_lanes : 1;
                const double gv = g1 == 0u ? -CUDART_INF : (double)key_value(g1) + (g2 ? (double)key_value(g2) : 0.0);
                int ahead = 0;
                for (int j = 0; j < a.n_groups; ++j) {
                    const double o = __shfl_sync(FULL, gv, j * every);
                    ahead += o > gv || (o == gv && j < mine) ? 1 : 0;
                }
                kept = mine < a.n_groups && ahead < a.top_groups;
            }
            groups = SCORED && near ? exact_groups<T, C>(a, row, lane, room) : __ballot_sync(FULL, kept);
            if (by_lane) {
                kept = (groups >> lane) & 1u;
#pragma unroll
                for (int i = 0; i < C; ++i) key[i] = kept ? key[i] : 0u;
            } else {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = lane * C + i;
                    if (e < a.experts && !((groups >> (e / gsize)) & 1u)) key[i] = 0u;
                }
            }
        }
        if (!SCORED && C > 1) {
#pragma unroll
            for (int i = 0; i < C; ++i) key[i] = key[i] ? (key[i] & ~LOW) | (LOW - i) : 0u;
        }
        sort_down<C>(key);
        // The top_k best, and behind them those too near the last to be told from it.
        int id = -1, n = 0;
        uint32_t mine = 0u, last = 0u;                 // this lane's candidate; the top_k-th
        bool lost = false;                             // candidates beyond the warp's lanes
        for (;; ++n) {
            const uint32_t head = key[0] & ~LOW, m = __reduce_max_sync(FULL, head);
            if (m == 0u) break;
            if (n >= a.top_k && !too_near<T, C, SCORED>(last, m)) break;
            if (n == 32) { lost = true; break; }
            if (n == a.top_k - 1) last = m;
            const int w = __ffs(__ballot_sync(FULL, head == m)) - 1;
            const int e = __shfl_sync(FULL, lane * C + (int)(LOW - (key[0] & LOW)), w);
            if (lane == n) { id = e; mine = m; }
            if (lane == w) {
#pragma unroll
                for (int i = 0; i + 1 < C; ++i) key[i] = key[i + 1];
                key[C - 1] = 0u;
            }
        }
        if (SCORED || std::is_same<T, float>::value) {
            const uint32_t behind = __shfl_down_sync(FULL, mine, 1);
            const bool unsure = lane < n - 1 && too_near<T, C, SCORED>(mine, behind);
            if (__any_sync(FULL, unsure || lost))
                id = lost ? route_exact<T, C>(a, row, lane, groups) : exact_order<T, C>(a, row, lane, id, n, room);
        }
        // Weights in f32; renormalised ones relative to the largest chosen, so
        // that small scores keep their ratios.
        const bool there = id >= 0 && lane < a.top_k;
        const float l = there ? ld1<T>(row + id) : -CUDART_INF_F;
        float w;
        if (a.sigmoid || a.renorm) {
            const float low = a.sigmoid ? fminf(l, 0.0f) : l;
            const float ref = a.renorm ? key_value(__reduce_max_sync(FULL, order_key(low))) : 0.0f;
            w = there ? exp_diff(low, ref) : 0.0f;
            if (a.sigmoid) w = __fdividef(w, 1.0f + expf(-fabsf(l)));   // sigmoid = exp(min(l, 0)) / (1 + exp(-|l|))
            if (a.renorm) {
                // Where f64 has no score left (exp(-746) is 0), there is nothing to share.
                const bool none = a.sigmoid ? ref < -745.0f : ref - top < -745.0f;
                float sum = there ? w : 0.0f;
                for (int o = a.sum_lanes; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
                w = sum > 0.0f && !none ? __fdividef(w, sum) : 0.0f;
            }
        } else {
            w = there ? exp_diff(l, top) * inv : 0.0f;
        }
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = id;
            a.weights[t * a.top_k + lane] = bad ? CUDART_NAN_F : there ? w * a.scale : 0.0f;
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
// relative to the largest chosen one, so that small scores do not vanish (unless
// f64 holds no score of the row's chosen either, where the weights are 0).
struct RouteBwdArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    int64_t tokens;
    int experts, top_k, sigmoid, renorm, vec;
    float scale;
    void* dlogits;
};

// One kernel for each form: together they would hold each other's registers (5.3 us
// against 4.7 at 8192 x 128). (Told that four CTAs of the widest rows share an SM, the
// compiler spends the registers that it has: 4096 x 1024 bf16 sigmoid 9.6 -> 7.6 us.)
enum RouteForm { ROUTE_SOFTMAX, ROUTE_SHARES, ROUTE_SIGMOID };   // softmax as it is, softmax renormalised, sigmoid

template <class T, int C, RouteForm F>
__global__ void __launch_bounds__(128, C > 16 ? 4 : 0) k_moe_route_bwd(const RouteBwdArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = (int64_t)blockIdx.x * 4 + warp; t < a.tokens; t += (int64_t)gridDim.x * 4) {
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.experts;
        int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
        if (id >= a.experts) id = -1;
        const float g = id >= 0 ? a.dweights[t * a.top_k + lane] : 0.0f;
        const float l = id >= 0 ? ld1<T>(row + id) : -CUDART_INF_F;
        constexpr bool DENSE = F == ROUTE_SOFTMAX;
        [[maybe_unused]] float p[C];
        float full[C], contrib;
        [[maybe_unused]] float shift = 0.0f;
        if constexpr (DENSE) {
            load_logits<T, C>(row, lane, a.experts, a.vec, p);
            float top = -CUDART_INF_F;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < C; ++i) { bad |= p[i] != p[i]; top = fmaxf(top, p[i]); }
            top = warp_max(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                p[i] = lane * C + i < a.experts ? exp_share<T>(p[i], top) : 0.0f;
                sum += p[i];
            }
            sum = warp_sum(sum);
            if (__any_sync(FULL, bad)) sum = CUDART_NAN_F;
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < C; ++i) p[i] *= inv;
            const float s = id >= 0 ? exp_share<T>(l, top) * inv : 0.0f;
            contrib = a.scale * g;
            shift = warp_sum(contrib * s);
        } else {
            // Scores up to a common factor, and s (1 - s) / s of the sigmoid.
            constexpr bool SIGMOID = F == ROUTE_SIGMOID;
            const bool renorm = !SIGMOID || a.renorm;
            const float low = SIGMOID ? fminf(l, 0.0f) : l;
            float s = 0.0f, tail = 1.0f;
            bool none = false;                             // no score left in f64: the weights are 0, not shares
            if (renorm) {
                const float top = warp_max(low);
                if constexpr (SIGMOID) {
                    none = top < -745.0f;
                } else {
                    load_logits<T, C>(row, lane, a.experts, a.vec, p);
                    float best = top;
#pragma unroll
                    for (int i = 0; i < C; ++i) best = fmaxf(best, p[i]);
                    none = top - warp_max(best) < -745.0f;
                }
                s = id >= 0 ? exp_diff(low, top) : 0.0f;
            } else {
                s = id >= 0 ? expf(low) : 0.0f;
            }
            if constexpr (SIGMOID) {
                const float u = expf(-fabsf(l));           // s = exp(min(l, 0)) / (1 + u)
                s = s / (1.0f + u);
                tail = (l >= 0.0f ? u : 1.0f) / (1.0f + u);   // 1 - s
            }
            float gs;
            if (renorm) {
                const float d = warp_sum(s), gm = warp_sum(g * s);
                s = d > 0.0f ? s / d : 0.0f;
                gs = a.scale * (g - (d > 0.0f ? gm / d : 0.0f));
            } else {
                gs = a.scale * g;
            }
            contrib = id >= 0 && !none ? gs * s * tail : 0.0f;
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
        if constexpr (DENSE) {
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
// CTAs of four warps that run at one time, so that every warp gets the same
// number of tokens (more CTAs than that would leave a ragged last round).
template <class K>
cudaError_t resident_ctas(K kern, size_t smem, int (&cache)[64], int64_t tokens, unsigned* grid) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    int n = __atomic_load_n(&cache[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 128, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        n *= sm_count();
        __atomic_store_n(&cache[dev], n, __ATOMIC_RELEASE);
    }
    const int64_t need = (tokens + 3) / 4, rounds = (need + n - 1) / n;
    *grid = (unsigned)((need + rounds - 1) / rounds);
    return cudaSuccess;
}
template <class T, int C>
struct RouteLaunch {
    static cudaError_t go(RouteArgs a, cudaStream_t st) {
        constexpr int VEC = Traits<T>::VEC;
        a.vec = a.experts % VEC == 0 && ((uintptr_t)a.logits & 15u) == 0;
        const int gsize = a.experts / a.n_groups, lanes = gsize / C;
        a.group_lanes = gsize % C == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
        const size_t smem = 4 * sizeof(double) * (size_t)a.experts;
        // (by the shared memory of a full width: the cached count serves every call)
        static int scored[64] = {0}, plain[64] = {0};
        unsigned grid = 0;
        const size_t most = 4 * sizeof(double) * 32 * C;
        const cudaError_t e = a.scored ? resident_ctas(k_moe_route<T, C, true>, most, scored, a.tokens, &grid)
                                       : resident_ctas(k_moe_route<T, C, false>, most, plain, a.tokens, &grid);
        if (e != cudaSuccess) return e;
        if (a.scored) k_moe_route<T, C, true><<<grid, 128, smem, st>>>(a);
        else k_moe_route<T, C, false><<<grid, 128, smem, st>>>(a);
        return cudaGetLastError();
    }
};
template <class T, int C>
struct RouteBwdLaunch {
    static cudaError_t go(RouteBwdArgs a, cudaStream_t st) {
        constexpr int VEC = Traits<T>::VEC;
        a.vec = a.experts % VEC == 0 && ((uintptr_t)a.logits & 15u) == 0 && ((uintptr_t)a.dlogits & 15u) == 0;
        return a.sigmoid ? as<ROUTE_SIGMOID>(a, st) : a.renorm ? as<ROUTE_SHARES>(a, st) : as<ROUTE_SOFTMAX>(a, st);
    }
    template <RouteForm F>
    static cudaError_t as(const RouteBwdArgs& a, cudaStream_t st) {
        static int ctas[64] = {0};
        unsigned grid = 0;
        const cudaError_t e = resident_ctas(k_moe_route_bwd<T, C, F>, 0, ctas, a.tokens, &grid);
        if (e != cudaSuccess) return e;
        k_moe_route_bwd<T, C, F><<<grid, 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

// ---------------------------------------------------------------- expert order
// A stable counting sort of the pairs (token, slot) by expert in one launch:
// the CTAs of a cluster (16, where the device allows that many) take consecutive runs of the pairs, each warp a
// consecutive run of its CTA's. Pass one counts per warp and expert; prefix
// sums over the warps, over the CTAs (through distributed shared memory) and
// over the experts give every (warp, expert) its first position; pass two
// hands out the positions in the order of the pairs: a lane's place among the
// equal experts of its 32 comes from ballots over the bits of the expert's
// number. The same result every time (only the counts use atomics).
// Bound by latency: a run's ids are loaded GROUP_ROWS at a time, so that few
// loads from memory follow one another, and kept where they are all.
constexpr int GROUP_CTAS = 16, GROUP_NT = 1024, GROUP_WARPS = GROUP_NT / 32, GROUP_ROWS = 16;

struct GroupArgs {
    const int32_t* ids;
    int pairs;                 // below 2^31
    int per;                   // pairs of a warp, a multiple of 32
    int first, n, bits;        // bits: of the largest expert number, n itself (other experts) included
    FastDiv top_k;
    int32_t *offsets, *rows, *pos;
};

__global__ void __launch_bounds__(GROUP_NT, 1) k_moe_group(const GroupArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ int32_t group_smem[];
    int32_t* table = group_smem;                        // [GROUP_WARPS][n]
    int32_t* mine = table + (size_t)GROUP_WARPS * a.n;  // [n] this CTA's counts
    __shared__ int32_t warp_tot[GROUP_WARPS];
    __shared__ int32_t total_all;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first_pair = ((int64_t)rank * GROUP_WARPS + warp) * a.per;
    const int lo = (int)min((int64_t)a.pairs, first_pair), hi = (int)min((int64_t)a.pairs, first_pair + a.per);
    int32_t* tw = table + (size_t)warp * a.n;
    int e[GROUP_ROWS];                                  // experts of GROUP_ROWS rows of 32 pairs; n: none of these
    auto load = [&](int at) {
#pragma unroll
        for (int r = 0; r < GROUP_ROWS; ++r) {
            e[r] = 32 * r + lane < hi - at ? __ldg(a.ids + at + 32 * r + lane) : -1;
        }
#pragma unroll
        for (int r = 0; r < GROUP_ROWS; ++r) {
            const unsigned u = (unsigned)e[r] - (unsigned)a.first;
            e[r] = e[r] >= a.first && u < (unsigned)a.n ? (int)u : a.n;
        }
    };
    for (int i = lane; i < a.n; i += 32) tw[i] = 0;
    __syncwarp();
    for (int at = lo; at < hi; at += 32 * GROUP_ROWS) {
        load(at);
#pragma unroll
        for (int r = 0; r < GROUP_ROWS; ++r)
            if (e[r] < a.n) atomicAdd(tw + e[r], 1);
        if (hi - at <= 32 * GROUP_ROWS) break;          // (at stays below 2^31)
    }
    __syncthreads();
    for (int x = tid; x < a.n; x += GROUP_NT) {
        int c[GROUP_WARPS], run = 0;
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) c[w] = table[w * a.n + x];
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) {
            table[w * a.n + x] = run;
            run += c[w];
        }
        mine[x] = run;
    }
    if (ctas > 1) cl.sync(); else __syncthreads();
    // Totals of every expert over the cluster, and of the CTAs before this one.
    int total = 0, before = 0;
    if (tid < a.n) {
        int c[GROUP_CTAS];
#pragma unroll
        for (int r = 0; r < GROUP_CTAS; ++r) c[r] = r < ctas ? cl.map_shared_rank(mine, r)[tid] : 0;
#pragma unroll
        for (int r = 0; r < GROUP_CTAS; ++r) {
            before += r < rank ? c[r] : 0;
            total += c[r];
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
        // The first position of this CTA's run goes into every warp's row.
        const int base = excl + before;
#pragma unroll 8
        for (int w = 0; w < GROUP_WARPS; ++w) table[w * a.n + tid] += base;
        if (rank == 0) {
            a.offsets[tid] = excl;
            if (tid == a.n - 1) a.offsets[a.n] = excl + total;
        }
    }
    __syncthreads();
    const bool kept = hi - lo <= 32 * GROUP_ROWS;       // pass one's ids are all of them
    for (int at = lo; at < hi; at += 32 * GROUP_ROWS) {
        if (!kept) load(at);
#pragma unroll
        for (int r = 0; r < GROUP_ROWS; ++r) {
            if (32 * r >= hi - at) break;               // uniform over the warp
            const int i = at + 32 * r + min(lane, hi - at - 32 * r - 1);
            unsigned same = FULL;
            for (int bit = 0; bit < a.bits; ++bit) {
                const unsigned set = __ballot_sync(FULL, (e[r] >> bit) & 1);
                same &= (e[r] >> bit) & 1 ? set : ~set;
            }
            const bool in = e[r] < a.n;
            const int p = in ? tw[e[r]] + __popc(same & ((1u << lane) - 1u)) : -1;
            __syncwarp();
            if (in && lane == 31 - __clz(same)) tw[e[r]] = p + 1;        // the last of the equal ones
            __syncwarp();
            if (in) a.rows[p] = (int32_t)fdiv((uint32_t)i, a.top_k);
            if (32 * r + lane < hi - at) a.pos[i] = p;
        }
        if (hi - at <= 32 * GROUP_ROWS) break;
    }
    // Rows behind the last expert's.
    for (int64_t i = total_all + (int64_t)rank * GROUP_NT + tid; i < a.pairs; i += (int64_t)ctas * GROUP_NT)
        a.rows[i] = -1;
    if (ctas > 1) cl.sync();       // no CTA leaves while another reads its counts
}

cudaError_t launch_group(GroupArgs a, cudaStream_t st) {
    const size_t smem = ((size_t)GROUP_WARPS + 1) * a.n * sizeof(int32_t);
    static int clusters[64] = {0};                      // CTAs of the largest cluster
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    int largest = __atomic_load_n(&clusters[dev], __ATOMIC_ACQUIRE);
    if (largest == 0) {
        cudaError_t e = cudaFuncSetAttribute(k_moe_group, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (GROUP_WARPS + 1) * 1024 * (int)sizeof(int32_t));
        if (e != cudaSuccess) return e;
        largest = 8;
        if (cudaFuncSetAttribute(k_moe_group, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
            cudaLaunchConfig_t probe = {};
            cudaLaunchAttribute size[1];
            size[0].id = cudaLaunchAttributeClusterDimension;
            size[0].val.clusterDim.x = GROUP_CTAS;
            size[0].val.clusterDim.y = 1;
            size[0].val.clusterDim.z = 1;
            probe.gridDim = dim3(GROUP_CTAS);
            probe.blockDim = dim3(GROUP_NT);
            probe.dynamicSmemBytes = (GROUP_WARPS + 1) * 1024 * sizeof(int32_t);
            probe.attrs = size;
            probe.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, k_moe_group, &probe) == cudaSuccess && n > 0) largest = GROUP_CTAS;
        }
        (void)cudaGetLastError();
        __atomic_store_n(&clusters[dev], largest, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    // One CTA alone while its warps have four rows of pairs at most.
    const unsigned ctas = a.pairs > 4 * GROUP_NT ? (unsigned)largest : 1u;
    a.per = (int)(((int64_t)a.pairs + (int64_t)ctas * GROUP_NT - 1) / ((int64_t)ctas * GROUP_NT)) * 32;
    a.bits = 1;
    while ((a.n >> a.bits) != 0) ++a.bits;
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
// and rounded once; NaN where a weight is. One pass over memory: a thread owns one 16-byte vector of
// out and loads that vector of every slot's row before it adds them up.
struct CombineArgs {
    const void* y;
    const int32_t* pos;
    const float* weights;
    const void* residual;
    void* out;
    int64_t tokens, y_rows, hidden;
    int top_k;
};

// A CTA takes a token (blockIdx.y: a share of its columns) and walks its columns
// with the slots' positions in registers, the rows of eight slots (f32: four) in
// flight at a time: with a thread per vector of the output, the wait for its
// positions before every load held 4096 x 8 x 7168 at 140 us. A thread has U runs
// of W columns: 8 in one where rows start on 16 bytes, else four of 2 or 1.
template <class TY, class TO, int W, int U>
__global__ void __launch_bounds__(128) k_moe_combine(const CombineArgs a) {
    constexpr int B = sizeof(TY) == 2 ? 8 : 4;
    const TO* res = reinterpret_cast<const TO*>(a.residual);
    const int64_t run = (int64_t)blockDim.x * W;       // columns from one run of a thread to its next
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int32_t* pos = a.pos + t * a.top_k;
        const float* weights = a.weights + t * a.top_k;
        int p[B];
        float w[B];
        // NaN weights mark a row of NaN logits, which may have no expert, here or
        // anywhere: its token becomes NaN with or without a row to add.
        bool bad = false;
        auto slots = [&](int j0) {
#pragma unroll
            for (int j = 0; j < B; ++j) {
                p[j] = j0 + j < a.top_k ? __ldg(pos + j0 + j) : -1;
                w[j] = j0 + j < a.top_k ? __ldg(weights + j0 + j) : 0.0f;
                if (p[j] >= a.y_rows) p[j] = -1;
                bad |= w[j] != w[j];
            }
        };
        slots(0);
        for (int64_t c0 = (int64_t)blockIdx.y * run * U + threadIdx.x * W; c0 < a.hidden; c0 += (int64_t)gridDim.y * run * U) {
            float acc[U][W];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < W; ++i) acc[u][i] = 0.0f;
            Cols<TO, W> r[U];
            if (res) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * run < a.hidden) r[u].load(res + t * a.hidden + c0 + u * run);
            }
            for (int j0 = 0; j0 < a.top_k; j0 += B) {
                if (a.top_k > B) slots(j0);
                Cols<TY, W> v[B][U];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (p[j] < 0) continue;
                    const TY* y = reinterpret_cast<const TY*>(a.y) + p[j] * a.hidden + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u == 0 || c0 + u * run < a.hidden) v[j][u].load(y + u * run);
                }
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (p[j] < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float x[W];
                        v[j][u].get(x);
#pragma unroll
                        for (int i = 0; i < W; ++i) acc[u][i] = fmaf(w[j], x[i], acc[u][i]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * run >= a.hidden) break;
                if (bad) {
#pragma unroll
                    for (int i = 0; i < W; ++i) acc[u][i] = CUDART_NAN_F;
                }
                if (res) {
                    float x[W];
                    r[u].get(x);
#pragma unroll
                    for (int i = 0; i < W; ++i) acc[u][i] += x[i];
                }
                Cols<TO, W> o;
                o.set(acc[u]);
                o.store(reinterpret_cast<TO*>(a.out) + t * a.hidden + c0 + u * run);
            }
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
    int32_t* pair_of;          // [y_rows] or null: the pair (token, slot) that names each row, for k_zero_unnamed
    int64_t tokens, y_rows, hidden;
    int top_k;
    int slice;                 // rows that each CTA looks over for names and zeroes, or 0
};
// Few enough pairs that every CTA can look through all of them for the names of its
// share of the rows, and the rows of a share at most.
constexpr int FEW_PAIRS = 2048, FEW_ROWS = 2048;
bool few_named(int64_t y_rows, int64_t pairs) { return y_rows <= FEW_ROWS && pairs <= FEW_PAIRS; }

// Zeros in a row of dy (its start and size in bytes), by nt threads.
__device__ __forceinline__ void zero_row(uint8_t* row, int64_t bytes, bool wide, int tid, int nt) {
    if (wide) {
        for (int64_t i = tid * 16; i < bytes; i += nt * 16) st16(row + i, U4{0u, 0u, 0u, 0u});
    } else {
        for (int64_t i = tid * 2; i < bytes; i += nt * 2) *reinterpret_cast<uint16_t*>(row + i) = 0;
    }
}
__device__ __forceinline__ bool rows_wide(const void* dy, int64_t row_bytes) {
    return row_bytes % 16 == 0 && ((uintptr_t)dy & 15u) == 0;
}

template <class T, int W, int U>
__global__ void __launch_bounds__(128) k_moe_combine_bwd(const CombineBwdArgs a) {
    __shared__ float part[32][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const T* dout = reinterpret_cast<const T*>(a.dout) + t * a.hidden;
        // Eight slots (f32: four) at a time: their rows are in flight together;
        // dout comes from the first level cache for all but the first of them.
        constexpr int B = sizeof(T) == 2 ? 8 : 4;
        for (int j0 = 0; j0 < a.top_k; j0 += B) {
            int p[B];
            float w[B], dot[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                p[j] = j0 + j < a.top_k ? __ldg(a.pos + t * a.top_k + j0 + j) : -1;
                w[j] = j0 + j < a.top_k ? __ldg(a.weights + t * a.top_k + j0 + j) : 0.0f;
                if (p[j] >= a.y_rows) p[j] = -1;
                dot[j] = 0.0f;
            }
            for (int64_t c0 = threadIdx.x * W; c0 < a.hidden; c0 += 128 * W * U) {
                Cols<T, W> y[B][U], d[U];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (p[j] < 0) continue;
                    const T* from = reinterpret_cast<const T*>(a.y) + p[j] * a.hidden + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u == 0 || c0 + 128 * W * u < a.hidden) y[j][u].load(from + 128 * W * u);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u == 0 || c0 + 128 * W * u < a.hidden) d[u].load(dout + c0 + 128 * W * u);
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (p[j] < 0) continue;
                    T* to = reinterpret_cast<T*>(a.dy) + p[j] * a.hidden + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (u > 0 && c0 + 128 * W * u >= a.hidden) break;
                        float g[W], x[W];
                        d[u].get(g);
                        y[j][u].get(x);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            dot[j] = fmaf(g[i], x[i], dot[j]);
                            g[i] *= w[j];
                        }
                        Cols<T, W> o;
                        o.set(g);
                        o.store(to + 128 * W * u);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (j0 + j >= a.top_k) break;
                const float s = warp_sum(dot[j]);
                if (lane == 0) part[j0 + j][warp] = s;
            }
        }
        __syncthreads();
        if (threadIdx.x < a.top_k) {
            float s = 0.0f;
            for (int w = 0; w < 4; ++w) s += part[threadIdx.x][w];
            const int64_t pair = t * a.top_k + threadIdx.x;
            a.dweights[pair] = s;
            if (a.pair_of) {
                const int p = a.pos[pair];
                if (p >= 0 && p < a.y_rows) a.pair_of[p] = (int32_t)pair;
            }
        }
        __syncthreads();
    }
    pdl_trigger();
    if (a.slice) {
        __shared__ uint32_t named[FEW_ROWS / 32];
        const int lo = blockIdx.x * a.slice, hi = min((int)a.y_rows, lo + a.slice), pairs = (int)a.tokens * a.top_k;
        const int64_t row_bytes = a.hidden * (int64_t)sizeof(T);
        const bool wide = rows_wide(a.dy, row_bytes);
        if (threadIdx.x < FEW_ROWS / 32) named[threadIdx.x] = 0u;
        __syncthreads();
        for (int i = threadIdx.x; i < pairs; i += 128) {
            const int p = __ldg(a.pos + i);
            if (p >= lo && p < hi) atomicOr(&named[(p - lo) >> 5], 1u << ((p - lo) & 31));
        }
        __syncthreads();
        for (int r = lo; r < hi; ++r)
            if (!((named[(r - lo) >> 5] >> ((r - lo) & 31)) & 1u))
                zero_row(reinterpret_cast<uint8_t*>(a.dy) + r * row_bytes, row_bytes, wide, threadIdx.x, 128);
    }
}

// Zeros in the rows of dy that no position names, where the kernel above does not
// look them over itself (with few pairs it does: one launch and no scratch). pair_of
// is not set up before: where a row is not named it holds anything, but then the pair
// it tells of, if there is one, has another position. Bound by the rows it writes
// (28672 of 32768 x 7168 bf16: 73 us, 5.6 TB/s); with every row named it reads 8
// bytes a row, and since it starts early costs 1.7 us behind the kernel before it
// (both 39.4 us at 2049 x 6 x 4096 bf16; zeros in all of dy beforehand would write it
// twice). A warp takes 8 rows.
__global__ void __launch_bounds__(128) k_zero_unnamed(const int32_t* pair_of, const int32_t* pos, int pairs, int64_t rows,
                                                      int64_t row_bytes, uint8_t* dy) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const bool wide = rows_wide(dy, row_bytes);
    for (int64_t r0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * 8; r0 < rows; r0 += (int64_t)gridDim.x * 32) {
        const int64_t r = r0 + lane;
        bool bare = false;
        if (lane < 8 && r < rows) {
            const int32_t pair = pairs > 0 ? pair_of[r] : -1;
            bare = pair < 0 || pair >= pairs || pos[pair] != r;
        }
        for (unsigned todo = __ballot_sync(FULL, bare); todo; todo &= todo - 1) {
            zero_row(dy + (r0 + __ffs(todo) - 1) * row_bytes, row_bytes, wide, lane, 32);
        }
    }
}

// Columns of an access: eight where a row's columns and the tensors' starts allow
// 16-byte ones, two where they are even, else one.
int col_width(int64_t hidden, uintptr_t starts, size_t most) {
    if (hidden % 8 == 0 && (starts & 15u) == 0) return 8;
    return hidden % 2 == 0 && (starts & (2 * most - 1)) == 0 ? 2 : 1;
}
// As many threads as a row has accesses, 128 at most; few tokens get several CTAs
// each.
template <class TY, class TO, int W, int U>
cudaError_t launch_combine_as(const CombineArgs& a, cudaStream_t st) {
    const int64_t per_row = (a.hidden + W * U - 1) / (W * U), sms = sm_count();
    const unsigned threads = per_row >= 128 ? 128u : (unsigned)((per_row + 31) / 32 * 32);
    const int64_t shares = (per_row + threads - 1) / threads, want = (4 * sms + a.tokens - 1) / a.tokens;
    const int64_t gx = a.tokens < 16 * sms ? a.tokens : 16 * sms, gy = want < shares ? want : shares;
    const dim3 grid((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535));
    k_moe_combine<TY, TO, W, U><<<grid, threads, 0, st>>>(a);
    return cudaGetLastError();
}
template <class TY, class TO>
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st) {
    const size_t most = sizeof(TY) > sizeof(TO) ? sizeof(TY) : sizeof(TO);
    switch (col_width(a.hidden, (uintptr_t)a.y | (uintptr_t)a.residual | (uintptr_t)a.out, most)) {
        case 8: return launch_combine_as<TY, TO, 8, 1>(a, st);
        case 2: return launch_combine_as<TY, TO, 2, 4>(a, st);
        default: return launch_combine_as<TY, TO, 1, 4>(a, st);
    }
}
template <class TY>
cudaError_t combine_out(const CombineArgs& a, bq_dtype out, cudaStream_t st) {
    if (out == BQ_F32) return launch_combine<TY, float>(a, st);
    if (out == BQ_F16) return launch_combine<TY, __half>(a, st);
    return launch_combine<TY, __nv_bfloat16>(a, st);
}
template <class T>
cudaError_t launch_combine_bwd(CombineBwdArgs a, bool look_over, cudaStream_t st) {
    const int64_t most = (int64_t)sm_count() * 16, share = look_over ? (a.y_rows + 7) / 8 : 0;   // (8 rows a CTA)
    const int64_t want = a.tokens > share ? a.tokens : share;
    const unsigned grid = (unsigned)(want < most ? want : most);
    a.slice = look_over ? (int)((a.y_rows + grid - 1) / grid) : 0;
    switch (col_width(a.hidden, (uintptr_t)a.dout | (uintptr_t)a.y | (uintptr_t)a.dy, sizeof(T))) {
        case 8: k_moe_combine_bwd<T, 8, 1><<<grid, 128, 0, st>>>(a); break;
        case 2: k_moe_combine_bwd<T, 2, 4><<<grid, 128, 0, st>>>(a); break;
        default: k_moe_combine_bwd<T, 1, 4><<<grid, 128, 0, st>>>(a); break;
    }
    return cudaGetLastError();
}
cudaError_t launch_zero_unnamed(const CombineBwdArgs& a, size_t es, cudaStream_t st) {
    const int64_t row_bytes = a.hidden * (int64_t)es, need = (a.y_rows + 31) / 32, most = 16ll * sm_count();
    const int pairs = (int)(a.tokens * a.top_k);
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (pairs > 0)
        return launch_pdl(k_zero_unnamed, grid, 128, 0, st, (const int32_t*)a.pair_of, a.pos, pairs, a.y_rows, row_bytes,
                          (uint8_t*)a.dy);
    k_zero_unnamed<<<grid, 128, 0, st>>>(a.pair_of, a.pos, pairs, a.y_rows, row_bytes, (uint8_t*)a.dy);
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
    const bool by_score = group_top == BQ_GROUP_SCORES;
    if (by_score) group_top = BQ_GROUP_TWO_BEST;
    if (group_top < 1 || group_top > 2 || top_k > top_groups * (experts / n_groups)) return BQ_ERR_INVALID_ARG;
    if (!pairs_fit(tokens, top_k)) return BQ_ERR_INVALID_ARG;
    if (tokens == 0) return BQ_OK;
    if (!logits || !ids || !weights) return BQ_ERR_INVALID_ARG;
    if (misaligned(logits, type_mask(dtype)) || misaligned(bias, 3) || misaligned(ids, 3) || misaligned(weights, 3))
        return BQ_ERR_MISALIGNED;
    RouteArgs a{logits, bias, tokens, experts, top_k, n_groups, top_groups, group_top, score == BQ_SCORE_SIGMOID,
                renormalize != 0, 0, bias || (by_score && n_groups > 1), 0, 0, scale, ids, weights};
    while (2 * a.sum_lanes < top_k) a.sum_lanes = a.sum_lanes ? 2 * a.sum_lanes : 1;
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
    GroupArgs a{ids, (int)(tokens * top_k), 0, first_expert, n_experts, 0, make_fastdiv((uint32_t)top_k), offsets, rows, pos};
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
    CombineArgs a{y, pos, weights, residual, out, tokens, y_rows, hidden, top_k};
    cudaStream_t st = (cudaStream_t)stream;
    if (y_dtype == BQ_F32) return from(combine_out<float>(a, out_dtype, st));
    if (y_dtype == BQ_F16) return from(combine_out<__half>(a, out_dtype, st));
    return from(combine_out<__nv_bfloat16>(a, out_dtype, st));
}

static bq_status combine_backward(const void* dout, const void* y, bq_dtype dtype, int64_t y_rows, int64_t hidden,
                                  const int32_t* pos, const float* weights, int64_t tokens, int32_t top_k, void* dy,
                                  float* dweights, bool whole, void* ws, size_t ws_bytes, void* stream) {
    if (!float_type(dtype)) return BQ_ERR_UNSUPPORTED;
    if (y_rows < 0 || hidden < 0 || hidden >= (1ll << 31) || tokens < 0 || top_k < 1 || top_k > 32 ||
        !pairs_fit(tokens, top_k))
        return BQ_ERR_INVALID_ARG;
    const bool zeros = whole && y_rows > 0 && hidden > 0;
    if (whole && y_rows >= (1ll << 31)) return BQ_ERR_INVALID_ARG;
    if (tokens == 0 && !zeros) return BQ_OK;
    if (tokens > 0 && ((!dout && hidden > 0) || (!y && y_rows > 0 && hidden > 0) || !pos || !weights || !dweights))
        return BQ_ERR_INVALID_ARG;
    if (!dy && y_rows > 0 && hidden > 0) return BQ_ERR_INVALID_ARG;
    const size_t scratch = zeros ? bq_moe_combine_backward_workspace_size(y_rows, tokens, top_k) : 0;
    if (scratch > 0 && (!ws || ws_bytes < scratch)) return BQ_ERR_INVALID_ARG;
    const uintptr_t m = type_mask(dtype);
    if (misaligned(dout, m) || misaligned(y, m) || misaligned(dy, m) || misaligned(pos, 3) || misaligned(weights, 3) ||
        misaligned(dweights, 3) || misaligned(ws, 3))
        return BQ_ERR_MISALIGNED;
    CombineBwdArgs a{dout, y, pos, weights, dy, dweights, scratch > 0 ? (int32_t*)ws : nullptr, tokens, y_rows, hidden, top_k, 0};
    cudaStream_t st = (cudaStream_t)stream;
    const bool few = zeros && few_named(y_rows, tokens * top_k);
    cudaError_t e = cudaSuccess;
    if (tokens > 0 || few)
        e = dtype == BQ_F32 ? launch_combine_bwd<float>(a, few, st)
            : dtype == BQ_F16 ? launch_combine_bwd<__half>(a, few, st)
                              : launch_combine_bwd<__nv_bfloat16>(a, few, st);
    if (e == cudaSuccess && zeros && !few) e = launch_zero_unnamed(a, dtype == BQ_F32 ? 4 : 2, st);
    return from(e);
}

extern "C" bq_status bq_moe_combine_backward(const void* dout, const void* y, bq_dtype dtype, int64_t y_rows,
                                             int64_t hidden, const int32_t* pos, const float* weights, int64_t tokens,
                                             int32_t top_k, void* dy, float* dweights, void* stream) {
    return combine_backward(dout, y, dtype, y_rows, hidden, pos, weights, tokens, top_k, dy, dweights, false, nullptr, 0, stream);
}

extern "C" size_t bq_moe_combine_backward_workspace_size(int64_t y_rows, int64_t tokens, int32_t top_k) {
    if (y_rows <= 0 || y_rows >= (1ll << 31) || tokens <= 0 || top_k < 1 || !pairs_fit(tokens, top_k)) return 0;
    return few_named(y_rows, tokens * top_k) ? 0 : (size_t)y_rows * sizeof(int32_t);
}

extern "C" bq_status bq_moe_combine_backward_whole(const void* dout, const void* y, bq_dtype dtype, int64_t y_rows,
                                                   int64_t hidden, const int32_t* pos, const float* weights, int64_t tokens,
                                                   int32_t top_k, void* dy, float* dweights, void* ws, size_t ws_bytes,
                                                   void* stream) {
    return combine_backward(dout, y, dtype, y_rows, hidden, pos, weights, tokens, top_k, dy, dweights, true, ws, ws_bytes, stream);
}
