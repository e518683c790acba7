// Epilogue of the block-FP8 products: bias, activation (or gate), residual and
// the conversion of a tile's f32 sums, a warp's 32 rows x 32 columns at a time.
//
// A promotion thread holds one row of the tile, so writing from its registers
// would touch 32 rows with every instruction. The columns go through shared memory
// instead (16-byte slots swizzled by row) and come back with four lanes along a
// row, eight columns each, so that residual and results are read and written in
// whole sectors with 16-byte accesses. A lane has four rows (gated: one) in flight at
// once: with two warps per scheduler the activation's chain of instructions would
// otherwise be waited for row by row.
#pragma once

#include "bq.h"
#include "bq_act.cuh"
#include "bq_device.cuh"

namespace bq {
namespace {

struct EpiArgs {
    const void* bias;       // [n] (grouped: [n_experts, n]) or null
    const void* residual;   // rows of c's shape and type, or null
    void* c;
    void* pre;              // like c, or null
    int64_t n;              // columns of the product
    int64_t n_out;          // columns of c: n, gated n / 2
    int bias_t, c_t, act;
    int bias_vec;           // eight biases in 16-byte loads: n a multiple of 8, the start on 16 bytes
};
[[maybe_unused]] EpiArgs make_epi(int64_t n, int64_t n_out, const void* bias, int bias_t, int act, const void* residual, void* c,
                                  int c_t, void* pre) {
    EpiArgs g = {};
    g.bias = bias; g.residual = residual; g.c = c; g.pre = pre;
    g.n = n; g.n_out = n_out;
    g.bias_t = bias_t; g.c_t = c_t; g.act = act;
    g.bias_vec = n % 8 == 0 && ((uintptr_t)bias & 15u) == 0;
    return g;
}

__device__ __forceinline__ float epi_load(const void* p, int t, int64_t i) {
    if (t == BQ_F32) return reinterpret_cast<const float*>(p)[i];
    if (t == BQ_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
// Eight columns from element i of a row (16-byte aligned).
__device__ __forceinline__ void epi_load8(const void* p, int t, int64_t i, U4 (&u)[2]) {
    if (t == BQ_F32) {
        u[0] = *reinterpret_cast<const U4*>(reinterpret_cast<const float*>(p) + i);
        u[1] = *reinterpret_cast<const U4*>(reinterpret_cast<const float*>(p) + i + 4);
    } else {
        u[0] = *reinterpret_cast<const U4*>(reinterpret_cast<const uint16_t*>(p) + i);
    }
}
__device__ __forceinline__ void epi_add8(int t, const U4 (&u)[2], float (&v)[8]) {
    float r[8];
    if (t == BQ_F32) {
        float a[4], b[4];
        unpack(u[0], a);
        unpack(u[1], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) { r[j] = a[j]; r[4 + j] = b[j]; }
    } else if (t == BQ_F16) {
        unpack8<__half>(u[0], r);
    } else {
        unpack8<__nv_bfloat16>(u[0], r);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
}
// The biases of eight columns.
__device__ __forceinline__ void epi_bias8(const EpiArgs& g, int64_t i, float (&v)[8]) {
    if (g.bias_vec) {
        U4 u[2];
        epi_load8(g.bias, g.bias_t, i, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        epi_add8(g.bias_t, u, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = epi_load(g.bias, g.bias_t, i + k);
    }
}
__device__ __forceinline__ void epi_store8(void* p, int t, int64_t i, const float (&v)[8]) {
    if (t == BQ_F32) {
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) { a[j] = v[j]; b[j] = v[4 + j]; }
        st16(reinterpret_cast<float*>(p) + i, pack_vec<float>(a));
        st16(reinterpret_cast<float*>(p) + i + 4, pack_vec<float>(b));
    } else if (t == BQ_F16) {
        st16(reinterpret_cast<__half*>(p) + i, pack_vec<__half>(v));
    } else {
        st16(reinterpret_cast<__nv_bfloat16*>(p) + i, pack_vec<__nv_bfloat16>(v));
    }
}
template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&z)[N][8]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = act_value<ACT>(z[i][j]);
}
template <int N>
__device__ __forceinline__ void epi_act(int act, float (&z)[N][8]) {
    switch (act) {
        case BQ_ACT_RELU: act_all<BQ_ACT_RELU>(z); break;
        case BQ_ACT_GELU: act_all<BQ_ACT_GELU>(z); break;
        case BQ_ACT_GELU_TANH: act_all<BQ_ACT_GELU_TANH>(z); break;
        case BQ_ACT_SILU: act_all<BQ_ACT_SILU>(z); break;
        default: break;
    }
}

// This lane's values (row `lane`) into the warp's staging block of ROW4 16-byte
// slots a row, from slot `first` on: the low three bits of a slot's number are
// xored with the row's. Zeros for a row without activations.
template <int ROW4, int N>
__device__ __forceinline__ void epi_stage(float* stage, int lane, bool row_in, int first, const F2 (&v)[N], int from, int count) {
    float4* st = reinterpret_cast<float4*>(stage) + lane * ROW4;
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
        if (c >= count / 4) break;
        float4 f;
        f2_split(v[from + 2 * c], f.x, f.y);
        f2_split(v[from + 2 * c + 1], f.z, f.w);
        if (!row_in) f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        st[(first + c) ^ (lane & 7)] = f;
    }
}

// The chunk where rows of c do not start on 16 bytes: V columns of a lane (two
// where the width is even), eight values in flight. In kernels of its own (FLAT):
// beside the other form it would spill registers of the widest tiles' promotion.
template <class T, int V, int ROW4>
__device__ __forceinline__ void epi_flat(const EpiArgs& g, const float* stage, int lane, int64_t row0, int rows, int64_t col,
                                         int64_t bias_at) {
    constexpr int N = 8 / V, LANES = 32 / V;       // rows of a lane at a time; lanes along a row
    using Pack = typename std::conditional<sizeof(T) * V == 8, uint2, typename std::conditional<sizeof(T) * V == 4, uint32_t, uint16_t>::type>::type;
    const int c = V * (lane % LANES);
    if (col + c >= g.n_out) return;
    float b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = g.bias ? epi_load(g.bias, g.bias_t, bias_at + c + v) : 0.0f;
    const int64_t first = row0 * g.n_out + col + c;
    const T* res = reinterpret_cast<const T*>(g.residual);
    auto put = [&](void* p, int64_t at, const float* v) {
        Pack k;
        T* t = reinterpret_cast<T*>(&k);
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = to_out<T>(v[j]);
        *reinterpret_cast<Pack*>(reinterpret_cast<T*>(p) + at) = k;
    };
#pragma unroll 1
    for (int r0 = lane / LANES; r0 < rows; r0 += 8) {     // (V rows of a warp a step, N steps)
        Pack raw[N];
        float z[1][8];
        if (res) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (r0 + V * i < rows) raw[i] = *reinterpret_cast<const Pack*>(res + first + (r0 + V * i) * g.n_out);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = r0 + V * i;
            const float* s = stage + r * 4 * ROW4 + 4 * ((c >> 2) ^ (r & 7)) + (c & 3);
#pragma unroll
            for (int v = 0; v < V; ++v) z[0][V * i + v] = r < 32 ? s[v] + b[v] : 0.0f;
            if (g.pre && r < rows) put(g.pre, first + r * g.n_out, &z[0][V * i]);
        }
        epi_act(g.act, z);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (r0 + V * i >= rows) break;
            if (res) {
#pragma unroll
                for (int v = 0; v < V; ++v) z[0][V * i + v] += (float)reinterpret_cast<const T*>(&raw[i])[v];
            }
            put(g.c, first + (r0 + V * i) * g.n_out, &z[0][V * i]);
        }
    }
}

// One staged chunk of a warp, whose rows are row0 + 0 .. of c, `rows` of them.
// Plain: the columns col .. col + 31. Gated: the gate's columns col .. col + 15,
// then the other half's. bias_at: the place of column col in the bias array.
// Rows of the staging block are ROW4 16-byte slots apart; a lane has ROWS rows in
// flight, as its registers allow.
template <bool GATED, bool FLAT, int ROWS, int ROW4>
__device__ __forceinline__ void epi_chunk(const EpiArgs& g, const float* stage, int lane, int64_t row0, int rows, int64_t col,
                                          int64_t bias_at) {
    const float4* st = reinterpret_cast<const float4*>(stage);
    // Lanes along a row; ROWS rows of a lane at a time.
    constexpr int LANES = GATED ? 2 : 4, RSTEP = 32 / LANES, N = ROWS;
    if constexpr (!FLAT) {
        const int c = lane % LANES;
        const int64_t j = col + 8 * c;
        if (!GATED && j >= g.n_out) return;        // (gated widths are multiples of 128)
#pragma unroll 1
        for (int r0 = lane / LANES; r0 < rows; r0 += N * RSTEP) {
            U4 res[N][2];
            if (!GATED && g.residual) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (r0 + i * RSTEP < rows) epi_load8(g.residual, g.c_t, (row0 + r0 + i * RSTEP) * g.n_out + j, res[i]);
            }
            float z[N][8], u[GATED ? N : 1][8];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = r0 + i * RSTEP;
                const float4 a = st[r * ROW4 + ((2 * c) ^ (r & 7))], b = st[r * ROW4 + ((2 * c + 1) ^ (r & 7))];
                z[i][0] = a.x; z[i][1] = a.y; z[i][2] = a.z; z[i][3] = a.w;
                z[i][4] = b.x; z[i][5] = b.y; z[i][6] = b.z; z[i][7] = b.w;
                if constexpr (GATED) {
                    const float4 d = st[r * ROW4 + ((4 + 2 * c) ^ (r & 7))], e = st[r * ROW4 + ((5 + 2 * c) ^ (r & 7))];
                    u[i][0] = d.x; u[i][1] = d.y; u[i][2] = d.z; u[i][3] = d.w;
                    u[i][4] = e.x; u[i][5] = e.y; u[i][6] = e.z; u[i][7] = e.w;
                }
            }
            if (g.bias) {
                if constexpr (GATED) {
                    // One by one: vectors of both halves' biases beside the sums not
                    // yet staged would spill registers of the promotion loop.
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float b = epi_load(g.bias, g.bias_t, bias_at + 8 * c + k);
                        const float d = epi_load(g.bias, g.bias_t, bias_at + g.n_out + 8 * c + k);
#pragma unroll
                        for (int i = 0; i < N; ++i) { z[i][k] += b; u[i][k] += d; }
                    }
                } else {
                    float bz[8];
                    epi_bias8(g, bias_at + 8 * c, bz);
#pragma unroll
                    for (int i = 0; i < N; ++i)
#pragma unroll
                        for (int k = 0; k < 8; ++k) z[i][k] += bz[k];
                }
            }
            if (!GATED && g.pre) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (r0 + i * RSTEP < rows) epi_store8(g.pre, g.c_t, (row0 + r0 + i * RSTEP) * g.n_out + j, z[i]);
            }
            epi_act(g.act, z);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (GATED) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[i][k] *= u[i][k];
                } else {
                    if (g.residual) epi_add8(g.c_t, res[i], z[i]);
                }
                if (r0 + i * RSTEP < rows) epi_store8(g.c, g.c_t, (row0 + r0 + i * RSTEP) * g.n_out + j, z[i]);
            }
        }
    } else {
        const bool even = g.n_out % 2 == 0;
        if (g.c_t == BQ_F32) {
            if (even) epi_flat<float, 2, ROW4>(g, stage, lane, row0, rows, col, bias_at);
            else epi_flat<float, 1, ROW4>(g, stage, lane, row0, rows, col, bias_at);
        } else if (g.c_t == BQ_F16) {
            if (even) epi_flat<__half, 2, ROW4>(g, stage, lane, row0, rows, col, bias_at);
            else epi_flat<__half, 1, ROW4>(g, stage, lane, row0, rows, col, bias_at);
        } else {
            if (even) epi_flat<__nv_bfloat16, 2, ROW4>(g, stage, lane, row0, rows, col, bias_at);
            else epi_flat<__nv_bfloat16, 1, ROW4>(g, stage, lane, row0, rows, col, bias_at);
        }
    }
}

// A tile's columns of one warp: acc holds two runs of SW columns of this lane's
// row; plain: consecutive ones from column col; gated: from col of each half.
// They are staged COLS at a time: consecutive ones, or half as many of each run. The sums still in registers beside the epilogue's code cost the
// promotion loop spilled registers, so as many leave at once as the staging holds.
template <int SW>
struct EpiPlan {
    static constexpr int COLS = SW == 64 ? 64 : 32;
    static constexpr uint32_t WARP_BYTES = 32 * COLS * 4;
};
template <int SW, bool GATED, bool FLAT>
__device__ __forceinline__ void epi_tile(const EpiArgs& g, float* stage, int lane, int64_t row0, int rows, int64_t col,
                                         int64_t bias_at, bool row_in, const F2 (&acc)[SW]) {
    constexpr int COLS = EpiPlan<SW>::COLS, ROW4 = COLS / 4;      // staged columns
#pragma unroll
    for (int part = 0; part < 2 * SW / COLS; ++part) {
        if constexpr (GATED) {
            // 16 columns of the gate, the same 16 of the other half, and so on.
#pragma unroll
            for (int c = 0; c < COLS / 32; ++c) {
                epi_stage<ROW4>(stage, lane, row_in, 8 * c, acc, part * COLS / 4 + 8 * c, 16);
                epi_stage<ROW4>(stage, lane, row_in, 8 * c + 4, acc, SW / 2 + part * COLS / 4 + 8 * c, 16);
            }
        } else {
            epi_stage<ROW4>(stage, lane, row_in, 0, acc, part * COLS / 2, COLS);
        }
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < COLS / 32; ++c) {
            const int64_t at = col + (GATED ? 16 : 32) * (part * (COLS / 32) + c);
            if (at < g.n_out)                           // uniform over the warp
                epi_chunk<GATED, FLAT, GATED ? 1 : SW < 64 ? 2 : 4, ROW4>(g, stage + 32 * c, lane, row0, rows, at, bias_at + (at - col));
        }
        __syncwarp();                                   // read before the next part is staged
    }
}

}  // namespace
}  // namespace bq
