// Epilogue of the block-FP8 products: bias, activation (or gate), residual and
// the conversion of a tile's f32 sums, a warp's 32 rows x 32 columns at a time.
//
// A promotion thread holds one row of the tile, so writing from its registers
// would touch 32 rows with every instruction. The 32 x 32 block goes through
// 4 KB of shared memory instead (16-byte slots swizzled by row: no bank
// conflicts either way) and comes back with eight lanes along a row, so that
// bias, residual and results are read and written in whole sectors, and the
// activation's code stands once per chunk instead of once per register.
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
    int vec;                // n_out a multiple of 4: vectors of four columns
};
constexpr uint32_t EPI_WARP_BYTES = 32 * 32 * 4;

__device__ __forceinline__ float epi_load(const void* p, int t, int64_t i) {
    if (t == BQ_F32) return reinterpret_cast<const float*>(p)[i];
    if (t == BQ_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
// Four columns from element i of a row; `left` of them exist.
__device__ __forceinline__ void epi_load4(const void* p, int t, int64_t i, int left, int vec, float (&v)[4]) {
    if (vec) {
        if (t == BQ_F32) {
            const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
            v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
            if (t == BQ_F16) { unpack_f16x2(u.x, v[0], v[1]); unpack_f16x2(u.y, v[2], v[3]); }
            else { unpack_bf16x2(u.x, v[0], v[1]); unpack_bf16x2(u.y, v[2], v[3]); }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? epi_load(p, t, i + j) : 0.0f;
}
__device__ __forceinline__ void epi_store4(void* p, int t, int64_t i, int left, int vec, const float (&v)[4]) {
    if (vec) {
        if (t == BQ_F32)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) =
                t == BQ_F16 ? make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]))
                            : make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j >= left) break;
        if (t == BQ_F32) reinterpret_cast<float*>(p)[i + j] = v[j];
        else if (t == BQ_F16) reinterpret_cast<__half*>(p)[i + j] = __float2half_rn(v[j]);
        else reinterpret_cast<__nv_bfloat16*>(p)[i + j] = __float2bfloat16_rn(v[j]);
    }
}
__device__ __forceinline__ void epi_act4(int act, float (&z)[4]) {
    switch (act) {
        case BQ_ACT_RELU:
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = act_value<BQ_ACT_RELU>(z[j]);
            break;
        case BQ_ACT_GELU:
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = act_value<BQ_ACT_GELU>(z[j]);
            break;
        case BQ_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = act_value<BQ_ACT_GELU_TANH>(z[j]);
            break;
        case BQ_ACT_SILU:
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = act_value<BQ_ACT_SILU>(z[j]);
            break;
        default: break;
    }
}

// One chunk of a warp: v holds this lane's row (row0 + lane of c). Plain: the
// columns col .. col + 31. Gated: the gate's columns col .. col + 15, then the
// other half's. `rows` of the 32 rows exist. bias_at: the first column's place
// in the bias array.
template <bool GATED>
__device__ __forceinline__ void epi_chunk(const EpiArgs& g, float* stage, int lane, int64_t row0, int rows, int64_t col,
                                          int64_t bias_at, const float (&v)[32]) {
    if (col >= g.n_out) return;                     // uniform over the warp
    float4* st = reinterpret_cast<float4*>(stage);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        st[lane * 8 + (c ^ (lane & 7))] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    __syncwarp();
    constexpr int LANES = GATED ? 4 : 8;            // lanes along a row
    const int c = lane % LANES;
    const int64_t j = col + 4 * c;
    const int left = (int)min((int64_t)4, g.n_out - j);
    if (left > 0) {
        const int vec = g.vec;
        float b0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (g.bias) {
            epi_load4(g.bias, g.bias_t, bias_at + 4 * c, left, 0, b0);
            if (GATED) epi_load4(g.bias, g.bias_t, bias_at + g.n_out + 4 * c, left, 0, b1);
        }
#pragma unroll 2
        for (int r = lane / LANES; r < rows; r += 32 / LANES) {
            const int64_t at = (row0 + r) * g.n_out + j;
            const float4 f = st[r * 8 + (c ^ (r & 7))];
            float z[4] = {f.x + b0[0], f.y + b0[1], f.z + b0[2], f.w + b0[3]};
            float res[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (!GATED && g.residual) epi_load4(g.residual, g.c_t, at, left, vec, res);
            if (!GATED && g.pre) epi_store4(g.pre, g.c_t, at, left, vec, z);
            epi_act4(g.act, z);
            if (GATED) {
                const float4 u = st[r * 8 + ((c + 4) ^ (r & 7))];
                z[0] *= u.x + b1[0]; z[1] *= u.y + b1[1]; z[2] *= u.z + b1[2]; z[3] *= u.w + b1[3];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] += res[i];
            }
            epi_store4(g.c, g.c_t, at, left, vec, z);
        }
    }
    __syncwarp();                                   // read before the next chunk is staged
}

}  // namespace
}  // namespace bq
