// Runs of W columns of a row in registers as they lie in memory, one access each
// (f32 runs of eight: two): W = 16 bytes' worth or 8, or 2, or 1.
#pragma once

#include "bq_device.cuh"

namespace bq {

template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = U4; };

template <class T, int W>
struct Cols {
    static constexpr int BYTES = W * (int)sizeof(T), N = BYTES > 16 ? BYTES / 16 : 1;
    using Raw = typename RawOf<(BYTES > 16 ? 16 : BYTES)>::type;
    Raw raw[N];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = reinterpret_cast<const Raw*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<Raw*>(p)[i] = raw[i];
    }
    __device__ __forceinline__ void get(float (&v)[W]) const {
        if constexpr (BYTES >= 16) {
            constexpr int V = Traits<T>::VEC;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[V];
                load_vec<T>(raw[i], x);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i * V + j] = x[j];
            }
        } else if constexpr (std::is_same<T, float>::value) {
            if constexpr (W == 2) { v[0] = __uint_as_float(raw[0].x); v[1] = __uint_as_float(raw[0].y); }
            else v[0] = __uint_as_float(raw[0]);
        } else if constexpr (W == 2) {
            if constexpr (std::is_same<T, __half>::value) unpack_f16x2(raw[0], v[0], v[1]);
            else unpack_bf16x2(raw[0], v[0], v[1]);
        } else {
            float none;
            if constexpr (std::is_same<T, __half>::value) unpack_f16x2(raw[0], v[0], none);
            else unpack_bf16x2(raw[0], v[0], none);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[W]) {
        if constexpr (BYTES >= 16) {
            constexpr int V = Traits<T>::VEC;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[V];
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = v[i * V + j];
                raw[i] = pack_vec<T>(x);
            }
        } else if constexpr (std::is_same<T, float>::value) {
            if constexpr (W == 2) raw[0] = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
            else raw[0] = __float_as_uint(v[0]);
        } else {
            const float hi = W == 2 ? v[W - 1] : 0.0f;
            raw[0] = (Raw)(std::is_same<T, __half>::value ? pack_f16x2(v[0], hi) : pack_bf16x2(v[0], hi));
        }
    }
};

}  // namespace bq
