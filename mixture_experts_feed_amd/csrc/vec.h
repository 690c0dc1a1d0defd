// Vectors of 1, 4 or 8 consecutive values widened to fp32, and back (shared by
// the elementwise and row kernels).
#pragma once

#include "common.h"

namespace inkling {

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
typedef float f32x2_v __attribute__((ext_vector_type(2)));

// two fp32 -> bf16, nearest even, NaN kept (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const f32x2_v v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_v));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a vector as loaded, V values of TE
template <typename TE, int V>
struct RawOf;
template <>
struct RawOf<bf16_t, 1> { using type = bf16_t; };
template <>
struct RawOf<bf16_t, 8> { using type = uint4; };
template <>
struct RawOf<float, 1> { using type = float; };
template <>
struct RawOf<float, 4> { using type = float4; };
template <typename TE, int V>
using Raw = typename RawOf<TE, V>::type;

template <typename TE, int V>
__device__ __forceinline__ Raw<TE, V> load_raw(const TE* p) {
    return *reinterpret_cast<const Raw<TE, V>*>(p);
}

__device__ __forceinline__ void widen(bf16_t r, float* v) { v[0] = bf16_to_f32(r); }
__device__ __forceinline__ void widen(float r, float* v) { v[0] = r; }
__device__ __forceinline__ void widen(const float4& r, float* v) {
    v[0] = r.x;
    v[1] = r.y;
    v[2] = r.z;
    v[3] = r.w;
}
__device__ __forceinline__ void widen(const uint4& r, float* v) {
    v[0] = bf16_lo(r.x);
    v[1] = bf16_hi(r.x);
    v[2] = bf16_lo(r.y);
    v[3] = bf16_hi(r.y);
    v[4] = bf16_lo(r.z);
    v[5] = bf16_hi(r.z);
    v[6] = bf16_lo(r.w);
    v[7] = bf16_hi(r.w);
}

// V fp32 values rounded once and stored
template <typename TE, int V>
__device__ __forceinline__ void store_vec(TE* p, const float* v) {
    if constexpr (sizeof(TE) == 4) {
        if constexpr (V == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else {
        if constexpr (V == 1) {
            *p = (bf16_t)(pack_bf16x2(v[0], 0.f) & 0xFFFFu);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 8)
                *reinterpret_cast<uint4*>(p + i) =
                    make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                               pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
        }
    }
}

// sum over the lanes of a wave, in a fixed order; every lane gets it
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

}  // namespace inkling
