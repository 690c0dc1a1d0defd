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

// v from the lane that a DPP control names (all of them stay inside 16 lanes)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// sum over G neighbouring lanes (8, 16, 32 or 64), in a fixed order; every lane
// gets it.  Up to 16 lanes through DPP: neighbours, pairs, then mirrored halves
// (each step adds two values that are equal over the lanes of a half, so the
// mirror is as good as an xor); beyond through LDS lane permutes.
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
    static_assert(G == 8 || G == 16 || G == 32 || G == 64, "lanes of a group");
    v += dpp<0xB1>(v);               // quad_perm [1, 0, 3, 2]
    v += dpp<0x4E>(v);               // quad_perm [2, 3, 0, 1]
    v += dpp<0x141>(v);              // row_half_mirror
    if constexpr (G >= 16) v += dpp<0x140>(v);   // row_mirror
    if constexpr (G >= 32) v += __shfl_xor(v, 16);
    if constexpr (G >= 64) v += __shfl_xor(v, 32);
    return v;
}

}  // namespace inkling
