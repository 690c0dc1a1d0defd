// Vectors of consecutive values widened to fp32, and back (shared by the
// elementwise and row kernels).
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

// V values of TE as loaded: 2, 8 or 16 bytes (fp32: 4, 8 or 16)
template <int BYTES>
struct RawBytes;
template <>
struct RawBytes<2> { typedef uint16_t type; };
template <>
struct RawBytes<4> { typedef uint32_t type; };
template <>
struct RawBytes<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <>
struct RawBytes<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <typename TE, int V>
using Raw = typename RawBytes<V * (int)sizeof(TE)>::type;

// NT: past the caches (data that is larger than they are, read or written once)
template <typename R, bool NT>
__device__ __forceinline__ R get(const void* p) {
    if constexpr (NT) return __builtin_nontemporal_load(static_cast<const R*>(p));
    else return *static_cast<const R*>(p);
}
template <bool NT, typename R>
__device__ __forceinline__ void put(void* p, const R& v) {
    if constexpr (NT) __builtin_nontemporal_store(v, static_cast<R*>(p));
    else *static_cast<R*>(p) = v;
}

// values of a raw vector as fp32
template <typename TE, int V>
__device__ __forceinline__ void widen(const Raw<TE, V>& r, float* v) {
    if constexpr (V == 1) {
        if constexpr (sizeof(TE) == 2) v[0] = bf16_to_f32((bf16_t)r);
        else v[0] = __uint_as_float(r);
    } else {
        constexpr int W = V * (int)sizeof(TE) / 4;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(TE) == 2) {
                v[2 * i] = bf16_lo(r[i]);
                v[2 * i + 1] = bf16_hi(r[i]);
            } else {
                v[i] = __uint_as_float(r[i]);
            }
        }
    }
}

// V fp32 values, rounded once to TE
template <typename TE, int V>
__device__ __forceinline__ Raw<TE, V> narrow(const float* v) {
    if constexpr (V == 1) {
        if constexpr (sizeof(TE) == 2) return (uint16_t)(pack_bf16x2(v[0], 0.f) & 0xFFFFu);
        else return __float_as_uint(v[0]);
    } else {
        Raw<TE, V> r;
        constexpr int W = V * (int)sizeof(TE) / 4;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(TE) == 2) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            else r[i] = __float_as_uint(v[i]);
        }
        return r;
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
