// Shared by the kernels of products in 8-bit floating point (e4m3, a scale for each
// block of 128): fragments, the product of one block, the caller's offsets made safe.
#pragma once

#include "common.h"
#include "vec.h"

namespace inkling {

namespace {

constexpr int kQBlock = 128;     // values that share a scale

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// A lane's part of a 16 x 128 operand block: row lane % 16, the columns 16 g .. 16 g + 15
// and 64 + 16 g .. 64 + 16 g + 15 for g = lane / 16.  (The matrix instruction only asks
// that both operands hold the same columns at the same place.)
union Frag {
    i32x8_t v;
    i32x4_t half[2];
    i32x2_t quarter[4];
};

__device__ __forceinline__ bf16x8_t fp8x8_to_bf16(const i32x2_t& w) {
    bf16x8_t r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], 1.0f, false);
        const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], 1.0f, true);
        r[4 * h] = lo[0];
        r[4 * h + 1] = lo[1];
        r[4 * h + 2] = hi[0];
        r[4 * h + 3] = hi[1];
    }
    return r;
}

// Sum over one block of 128 of a 16 x 128 by a 128 x 16 block.  The 8-bit matrix units
// add products in groups of 8 whose addends keep 13 bits below the largest one's
// leading bit (measured: 2^-14 of the largest and less is lost; groups and blocks are
// then added in fp32).  That is about 1.3e-5 of a result's size on normally
// distributed values, 1/300 of what rounding to bf16 costs, and what bf16 results take.
// EXACT: results in fp32 promise fp32 sums, so their values go through the bf16 units,
// which hold every e4m3 value and add without that loss (measured), at half the rate.
template <bool EXACT>
__device__ __forceinline__ f32x4_t block_product(const Frag& a, const Frag& b) {
    f32x4_t d = {0.f, 0.f, 0.f, 0.f};
    if constexpr (EXACT) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16(a.quarter[q]), fp8x8_to_bf16(b.quarter[q]), d, 0,
                                                        0, 0);
        return d;
    } else {
        // (both scale operands 0: the form without the instruction's own scales)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, d, 0, 0, 0, 0, 0, 0);
    }
}

// a value at an address that is the same for the whole wave, written by an earlier
// kernel only: a scalar load
template <typename V>
__device__ __forceinline__ V scalar_load(const V* p) {
    return *(const __attribute__((address_space(4))) V*)p;
}

struct Fp8Args {
    const uint8_t* weight;        // [E][N][K]
    const float* weight_scale;    // [E][ceil(N/128)][ceil(K/128)]
    const uint8_t* x;             // [x_rows][len]: rows of the other operand, len = K (forward) or N (input gradient)
    const float* x_scale;         // [x_rows][ceil(len/128)]
    const int32_t* row_index;     // row r reads x[row_index[r]] (NULL: x[r])
    const int32_t* offsets;       // [E + 1] (NULL, E == 1: all rows)
    void* out;                    // [rows][cols], cols = N or K
    int rows, x_rows, E, N, K;
    int out_bf16;
};

}  // namespace

}  // namespace inkling
