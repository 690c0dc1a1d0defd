// Shared by the kernels of products in 8-bit floating point (e4m3, a scale for each
// block of 128): fragments, the product of one block, the caller's offsets made safe.
#pragma once

#include <type_traits>

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
// then added in fp32).  That is about 1.4e-5 of a result's size on normally
// distributed values (rms; tested against the products' cut bits), less than 1/100 of what
// rounding to bf16 costs, and what bf16 results take.
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
    int tile_rows;                // rows of a tile (fp8_tiles.h), a multiple of 64
};

constexpr int kMaxFp8Groups = 512;

// The experts' rows and row tiles of bm, found from the caller's offsets by the whole
// workgroup: offs[0 .. E] clamped to [0, rows], each at least the largest before it;
// first[e] = row tiles of the experts before e.  Ends with a barrier.
template <int THREADS>
__device__ __forceinline__ void plan_experts(const Fp8Args& a, int bm, int32_t* offs, int32_t* first) {
    constexpr int PER = kMaxFp8Groups / THREADS, NW = THREADS / kWave;
    static_assert(PER >= 1 && PER * THREADS == kMaxFp8Groups, "a thread takes PER experts");
    __shared__ int32_t wave_max[NW], wave_sum[NW];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    if (a.offsets == nullptr) {
        if (tid == 0) {
            offs[0] = first[0] = 0;
            offs[1] = a.rows;
            first[1] = (a.rows + bm - 1) / bm;
        }
        __syncthreads();
        return;
    }
    const int start = max(0, min(a.offsets[0], a.rows));
    int end[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        end[i] = e < a.E ? max(0, min(a.offsets[e + 1], a.rows)) : 0;
    }
    end[0] = max(end[0], start);
#pragma unroll
    for (int i = 1; i < PER; ++i) end[i] = max(end[i], end[i - 1]);
    int top = end[PER - 1];   // running maximum over the threads
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(top, d);
        if (lane >= d) top = max(top, o);
    }
    if (lane == kWave - 1) wave_max[wv] = top;
    __syncthreads();
    int before = start;
    for (int w = 0; w < wv; ++w) before = max(before, wave_max[w]);
    const int prev = __shfl_up(top, 1);
    if (lane > 0) before = max(before, prev);
    int tiles[PER], sum = 0, begin = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        end[i] = max(end[i], before);
        tiles[i] = tid * PER + i < a.E ? (end[i] - begin + bm - 1) / bm : 0;
        begin = end[i];
        sum += tiles[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) wave_sum[wv] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < wv; ++w) at += wave_sum[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        at += tiles[i];
        if (e < a.E) {
            offs[e + 1] = end[i];
            first[e + 1] = at;
        }
    }
    if (tid == 0) {
        offs[0] = start;
        first[0] = 0;
    }
    __syncthreads();
}

// The last expert whose first row tile is not after rt.  Whole waves.
__device__ __forceinline__ int expert_of(const int32_t* first, int E, int rt) {
    int count = 0;
    for (int c = 0; c < E; c += kWave) {
        const int e = c + lane_id();
        count += __popcll(__ballot(e < E && first[min(e, E)] <= rt));
    }
    return __builtin_amdgcn_readfirstlane(count - 1);
}

typedef __attribute__((address_space(3))) void fp8_lds_t;
typedef const __attribute__((address_space(1))) void fp8_glb_t;
typedef __attribute__((address_space(3))) i32x2_t fp8_lds_i32x2_t;

// what lanes past an end load
__device__ uint4 fp8_zero_chunk = {0u, 0u, 0u, 0u};

constexpr int kLoadOnce = 2;   // cache policy of loads that nothing reads again (non-temporal)
template <int POLICY>
__device__ __forceinline__ void copy16_to_lds(const void* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds((fp8_glb_t*)src, (fp8_lds_t*)dst, 16, 0, POLICY);
}

// s_waitcnt vmcnt(N) and lgkmcnt(0), each alone
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4)); }
__device__ __forceinline__ void barrier_only() { __asm__ volatile("s_barrier" ::: "memory"); }

template <int B, int E, typename F>
__device__ __forceinline__ void static_for8(F&& f) {
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for8<B + 1, E>(f);
    }
}

}  // namespace

}  // namespace inkling
