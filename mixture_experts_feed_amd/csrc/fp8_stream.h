// The forward product of fp8_tiles.h for experts with few rows, whose weights are
// read once: a workgroup takes BN output columns of one expert and all of its rows,
// up to 64 at a time.  The waves share out the reduction by blocks of 128 (wave w
// takes blocks w, w + NW, ...), so each streams its own weights straight into
// registers, without LDS or barriers, two blocks ahead; the rows come from the caches.
// The waves' sums are added in LDS, in the order of the waves, and stored once.
// HBM bounds it: W is read once and little else moves.
#pragma once

#include "fp8_common.h"

namespace inkling {

namespace {

// offsets[0..e + 1] made safe: the rows of expert e.  Whole workgroup.
template <int THREADS>
__device__ __forceinline__ void expert_rows(const Fp8Args& a, int e, int32_t* scratch, int& begin, int& end) {
    if (a.offsets == nullptr) {
        begin = 0;
        end = a.rows;
        return;
    }
    // each offset is raised to the largest before it
    int top = 0;
    for (int i = threadIdx.x; i <= e; i += THREADS) top = max(top, a.offsets[i]);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = max(top, __shfl_xor(top, d));
    if (lane_id() == 0) scratch[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) top = max(top, scratch[w]);
    begin = __builtin_amdgcn_readfirstlane(min(top, a.rows));
    end = __builtin_amdgcn_readfirstlane(min(max(top, scalar_load(a.offsets + e + 1)), a.rows));
}

template <int BN, int NW, bool EXACT>
__global__ __launch_bounds__(NW * 64, 2) void fp8_stream_kernel(const Fp8Args a) {
    constexpr int THREADS = NW * 64;
    constexpr int MAXM = 64;   // rows at a time
    __shared__ __attribute__((aligned(16))) float part[NW][MAXM][BN + 4];
    __shared__ int32_t scratch[NW];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rl = lane & 15, g = lane >> 4;
    const int ntn = (a.N + BN - 1) / BN;
    const int e = blockIdx.x / ntn, n0 = (blockIdx.x - e * ntn) * BN;
    int begin, end;
    expert_rows<THREADS>(a, e, scratch, begin, end);
    if (begin >= end) return;   // the same for the workgroup
    const int kb = (a.K + kQBlock - 1) / kQBlock;
    const uint8_t* w = a.weight + (size_t)e * a.N * a.K;
    const float* ws = a.weight_scale + ((size_t)e * ((a.N + kQBlock - 1) / kQBlock) + n0 / kQBlock) * kb;
    w += (size_t)n0 * a.K;
    const bool tail = (a.K % kQBlock) != 0;

    // FM blocks of 16 rows by FN of 16 columns from n0 + c0
    auto pass = [&](auto FM_, auto FN_, int c0, int row0, int valid) __attribute__((always_inline)) {
        constexpr int FM = decltype(FM_)::value, FN = decltype(FN_)::value;
        uint32_t w_off[FN];   // columns past the end: the last one
#pragma unroll
        for (int i = 0; i < FN; ++i) w_off[i] = (uint32_t)(min(n0 + c0 + 16 * i + rl, a.N - 1) - n0) * a.K + 16 * g;
        const uint8_t* x[FM];
        const float* xs[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            int row = row0 + min(16 * j + rl, valid - 1);   // rows past the end: the last one
            if (a.row_index != nullptr) row = max(0, min(a.row_index[row], a.x_rows - 1));
            x[j] = a.x + (size_t)row * a.K + 16 * g;
            xs[j] = a.x_scale + (size_t)row * kb;
        }
        f32x4_t acc[FN][FM];
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        struct Block {
            Frag fw[FN], fx[FM];
            float sx[FM], sw;
        };
        auto load = [&](Block& B, int b) __attribute__((always_inline)) {
            const uint32_t k0 = (uint32_t)b * kQBlock;
            if (!tail || b + 1 < kb) {
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const uint8_t* p = w + w_off[i] + k0;
                    B.fw[i].half[0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(p));
                    B.fw[i].half[1] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(p + 64));
                }
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    B.fx[j].half[0] = *reinterpret_cast<const i32x4_t*>(x[j] + k0);
                    B.fx[j].half[1] = *reinterpret_cast<const i32x4_t*>(x[j] + k0 + 64);
                }
            } else {
                // chunks past the end are zeros on both sides
                const bool in0 = (int)k0 + 16 * g < a.K, in1 = (int)k0 + 64 + 16 * g < a.K;
                const i32x4_t zero = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const uint8_t* p = w + w_off[i] + k0;
                    B.fw[i].half[0] = zero;
                    B.fw[i].half[1] = zero;
                    if (in0) B.fw[i].half[0] = *reinterpret_cast<const i32x4_t*>(p);
                    if (in1) B.fw[i].half[1] = *reinterpret_cast<const i32x4_t*>(p + 64);
                }
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    B.fx[j].half[0] = zero;
                    B.fx[j].half[1] = zero;
                    if (in0) B.fx[j].half[0] = *reinterpret_cast<const i32x4_t*>(x[j] + k0);
                    if (in1) B.fx[j].half[1] = *reinterpret_cast<const i32x4_t*>(x[j] + k0 + 64);
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j) B.sx[j] = xs[j][b];
            B.sw = scalar_load(ws + b);
        };
        auto multiply = [&](const Block& B) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const float s = B.sx[j] * B.sw;
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const f32x4_t p = block_product<EXACT>(B.fw[i], B.fx[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s, acc[i][j][r]);
                }
            }
        };
        Block b0, b1;
        if (wv < kb) load(b0, wv);
        for (int b = wv; b < kb; b += 2 * NW) {
            if (b + NW < kb) load(b1, b + NW);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b0);
            __builtin_amdgcn_sched_barrier(0);
            if (b + 2 * NW < kb) load(b0, b + 2 * NW);
            __builtin_amdgcn_sched_barrier(0);
            if (b + NW < kb) multiply(b1);
            __builtin_amdgcn_sched_barrier(0);
        }
        // (a lane holds columns 16 i + 4 g .. + 3 of row 16 j + rl)
        if (c0 == 0) __syncthreads();   // the sums of the rows before are read
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int i = 0; i < FN; ++i)
                *reinterpret_cast<f32x4_t*>(&part[wv][16 * j + rl][c0 + 16 * i + 4 * g]) = acc[i][j];
    };
    auto store = [&](int row0, int valid) __attribute__((always_inline)) {
        __syncthreads();
        constexpr int Q = BN / 4;   // four columns a thread
        for (int c = tid; c < valid * Q; c += THREADS) {
            const int m = c / Q, n = c % Q * 4;
            f32x4_t s = *reinterpret_cast<const f32x4_t*>(&part[0][m][n]);
#pragma unroll
            for (int v = 1; v < NW; ++v) s += *reinterpret_cast<const f32x4_t*>(&part[v][m][n]);
            if (n0 + n < a.N) {
                const size_t at = (size_t)(row0 + m) * a.N + n0 + n;
                if (a.out_bf16)
                    *reinterpret_cast<uint2*>(static_cast<bf16_t*>(a.out) + at) =
                        make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
                else
                    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = s;
            }
        }
    };
    constexpr std::integral_constant<int, BN / 16> all{};
    for (int row0 = begin; row0 < end; row0 += MAXM) {
        const int valid = min(MAXM, end - row0);
        if (valid <= 16) {
            pass(std::integral_constant<int, 1>{}, all, 0, row0, valid);
        } else if (valid <= 32) {
            pass(std::integral_constant<int, 2>{}, all, 0, row0, valid);
        } else if constexpr (BN <= 32) {
            pass(std::integral_constant<int, 4>{}, all, 0, row0, valid);
        } else {
            // half of the columns at a time: both need the registers
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += BN / 2)
                pass(std::integral_constant<int, 4>{}, std::integral_constant<int, BN / 32>{}, c0, row0, valid);
        }
        store(row0, valid);
    }
}

}  // namespace

}  // namespace inkling
