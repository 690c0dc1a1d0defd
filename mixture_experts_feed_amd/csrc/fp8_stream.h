// The forward product of fp8_tiles.h for experts with few rows, whose weights are
// read once: HBM bounds it, so the aim is to keep enough of W on its way.
//
// A task is BN output columns of one expert for up to 16 FM of its rows.  Persistent
// workgroups of NW waves, as many a CU as its LDS holds (stream_per_cu), walk the tasks
// with stride.  The waves share out the reduction by blocks of 128 (wave w takes blocks w,
// w + NW, ...).  Each wave loads its weights straight into LDS rings of its own, DEPTH
// blocks of BN x 128 deep and whole 128-byte lines at a time, and its rows into registers
// as far ahead; nobody waits for anybody until the waves' sums are added in LDS at the end
// of a task, in the order of the waves.  The loads run ahead over the end of a task, so
// that the next one's weights are on their way while the sums are added and stored.
// 128 experts of 2 rows, 6144 x 4096: 381 to 404 us (2.72 GB read, 7.0 TB/s at the median), up
// to 470 with weights in memory that other tensors had before; one expert of one row: 9.5 us,
// whose 25 MB lie in the last cache (a chain of latencies: offsets, rows, sums).  Results in
// fp32: 442 and 10.8.
#pragma once

#include "fp8_common.h"

namespace inkling {

namespace {

typedef const __attribute__((address_space(1))) i32x4_t glb_i32x4_t;

// Reads of LDS that loads have written (waited for already), by themselves: the compiler
// would wait for every load on its way before them.  Each block waits for its results.
__device__ __forceinline__ uint32_t lds_address(void* p) {
    return (uint32_t)(uintptr_t)(fp8_lds_t*)p;
}
__device__ __forceinline__ int lds_word(void* p) {
    int v;
    __asm__ volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(lds_address(p)) : "memory");
    return v;
}
// 16 bytes at p0 and p1 of each block of 16 rows of 128 bytes
__device__ __forceinline__ void lds_blocks(Frag (&f)[1], uint32_t p0, uint32_t p1) {
    __asm__ volatile(
        "ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(f[0].half[0]), "=&v"(f[0].half[1])
        : "v"(p0), "v"(p1)
        : "memory");
}
__device__ __forceinline__ void lds_blocks(Frag (&f)[4], uint32_t p0, uint32_t p1) {
    __asm__ volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
        "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
        "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(f[0].half[0]), "=&v"(f[0].half[1]), "=&v"(f[1].half[0]), "=&v"(f[1].half[1]), "=&v"(f[2].half[0]),
          "=&v"(f[2].half[1]), "=&v"(f[3].half[0]), "=&v"(f[3].half[1])
        : "v"(p0), "v"(p1)
        : "memory");
}

// A ring place of a wave: BN rows of 128 bytes of weights, then the row scales (lane m: of
// row m).
template <int BN>
constexpr int stream_slot() { return BN * kQBlock + kWave * 4; }
// blocks of 16 columns whose sums the waves join at a time
template <int BN, int FM>
constexpr int stream_joined() { return BN / 16 / FM > 0 ? BN / 16 / FM : 1; }

// LDS of a workgroup: rings, row numbers, the waves' sums, the plan and its scan; given out
// by 1280 bytes
template <int BN, int NW, int DEPTH, int FM>
constexpr int stream_lds() {
    constexpr int ring = DEPTH * NW * stream_slot<BN>(), index = NW * kWave * 4,
                  part = NW * 16 * FM * (16 * stream_joined<BN, FM>() + 4) * 4,
                  plan = 2 * (kMaxFp8Groups + 1) * 4 + 2 * NW * 4;
    return (ring + index + part + plan + 1279) / 1280 * 1280;
}
// Workgroups that a CU's LDS holds: one of 64 columns or of eight waves, three of 16 columns
// (two with 64 rows).  No more are launched: the others would start when these have ended,
// with a scan and empty rings of their own (us, four workgroups a CU of 16 columns against
// three: 14.9 / 10.9 for 50 experts of 6 rows, 2048 x 256, and 20.8 / 16.3 for 100; 19.8 /
// 15.7 for 7 of 2048 x 4096).
constexpr int kLdsBytes = 160 * 1024;
template <int BN, int NW, int DEPTH, int FM>
constexpr int stream_per_cu() {
    static_assert(stream_lds<BN, NW, DEPTH, FM>() <= kLdsBytes, "a workgroup's LDS");
    return kLdsBytes / stream_lds<BN, NW, DEPTH, FM>();
}

template <int BN, int NW, int DEPTH, int FM, bool EXACT>
__global__ __launch_bounds__(NW * 64, (NW / 4 * stream_per_cu<BN, NW, DEPTH, FM>())) void fp8_stream_kernel(const Fp8Args a) {
    constexpr int THREADS = NW * 64, BM = 16 * FM, FN = BN / 16;
    constexpr int LW = BN / 8;                    // wave loads of a block's weights (8 rows of 128 bytes each)
    constexpr int PER = LW + 2 * FM + 1;          // loads of a block: weights, rows, the rows' scales
    static_assert((DEPTH - 1) * PER < 64, "loads in flight are counted in six bits");
    static_assert(DEPTH >= 4 && DEPTH <= 8, "ring depth");
    // Weights and row scales of a place in one object: the compiler tells few apart, and
    // waits for every load on its way where it cannot.
    constexpr int SLOT = stream_slot<BN>(), RING = NW * SLOT, NONE = 16;
    __shared__ __attribute__((aligned(16))) uint8_t r0[RING], r1[RING], r2[RING], r3[RING];
    __shared__ __attribute__((aligned(16))) uint8_t r4[DEPTH > 4 ? RING : NONE], r5[DEPTH > 5 ? RING : NONE],
        r6[DEPTH > 6 ? RING : NONE], r7[DEPTH > 7 ? RING : NONE];
    auto ring = [&](auto D_) -> uint8_t* {
        constexpr int d = decltype(D_)::value;
        if constexpr (d == 0) return r0;
        else if constexpr (d == 1) return r1;
        else if constexpr (d == 2) return r2;
        else if constexpr (d == 3) return r3;
        else if constexpr (d == 4) return r4;
        else if constexpr (d == 5) return r5;
        else if constexpr (d == 6) return r6;
        else return r7;
    };
    // the next task's row_index entries (lane m: of row m)
    __shared__ __attribute__((aligned(16))) int32_t index[NW][kWave];
    // sums of the waves, RI blocks of 16 columns at a time
    constexpr int RI = stream_joined<BN, FM>(), RC = 16 * RI;
    __shared__ __attribute__((aligned(16))) float part[NW][BM][RC + 4];
    __shared__ int32_t offs[kMaxFp8Groups + 1], first[kMaxFp8Groups + 1];
    static_assert(DEPTH * RING + sizeof(index) + sizeof(part) + sizeof(offs) + sizeof(first) + 2 * NW * 4 <=
                      stream_lds<BN, NW, DEPTH, FM>(), "the LDS that the launch counts on");

    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rl = lane & 15, g = lane >> 4;
    const int ntn = (a.N + BN - 1) / BN;
    const int kb = (a.K + kQBlock - 1) / kQBlock;
    // blocks of a task for each wave, the missing ones as zeros
    const int steps = ((kb + NW - 1) / NW + DEPTH - 1) / DEPTH * DEPTH;
    plan_experts<THREADS>(a, BM, offs, first);
    const int total = first[a.E] * ntn;
    if ((int)blockIdx.x >= total) return;

    struct Task {
        int e, row0, valid, n0;
    };
    auto decode = [&](int t) {
        Task k;
        const int rt = t / ntn;
        k.e = expert_of(first, a.E, rt);
        k.row0 = __builtin_amdgcn_readfirstlane(offs[k.e] + (rt - first[k.e]) * BM);
        k.valid = __builtin_amdgcn_readfirstlane(min(BM, offs[k.e + 1] - k.row0));
        k.n0 = (t - rt * ntn) * BN;
        return k;
    };
    // ---- loads, ahead of the products ----------------------------------------------
    uint64_t zero = reinterpret_cast<uint64_t>(&fp8_zero_chunk);
    __asm__("" : "+v"(zero));
    // p or zeros, as a select of addresses: one load either way
    auto either = [&](bool in, const uint8_t* p) __attribute__((always_inline)) {
        uint64_t v = in ? reinterpret_cast<uint64_t>(p) : zero;
        __asm__("" : "+v"(v));
        return v;
    };
    const int c16 = 16 * ((lane & 7) ^ (lane >> 3));   // the lane's chunk of its 128-byte rows (place lane % 8)
    int ld_task = blockIdx.x, ld_step = 0, ld_b = wv;
    const uint8_t* w_base;
    uint32_t w_off[LW];
    const uint8_t* x_src[FM];
    const float* s_src;
    // The row_index entries of the task after, loaded a whole task ahead, are in LDS:
    // at least DEPTH blocks are loaded and waited for in between.
    auto row_of = [&](const Task& k, int m) { return k.row0 + min(m, k.valid - 1); };   // past the end: the last one
    auto load_index = [&](int t) __attribute__((always_inline)) {
        const Task k = decode(min(t, total - 1));
        if (a.row_index != nullptr)
            __builtin_amdgcn_global_load_lds((fp8_glb_t*)(a.row_index + row_of(k, lane)), (fp8_lds_t*)index[wv], 4, 0, 0);
    };
    auto begin_weights = [&](int t) __attribute__((always_inline)) {
        const Task k = decode(min(t, total - 1));
        w_base = a.weight + ((size_t)k.e * a.N + k.n0) * a.K;
#pragma unroll
        for (int q = 0; q < LW; ++q)   // columns past the end: the last one
            w_off[q] = (uint32_t)min(8 * q + (lane >> 3), a.N - 1 - k.n0) * a.K + c16;
        return k;
    };
    auto begin_rows = [&](const Task& k) __attribute__((always_inline)) {
        auto source = [&](int m) {
            return (size_t)(a.row_index != nullptr ? max(0, min(lds_word(&index[wv][m]), a.x_rows - 1)) : row_of(k, m));
        };
#pragma unroll
        for (int j = 0; j < FM; ++j) x_src[j] = a.x + source(16 * j + rl) * a.K + 16 * g;
        s_src = a.x_scale + source(lane & (BM - 1)) * kb;
    };
    Frag fx[DEPTH][FM];
    // The next block into ring place d: always the same number of loads (past the end of
    // the row, of the blocks or of the tasks: zeros), which the waits count.  Weights
    // first, then, once the place's rows are multiplied, rows and scales; then advance.
    auto issue_weights = [&](auto D_) __attribute__((always_inline)) {
        uint8_t* dst = ring(D_) + wv * SLOT;
        const int k0 = ld_task < total ? ld_b * kQBlock : a.K;
        const bool in = k0 + c16 < a.K;
#pragma unroll
        for (int q = 0; q < LW; ++q)
            __builtin_amdgcn_global_load_lds((fp8_glb_t*)either(in, w_base + (size_t)k0 + w_off[q]), (fp8_lds_t*)(dst + q * 1024), 16,
                                             0, kLoadOnce);
    };
    auto issue_rows = [&](auto D_) __attribute__((always_inline)) {
        constexpr int d = decltype(D_)::value;
        const int k0 = ld_task < total ? ld_b * kQBlock : a.K;
        const bool in0 = k0 + 16 * g < a.K, in1 = k0 + 64 + 16 * g < a.K;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            fx[d][j].half[0] = *(glb_i32x4_t*)either(in0, x_src[j] + k0);
            fx[d][j].half[1] = *(glb_i32x4_t*)either(in1, x_src[j] + k0 + 64);
        }
        __builtin_amdgcn_global_load_lds((fp8_glb_t*)(s_src + min(ld_b, kb - 1)),
                                         (fp8_lds_t*)(ring(D_) + wv * SLOT + BN * kQBlock), 4, 0, 0);
    };
    auto advance = [&]() __attribute__((always_inline)) {
        ld_b += NW;
        if (++ld_step == steps) {
            ld_step = 0;
            ld_b = wv;
            ld_task += gridDim.x;
            begin_rows(begin_weights(ld_task));
            load_index(ld_task + gridDim.x);
        }
    };
    // The first DEPTH blocks: their weights do not wait for the rows' numbers.  (A task has
    // at least DEPTH blocks for each wave.)
    load_index(ld_task);
    const Task k0 = begin_weights(ld_task);
    static_for8<0, DEPTH>([&](auto D_) __attribute__((always_inline)) {
        issue_weights(D_);
        ld_b += NW;
    });
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<DEPTH * LW>();
    begin_rows(k0);
    load_index(ld_task + gridDim.x);
    ld_b = wv;
    static_for8<0, DEPTH>([&](auto D_) __attribute__((always_inline)) {
        issue_rows(D_);
        if constexpr (decltype(D_)::value + 1 < DEPTH) {
            ld_b += NW;
            ++ld_step;
        }
    });
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<0>();
    advance();

    // ---- products --------------------------------------------------------------------
    const int p0 = (g ^ (rl & 7)) << 4, p1 = ((4 + g) ^ (rl & 7)) << 4;   // places of chunks g and 4 + g
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Task k = decode(t);
        const float* ws = a.weight_scale + ((size_t)k.e * ((a.N + kQBlock - 1) / kQBlock) + k.n0 / kQBlock) * kb;
        f32x4_t acc[FN][FM];
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        int b = wv;
        for (int s = 0; s < steps; s += DEPTH) {
            static_for8<0, DEPTH>([&](auto D_) __attribute__((always_inline)) {
                constexpr int d = decltype(D_)::value;
                const float w = scalar_load(ws + min(b, kb - 1));
                wait_loads<(DEPTH - 1) * PER>();   // this block's loads; the DEPTH - 1 after it stay on their way
                const uint32_t src = lds_address(ring(D_) + wv * SLOT);
                Frag fw[FN];
                lds_blocks(fw, src + rl * kQBlock + p0, src + rl * kQBlock + p1);
                float f[FM];
#pragma unroll
                for (int j = 0; j < FM; ++j) f[j] = __int_as_float(lds_word(ring(D_) + wv * SLOT + BN * kQBlock + (16 * j + rl) * 4)) * w;
                __builtin_amdgcn_sched_barrier(0);
                issue_weights(D_);
                __builtin_amdgcn_sched_barrier(0);
                f32x4_t p[2][FN];
#pragma unroll
                for (int j = 0; j <= FM; ++j) {
                    if (j < FM) {
#pragma unroll
                        for (int i = 0; i < FN; ++i) p[j & 1][i] = block_product<EXACT>(fw[i], fx[d][j]);
                        if (j + 1 == FM) {
                            __builtin_amdgcn_sched_barrier(0);
                            issue_rows(D_);
                            advance();
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    if (j > 0) {
                        const float s1 = b < kb ? f[j - 1] : 0.0f;   // a block that does not exist: 0, whatever its scale
#pragma unroll
                        for (int i = 0; i < FN; ++i) {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                acc[i][j - 1][r] = __builtin_fmaf(p[(j - 1) & 1][i][r], s1, acc[i][j - 1][r]);
                            __asm__("" : "+v"(acc[i][j - 1]));   // here, not where the sum is next read
                        }
                    }
                }
                b += NW;
            });
        }
        // a lane holds columns 16 i + 4 g .. + 3 of row 16 j + rl
#pragma unroll
        for (int i0 = 0; i0 < FN; i0 += RI) {
            // (barriers that leave the loads on their way)
            wait_lds();
            barrier_only();   // the sums before are read
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int i = 0; i < RI; ++i)
                    *reinterpret_cast<f32x4_t*>(&part[wv][16 * j + rl][16 * i + 4 * g]) = acc[i0 + i][j];
            wait_lds();
            barrier_only();
            constexpr int Q = RC / 4;   // four columns a thread
            for (int c = tid; c < k.valid * Q; c += THREADS) {
                const int m = c / Q, n = c % Q * 4, col = k.n0 + 16 * i0 + n;
                f32x4_t v = *reinterpret_cast<const f32x4_t*>(&part[0][m][n]);
#pragma unroll
                for (int u = 1; u < NW; ++u) v += *reinterpret_cast<const f32x4_t*>(&part[u][m][n]);
                if (col < a.N) {
                    const size_t at = (size_t)(k.row0 + m) * a.N + col;
                    if (a.out_bf16)
                        *reinterpret_cast<uint2*>(static_cast<bf16_t*>(a.out) + at) =
                            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                    else
                        *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
                }
            }
        }
    }
    wait_loads<0>();   // the zeros loaded past the last task: nothing may reach the LDS after the end
}

}  // namespace

}  // namespace inkling
