// Gradients of grouped matrix products of bf16 operands on 256 x 256 tiles of
// four waves (gfx950); grouped.hip says which calls take it.
//
//   out[m][n] = sum_k B[m][k] A[n][k] over the rows m of one expert, as
//   kProdDx     A = weight read as [k][n], B = rows,        K = out_features
//   kProdWgrad  A = x and B = dout, both read as [k][...],  K = the expert's rows
//
// What bounds a product of this kind on a CU besides the matrix instructions is
// the LDS port: 128 bytes a clock carry both the fragments that the waves read
// and the stages that the loads write.  A wave tile of 64 x 128 reads 96 KB for
// each 32-K step of a 256 x 256 tile, 768 clocks of the 1024 that its matrix
// instructions take, and the stages take 256 more: nothing left.  Four waves of
// 128 x 128, one for each SIMD, read 64 KB (512 clocks), so the port is free a
// quarter of the time.  Their 256 accumulators a lane fill the accumulation
// registers; the fragments of two k-steps take 64 vector registers.
//
// With one wave a SIMD nothing else runs while it waits, so the loop is built
// for that: the fragments of the next k-step and the loads of a later stage are
// issued one by one between matrix instructions (a burst of 8 loads cost 5%),
// a stage's loads are spread over two k-steps, the next tile is looked up
// during the current one, and the first waits of a tile count the stores of the
// tile before instead of waiting for them.
//
// Stages: 128 KB of LDS as 4 buffers of 32 K where both operands are [k][...]
// (512 bytes a K row), as 2 of 64 K where B is K-major: 32 K would be 64-byte
// pieces of rows, and L2 answers a request a clock and channel whatever its
// size, so half-line requests alone took as long as the matrix instructions.
//
// Measured (4096 rows an expert, 4096 x 8192 weights): weight gradients 1.28
// PFLOP/s, input gradients 1.13; a tile's change-over (drain, epilogue, first
// loads) takes 9 to 13 us beside 0.74 us for 32 K, which is what bounds experts
// of few rows.
#pragma once

#include "gemm_kernel.h"
#include "grouped_small.h"

namespace inkling {

namespace {

struct ProductArgs {
    const bf16_t* A;            // weights [E][K][N]; kProdWgrad: x rows [rows][N]
    const bf16_t* B;            // rows [rows][K]; kProdWgrad: dout rows [rows][M]
    const int32_t* offs;        // [E + 1]
    const RoutedTile* tiles;    // kProdDx: row tiles of 256
    const int32_t* num_tiles;
    int E, K, N, M;             // N: columns of out; M, E: kProdWgrad (rows of out, problems)
    int ntn, ntm;               // column tiles; kProdWgrad: row tiles
    void* out;                  // [rows][N]; kProdWgrad: [E][M][N]
    int out_bf16;
    int32_t* counters;          // [8], zero at launch: tiles taken of each XCD's range
};

struct ProductTile {
    const bf16_t* A;
    const bf16_t* B;
    char* out;
    int K;            // values of K
    int n0;           // first column of out
    int m0;           // first row of out
    int rows;         // rows of out in this tile
};

// an int at an address that is the same for the whole wave, written by an earlier
// kernel only: a scalar load, which the vector-memory waits do not count
__device__ __forceinline__ int uniform_load(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)p;
}

template <int MODE>
__device__ __forceinline__ ProductTile product_tile(const ProductArgs& a, int L) {
    ProductTile t;
    const int ob = a.out_bf16 ? 2 : 4;
    if constexpr (MODE == kProdWgrad) {
        // problem by problem; inside, groups of 4 row tiles walk the column tiles
        const int per = a.ntm * a.ntn, e = L / per;
        int mt, nt;
        grouped<4>(L - e * per, a.ntm, a.ntn, mt, nt);
        const int r0 = uniform_load(a.offs + e);
        t.K = uniform_load(a.offs + e + 1) - r0;
        t.A = a.A + (size_t)r0 * a.N;
        t.B = a.B + (size_t)r0 * a.M;
        t.n0 = nt * 256;
        t.m0 = mt * 256;
        t.rows = min(256, a.M - t.m0);
        t.out = static_cast<char*>(a.out) + (size_t)e * a.M * a.N * ob;
    } else {
        // the row tiles of an expert for weight tile 0, then for 1, ...: the
        // workgroups side by side on an XCD share weight tiles
        const int l0 = L / a.ntn;
        const int32_t* tile = reinterpret_cast<const int32_t*>(a.tiles + l0);
        const int expert = uniform_load(tile);
        const int tb = l0 - (uniform_load(tile + 1) >> 8);   // first row tile of the expert
        const int base = uniform_load(a.offs + expert), cnt = uniform_load(a.offs + expert + 1) - base;
        const int c = (cnt + 255) >> 8;
        const int l = L - tb * a.ntn, nt = l / c, row0 = (l - nt * c) << 8;
        t.K = a.K;
        t.A = a.A + (size_t)expert * a.N * a.K;
        t.B = a.B;
        t.n0 = nt * 256;
        t.m0 = base + row0;
        t.rows = min(256, cnt - row0);
        t.out = static_cast<char*>(a.out);
    }
    return t;
}

typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <int MODE>
__global__ __launch_bounds__(256, 1) void product_kernel(const ProductArgs a) {
    constexpr bool BKN = MODE == kProdWgrad;    // (A is [k][n] in both)
    constexpr int BK = BKN ? 32 : 64, S = 128 / BK;   // K of a stage, stages
    constexpr int KS = BK / 16;                 // k-steps of a stage
    constexpr int STAGE = 256 * BK * 2;         // bytes of an operand's stage
    constexpr int PW = STAGE / 1024 / 4;        // 1 KB wave loads of an operand and stage for each wave
    constexpr int FN = 4, FM = 4;               // 32 x 32 blocks of a wave
    constexpr int RB = 512;                     // bytes of a K row of a [K][...] stage
    __shared__ __attribute__((aligned(16))) uint8_t sa0[STAGE], sa1[STAGE], sa2[S > 2 ? STAGE : 16], sa3[S > 2 ? STAGE : 16];
    __shared__ __attribute__((aligned(16))) uint8_t sb0[STAGE], sb1[STAGE], sb2[S > 2 ? STAGE : 16], sb3[S > 2 ? STAGE : 16];
    constexpr int kEpRow = 144;                 // 128 bytes of a row + 16
    __shared__ __attribute__((aligned(16))) uint8_t ep_lds[4 * 32 * kEpRow];
    __shared__ int q_next;
    auto stage_a = [&](auto S_) -> uint8_t* {
        constexpr int i = decltype(S_)::value % S;
        if constexpr (i == 0) return sa0;
        else if constexpr (i == 1) return sa1;
        else if constexpr (i == 2) return sa2;
        else return sa3;
    };
    auto stage_b = [&](auto S_) -> uint8_t* {
        constexpr int i = decltype(S_)::value % S;
        if constexpr (i == 0) return sb0;
        else if constexpr (i == 1) return sb1;
        else if constexpr (i == 2) return sb2;
        else return sb3;
    };

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn0 = (wv & 1) * 128, wm = wv >> 1;   // columns wn0 ..; row blocks wm, wm + 2, ...

    // ---- tiles: a contiguous range for each XCD, taken from its counter --------
    const int total = MODE == kProdWgrad ? a.E * a.ntm * a.ntn : uniform_load(a.num_tiles) * a.ntn;
    const int xcd = blockIdx.x & 7, nloc = gridDim.x >> 3;
    const int L_beg = (int)((long long)total * xcd / 8), L_end = (int)((long long)total * (xcd + 1) / 8);
    int L = L_beg + (blockIdx.x >> 3);
    if (L >= L_end) return;

    // ---- loads -------------------------------------------------------------------
    // K-major: 64-byte rows, 16 rows a wave load; the 16-byte chunk c of row r
    // sits at c ^ ((r >> 2) & 3): any 16 rows of a read that differ in r / 4 mod 4
    // or r mod 4 lie on different banks.  [K][...]: two K rows a wave load; chunk c of K
    // row r sits at c ^ swk(r), so that the eight 32-byte pieces that half a wave
    // reads at once (4 K rows of 2 x 16 columns) lie on different banks.
    auto swk = [](int r) { return (r & 3) << 2; };
    constexpr int CH = BK / 8, RW = 64 / CH;   // 16-byte chunks of a K-major row, rows of a wave load
    const int lr = lane / CH;
    const int lc = BK == 32 ? (lane & 3) ^ (lr >> 2) : (lane & 7) ^ ((lr >> 1) | ((wv & 1) << 2));
    const bf16_t* a_src[PW];
    const bf16_t* b_src[PW];
    int k_ld = 0, K_ld = 0;
    auto setup = [&](const ProductTile& t) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            const int kr = 2 * (wv + 4 * q) + (lane >> 5), c = (lane & 31) ^ swk(kr);
            a_src[q] = t.A + (size_t)kr * a.N + min(t.n0 + 8 * c, a.N - 8);   // columns past N re-read its last ones
            if constexpr (BKN) {
                b_src[q] = t.B + (size_t)kr * a.M + min(t.m0 + 8 * c, a.M - 8);
            } else {
                const int r = t.m0 + min(RW * (wv + 4 * q) + lr, t.rows - 1);   // rows past the end re-read the last
                b_src[q] = t.B + (size_t)r * a.K + 8 * lc;
            }
        }
        k_ld = 0;
        K_ld = t.K;
    };
    const bf16_t* zeros = reinterpret_cast<const bf16_t*>(&zero_chunk);
    // TAIL: the stage may hold K values past the end, which are zeros on both sides
    auto issue_a = [&](auto S_, auto TAIL_) __attribute__((always_inline)) {
        uint8_t* __restrict__ da = stage_a(S_);
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            const int qi = wv + 4 * q;
            const bf16_t* src = a_src[q];
            if (decltype(TAIL_)::value && k_ld + 2 * qi + (lane >> 5) >= K_ld) src = zeros;
            __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(da + qi * 1024), 16, 0, 0);
            a_src[q] += (size_t)BK * a.N;
        }
    };
    auto issue_b = [&](auto S_, auto TAIL_) __attribute__((always_inline)) {
        uint8_t* __restrict__ db = stage_b(S_);
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            const int qi = wv + 4 * q;
            const bf16_t* src = b_src[q];
            if (decltype(TAIL_)::value && k_ld + (BKN ? 2 * qi + (lane >> 5) : 8 * lc) >= K_ld) src = zeros;
            __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(db + qi * 1024), 16, 0, 0);
            b_src[q] += BKN ? (size_t)BK * a.M : BK;
        }
        k_ld += BK;
    };
    auto issue_first = [&](int nk) __attribute__((always_inline)) {
        static_for<0, S>([&](auto S_) {
            if (decltype(S_)::value < nk) {
                issue_a(S_, std::true_type{});
                issue_b(S_, std::true_type{});
            }
        });
    };

    // ---- fragments -----------------------------------------------------------------
    // 32 x 32 x 16: lane l holds k = 8 (l / 32) .. + 7 of row (column) l % 32
    int a_rd[KS], b_rd[KS];   // by the k-step of a stage
    {
        const int rl = lane & 31, h = lane >> 5;
        const int g = lane >> 4, j4 = (lane >> 2) & 3, q4 = lane & 3;
        const int kn = (8 * h + j4) * RB + ((2 * (g & 1) + (q4 >> 1)) ^ (j4 << 2)) * 16 + (q4 & 1) * 8;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int sw = BK == 32 ? (rl >> 2) & 3 : (rl >> 1) & 7;
            const int kmaj = rl * (2 * BK) + (((2 * s + h) ^ sw) << 4);
            a_rd[s] = (kn ^ (2 * wn0)) + 16 * s * RB;
            b_rd[s] = BKN ? (kn ^ (64 * wm)) + 16 * s * RB : 32 * wm * (2 * BK) + kmaj;
        }
    }
    auto read_a = [&](const uint8_t* __restrict__ st, int ks, int i) __attribute__((always_inline)) -> uint4 {
        return read_tr16_frag(st + (a_rd[ks] ^ (64 * i)), RB);
    };
    auto read_b = [&](const uint8_t* __restrict__ st, int ks, int j) __attribute__((always_inline)) -> uint4 {
        if constexpr (BKN) return read_tr16_frag(st + (b_rd[ks] ^ (128 * j)), RB);
        else return *reinterpret_cast<const uint4*>(st + b_rd[ks] + j * 128 * BK);
    };

    // NJ: row blocks computed.  The fragments of a k-step are read while the one
    // before multiplies; before a stage's second k-step: wait for stage kt + 1,
    // meet, read its first fragments, load stage kt + 4 into the buffers just
    // read (their last fragments are in registers).
    auto kloop = [&](auto& acc, auto NJ_, int cur_K, int past) __attribute__((always_inline)) {
        constexpr int NJ = decltype(NJ_)::value;
        const int nk = (cur_K + BK - 1) / BK;
        constexpr int READS = 4 * 2 + NJ * (BKN ? 2 : 1);   // LDS reads of a k-step
        uint4 fa[2][FN], fb[2][NJ];
        // `past`: epilogue stores of the tile before, younger than the first S
        // stages (0: unknown, waited for)
        auto wait_first = [&](auto AHEAD_) __attribute__((always_inline)) {
            constexpr int loads = decltype(AHEAD_)::value * 2 * PW;
            if (past == 0) wait_vmcnt<loads>();
            else if (past == 32) wait_vmcnt<(loads + 32 < 63 ? loads + 32 : 63)>();
            else wait_vmcnt<63>();
        };
        auto wait_stage = [&](int ahead) __attribute__((always_inline)) {   // stages loaded after the one waited for
            if (S > 3 && ahead >= 3) wait_vmcnt<(S - 1) * 2 * PW>();
            else if (S > 2 && ahead == 2) wait_vmcnt<S / 2 * 2 * PW>();
            else if (ahead == 1) wait_vmcnt<2 * PW>();
            else wait_vmcnt<0>();
        };
        auto read = [&](const uint8_t* __restrict__ sta, const uint8_t* __restrict__ stb,
                        auto KS_) __attribute__((always_inline)) {
            constexpr int ks = decltype(KS_)::value;
#pragma unroll
            for (int i = 0; i < FN; ++i) fa[ks & 1][i] = read_a(sta, ks, i);
#pragma unroll
            for (int j = 0; j < NJ; ++j) fb[ks & 1][j] = read_b(stb, ks, j);
        };
        auto multiply = [&](auto KS_) __attribute__((always_inline)) {
            constexpr int ks = decltype(KS_)::value;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < FN; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa[ks & 1][i]),
                                                                        __builtin_bit_cast(bf16x8_t, fb[ks & 1][j]),
                                                                        acc[i][j], 0, 0, 0);
        };
        // a k-step's LDS reads and `loads` stage loads between its matrix instructions
        auto spread = [&](auto LOADS_) __attribute__((always_inline)) {
            constexpr int LOADS = decltype(LOADS_)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, (READS + 7) / 8, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (i < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                if (i < LOADS) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
        };
        using K0 = std::integral_constant<int, 0>;
        using None = std::integral_constant<int, 0>;
        using Loads = std::integral_constant<int, PW>;
        // Stage kt.  STEADY: stages kt + 1 and kt + S exist and are whole.  A's part
        // of stage kt + S is loaded in the last k-step, once every wave has read
        // the last of stage kt, B's in the next stage's first (FIRST: stage 0).
        // The waits of a steady first round (FIRST_ROUND) count the stores of the
        // tile before, which are younger than the S stages loaded ahead of it.
        auto step = [&](auto S_, auto STEADY_, auto ROUND_, int kt) __attribute__((always_inline)) {
            constexpr bool STEADY = decltype(STEADY_)::value, FIRST_ROUND = decltype(ROUND_)::value;
            constexpr int sidx = decltype(S_)::value;
            using Next = std::integral_constant<int, (sidx + 1) % S>;
            using Prev = std::integral_constant<int, (sidx + S - 1) % S>;
            using Tail = std::integral_constant<bool, !STEADY>;
            static_for<0, KS - 1>([&](auto KS_) __attribute__((always_inline)) {
                constexpr int ks = decltype(KS_)::value;
                constexpr bool load = ks == 0 && !(FIRST_ROUND && sidx == 0);
                wait_lgkmcnt0();
                __builtin_amdgcn_sched_barrier(0);
                read(stage_a(S_), stage_b(S_), std::integral_constant<int, ks + 1>{});
                if constexpr (load)
                    if (STEADY || (kt > 0 && kt - 1 + S < nk)) issue_b(Prev{}, Tail{});
                multiply(KS_);
                if constexpr (STEADY) spread(std::conditional_t<load, Loads, None>{});
                __builtin_amdgcn_sched_barrier(0);
            });
            wait_lgkmcnt0();
            if (STEADY || kt + 1 < nk) {
                // younger than stage kt + 1: the loads of stages kt + 2 .. kt + S - 1
                if constexpr (STEADY && FIRST_ROUND && sidx + 1 < S) wait_first(std::integral_constant<int, S - 2>{});
                else if constexpr (STEADY) wait_vmcnt<(S - 2) * 2 * PW>();
                else wait_stage(min(nk - 1, kt + S - 1) - (kt + 1));
                barrier_keep_loads();
                __builtin_amdgcn_sched_barrier(0);
                read(stage_a(Next{}), stage_b(Next{}), K0{});
                if (STEADY || kt + S < nk) issue_a(S_, Tail{});
            }
            multiply(std::integral_constant<int, KS - 1>{});
            if constexpr (STEADY) spread(Loads{});
            __builtin_amdgcn_sched_barrier(0);
        };
        using std::true_type;
        using std::false_type;
        int kt0 = 0;
        if (2 * S * BK <= cur_K) {
            wait_first(std::integral_constant<int, S - 1>{});
            barrier_keep_loads();
            read(sa0, sb0, K0{});
            static_for<0, S>([&](auto S_) __attribute__((always_inline)) {
                step(S_, true_type{}, true_type{}, decltype(S_)::value);
            });
            for (kt0 = S; (kt0 + 2 * S) * BK <= cur_K; kt0 += S)
                static_for<0, S>([&](auto S_) __attribute__((always_inline)) {
                    step(S_, true_type{}, false_type{}, kt0 + decltype(S_)::value);
                });
        } else {
            wait_stage(min(nk, S) - 1);
            barrier_keep_loads();
            read(sa0, sb0, K0{});
        }
        for (; kt0 < nk; kt0 += S)
            static_for<0, S>([&](auto S_) __attribute__((always_inline)) {
                if (kt0 + decltype(S_)::value < nk) step(S_, false_type{}, false_type{}, kt0 + decltype(S_)::value);
            });
    };

    // The tile after the current one is taken and looked up while the current one
    // multiplies, so that its loads start as soon as the stages are free.
    auto take = [&]() { return __hip_atomic_fetch_add(a.counters + xcd, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    ProductTile cur = product_tile<MODE>(a, L);
    setup(cur);
    issue_first((cur.K + BK - 1) / BK);
    if (tid == 0) q_next = take();
    __syncthreads();
    L = __builtin_amdgcn_readfirstlane(L_beg + nloc + q_next);
    int past = 0;
    bool more = false;
    ProductTile nxt = cur;
    // A tile's K loop, the next one's first loads, its epilogue; NJ row blocks a
    // wave (each count has its own accumulators, which so stay where the matrix
    // instructions want them).
    auto run_tile = [&](auto NJ_, int nvb) __attribute__((always_inline)) {
        constexpr int NJ = decltype(NJ_)::value;
        f32x16_t acc[FN][NJ];
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16_t{};
        int taken = 0;
        if (more && tid == 0) taken = take();
        if (cur.K > 0) kloop(acc, NJ_, cur.K, past);
        // keeps a block's sums in the accumulation registers up to here: left to
        // itself the compiler moves all of them out at once, and spills
        auto hold = [&](f32x16_t& v) __attribute__((always_inline)) { __asm__ volatile("" : "+a"(v)); };
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) hold(acc[i][j]);
        // every wave is done with the stages: start the next tile's loads
        if (more) {
            if (tid == 0) q_next = taken;
            __syncthreads();
            L = __builtin_amdgcn_readfirstlane(L_beg + nloc + q_next);
            setup(nxt);
            issue_first((nxt.K + BK - 1) / BK);
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- epilogue: acc[i][j][4 q + r] is column wn0 + 32 i + 8 q + 4 (lane / 32)
        // + r of row 32 (2 j + wm) + lane % 32.  32 rows at a time pass through
        // the wave's LDS block, 128 bytes each, so that stores write whole row
        // segments (one wave's LDS operations complete in order).
        int ln = lane;
        __asm__ volatile("" : "+v"(ln));   // recomputed a tile: nothing lane-derived lives across the K loop
        const int h = ln >> 5, rw = ln & 31, r8 = ln >> 3, c8 = ln & 7;
        uint8_t* __restrict__ ep = ep_lds + wv * 32 * kEpRow;
        const int width = a.N - cur.n0 - wn0;   // columns from the wave's first on
        const size_t first = (size_t)cur.m0 * a.N + cur.n0 + wn0;   // of the tile's first row
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int mb = 32 * (2 * j + wm);
            if (j >= nvb) continue;
            if (a.out_bf16) {
                char* o = cur.out + 2 * first;
#pragma unroll
                for (int i0 = 0; i0 < FN; i0 += 2) {
#pragma unroll
                    for (int i = i0; i < i0 + 2; ++i) {
                        hold(acc[i][j]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                               acc[i][j][4 * q + 3]};
                            *reinterpret_cast<uint2*>(ep + rw * kEpRow + (32 * (i - i0) + 8 * q + 4 * h) * 2) =
                                pack_bf16x4(v);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = 8 * q + r8, c = 32 * i0 + 8 * c8;
                        const uint4 d = *reinterpret_cast<const uint4*>(ep + r * kEpRow + c8 * 16);
                        if (mb + r < cur.rows && c < width)
                            *reinterpret_cast<uint4*>(o + (uint32_t)(2 * ((mb + r) * a.N + c))) = d;
                    }
                }
            } else {
                char* o = cur.out + 4 * first;
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    hold(acc[i][j]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                           acc[i][j][4 * q + 3]};
                        *reinterpret_cast<f32x4_t*>(ep + rw * kEpRow + (8 * q + 4 * h) * 4) = v;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = 8 * q + r8, c = 32 * i + 4 * c8;
                        const f32x4_t d = *reinterpret_cast<const f32x4_t*>(ep + r * kEpRow + c8 * 16);
                        if (mb + r < cur.rows && c < width)
                            *reinterpret_cast<f32x4_t*>(o + (uint32_t)(4 * ((mb + r) * a.N + c))) = d;
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    while (true) {
        more = L < L_end;
        if (more) nxt = product_tile<MODE>(a, L);
        // row blocks of this wave that hold rows (none: takes part in the loads and barriers)
        const int nvb = min(FM, max(0, (((cur.rows + 31) >> 5) - wm + 1) >> 1));
        if (nvb == 4) run_tile(std::integral_constant<int, 4>{}, nvb);
        else if (nvb == 3) run_tile(std::integral_constant<int, 3>{}, nvb);
        else if (nvb == 2) run_tile(std::integral_constant<int, 2>{}, nvb);
        else run_tile(std::integral_constant<int, 1>{}, nvb);
        if (!more) break;
        // a whole tile's stores all go out: 4 x 2 x 4 of 16 bytes a lane, or 4 x 4 x 4
        past = cur.rows == 256 && cur.n0 + 256 <= a.N ? (a.out_bf16 ? 32 : 64) : 0;
        cur = nxt;
    }
}

}  // namespace

}  // namespace inkling
