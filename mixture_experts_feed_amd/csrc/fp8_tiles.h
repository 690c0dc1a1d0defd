// Products of e4m3 rows and weights grouped by expert on 256 x 256 tiles:
//   forward         out[r][n] = sum_b xs[r][b] ws[n/128][b] sum_{k in block b} x[r][k] W[n][k]
//   input gradient  dx[r][k]  = sum_b ds[r][b] ws[b][k/128] sum_{n in block b} d[r][n] W[n][k]
// Weights are the matrix instruction's first operand (its rows = output columns), token
// rows the second, so that a lane holds four consecutive output columns of one row.
// One instruction takes a whole block of 128, so a block's sum starts at zero, and its
// four values a lane are added to the running sums with one fp32 multiply-add each by
// xs ws, whose row factor is a lane's own and whose weight factor is uniform.
//
// Persistent workgroups of eight waves (four along the columns, two along the rows, 64 x
// 128 of the tile each), one a CU.  A K stage is one block of 128: 32 KB of weights, 32
// KB of rows and the rows' 1 KB of scales, loaded straight into LDS, two stages in turn.
// The first stages of the next tile are loaded before the results of the current one
// are stored.
// Every workgroup finds the tiles from the caller's offsets by itself (a scan over at
// most 512 experts in LDS), so there is no plan, no workspace and nothing to clear.  A
// XCD takes a contiguous range of tiles, an expert's row tiles innermost, so that the
// workgroups that run side by side share weights and rows through its L2.
// 8192 x 8192 x 8192: 515 to 545 us (2.0 to 2.1 PFLOP/s); 128 experts of 316 to 754 rows, 6144 x
// 4096: 1800 to 1900 us, matrix units busy 46% of the cycles.  Beside the 2048 cycles that a
// stage's products take on a SIMD's matrix unit stand 1024 for adding them by their scales
// and 1536 of LDS reads; and the card lowers its clock to 1.7 to 1.9 GHz.  Results in fp32
// (EXACT) take twice the time: 1052 to 1065 us (1.04 PFLOP/s) and 3700 to 3800, where the
// conversions to bf16 stand beside the products.
#pragma once

#include "fp8_common.h"

namespace inkling {

namespace {

constexpr int kTileThreads = 512;

struct Fp8Tile {
    int e, row0, valid, n0;   // expert; first row and rows of the tile; first output column
};

// KN: the input gradient (weights read as [reduction][column])
// FM: 16-row blocks of a wave's tile; the workgroup's tile has BM = 32 FM rows.
// FAR: x is larger than 32 bits reach.
template <int FM, bool KN, bool EXACT, bool FAR>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_tile_kernel(const Fp8Args a) {
    constexpr int BN = 256, BM = 32 * FM, WN = 4, NW = 8, FN = 4;
    constexpr int BH = FM / 4;                     // wave loads of half a stage's rows
    static_assert(FM == 4 || FM == 8, "128 or 256 rows");
    constexpr int STAGE = BN * kQBlock, STAGE_B = BM * kQBlock;
    // each stage its own object: the compiler then needs no wait for the loads into one
    // before reads of the other
    __shared__ __attribute__((aligned(16))) uint8_t sa0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t sa1[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t sb0[STAGE_B];
    __shared__ __attribute__((aligned(16))) uint8_t sb1[STAGE_B];
    // scales of a stage: of 256 rows, then those of each column group's weights (64 times)
    __shared__ __attribute__((aligned(16))) float ss0[kTileThreads];
    __shared__ __attribute__((aligned(16))) float ss1[kTileThreads];
    constexpr int kEpRow = 144;   // 128 bytes of a result row and 16 of padding
    __shared__ __attribute__((aligned(16))) uint8_t ep_lds[NW * 16 * kEpRow];
    __shared__ int32_t offs[kMaxFp8Groups + 1], first[kMaxFp8Groups + 1];

    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn0 = (wv % WN) * 64, wm = wv / WN;
    const int rl = lane & 15, g = lane >> 4;
    const int len = KN ? a.N : a.K, cols = KN ? a.K : a.N;   // reduction length, output columns
    const int nb = (len + kQBlock - 1) / kQBlock;            // blocks of the reduction
    const int cb = (cols + kQBlock - 1) / kQBlock;
    const int ntn = (cols + BN - 1) / BN;

    // ---- the experts' rows and row tiles -----------------------------------------
    plan_experts<kTileThreads>(a, a.tile_rows, offs, first);
    const long long total = (long long)first[a.E] * ntn;
    const int xcd = blockIdx.x & 7, nloc = gridDim.x >> 3;
    const int L_end = (int)(total * (xcd + 1) / 8);
    int L = (int)(total * xcd / 8) + (int)(blockIdx.x >> 3);
    if (L >= L_end) return;

    auto decode = [&](int l) {
        Fp8Tile t;
        const int rt = l / ntn;
        t.e = expert_of(first, a.E, rt);
        const int f = first[t.e], c = first[t.e + 1] - f;
        const int in = l - f * ntn, nt = in / c, mt = in - nt * c;
        // the expert's row tiles share its rows evenly, by 64
        const int rows = offs[t.e + 1] - offs[t.e], per = ((rows + 63) / 64 + c - 1) / c * 64;
        t.row0 = __builtin_amdgcn_readfirstlane(offs[t.e] + mt * per);
        t.valid = __builtin_amdgcn_readfirstlane(min(per, rows - mt * per));
        t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
        return t;
    };

    // ---- loads -------------------------------------------------------------------
    // 128-byte rows (token rows; weights of the forward): the 16-byte chunk c of row r
    // sits at chunk place c ^ (r & 7); 256-byte rows (weights of the input gradient, a
    // row of the reduction each): at c ^ swk(r).  Both keep the reads below spread over
    // the banks.  A wave load is 1 KB: eight 128-byte rows (lane / 8 of them; chunk place
    // lane % 8) or four 256-byte rows.
    auto swk = [](int r) { return (r & 7) | ((r >> 1) & 8); };
    const int c16 = 16 * ((lane & 7) ^ (lane >> 3));   // the lane's chunk of its 128-byte rows
    // A load adds a lane's 32-bit offset to a scalar base.  Weights: from the expert's,
    // the tile's first row (input gradient: the reduction's first); rows: from a.x (FAR:
    // the row's number, and 64-bit arithmetic for every load).
    const uint8_t* a_base = nullptr;
    const float* ws_base = nullptr;     // weight scale of block 0 of this wave's columns
    uint32_t a_off[4], b_off[2 * BH], s_off = 0;
    auto setup = [&](const Fp8Tile& t) __attribute__((always_inline)) {
        const int kb = (a.K + kQBlock - 1) / kQBlock, c = min((t.n0 + wn0) / kQBlock, cb - 1);
        a_base = a.weight + (size_t)t.e * a.N * a.K + (KN ? 0 : (size_t)t.n0 * a.K);
        ws_base = a.weight_scale + (size_t)t.e * cb * nb + (KN ? c : c * kb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (KN) {
                const int r = 4 * (wv + NW * q) + (lane >> 4);
                const int ch = (lane & 15) ^ swk(r);
                a_off[q] = (uint32_t)r * a.K + min(t.n0 + 16 * ch, a.K - 16);   // columns past the end: the last chunk
            } else {
                const int r = 8 * (wv + NW * q) + (lane >> 3);
                a_off[q] = (uint32_t)min(r, a.N - 1 - t.n0) * a.K + c16;        // rows past the end: the last row
            }
        }
        auto source = [&](int m) {   // x row of the tile's row m (past the end: the last one)
            int row = t.row0 + min(m, t.valid - 1);
            if (!KN && a.row_index != nullptr) row = max(0, min(a.row_index[row], a.x_rows - 1));
            return (uint32_t)row;
        };
#pragma unroll
        for (int q = 0; q < 2 * BH; ++q) {
            const uint32_t row = source(8 * (wv + NW * q) + (lane >> 3));
            b_off[q] = FAR ? row : row * (uint32_t)len + c16;
        }
        const uint32_t row = source(64 * (wv & 3) + lane);
        s_off = FAR ? row : row * (uint32_t)nb;
    };
    // (Offsets pass through an empty asm so that no address is kept over the K loop, which
    // needs the registers: a spilled one's reload would wait for all loads.)
    auto fresh = [](uint32_t v) __attribute__((always_inline)) {
        __asm__ volatile("" : "+v"(v));
        return v;
    };
    // The loads of a block, in two parts (see the schedule below): weights and the first
    // half of the rows; the scales and the second half.  Always the same number, which
    // the waits count.  Past the end of the reduction the rows' chunks read zeros; the
    // weights read their row's last chunk (input gradient: earlier rows), whose numbers do
    // not matter, since one that is NaN also stands in the sums of the same column before.
    constexpr int FIRST = 4 + BH, SECOND = 1 + BH;
    auto past = [&](int b) __attribute__((always_inline)) {   // bytes of the lane's chunk past the end
        return (uint32_t)max(0, c16 + 16 + b * kQBlock - len);
    };
    auto load_a = [&](int q, uint8_t* da, int b) __attribute__((always_inline)) {
        uint8_t* dst = da + (wv + NW * q) * 1024;
        if constexpr (KN) {
            // (four rows of the reduction, all before its end or all past it)
            const int r = 4 * (wv + NW * q);
            const uint8_t* base = a_base + ((size_t)b * kQBlock - (b * kQBlock + r < len ? 0 : r)) * a.K;
            copy16_to_lds<0>(base + fresh(a_off[q]), dst);
        } else {
            copy16_to_lds<0>(a_base + b * kQBlock + (fresh(a_off[q]) - past(b)), dst);
        }
    };
    auto load_b = [&](int q, uint8_t* db, int b) __attribute__((always_inline)) {
        uint8_t* dst = db + (wv + NW * q) * 1024;
        const uint32_t off = fresh(b_off[q]);
        const int k0 = b * kQBlock;
        if (k0 + kQBlock <= len) {
            copy16_to_lds<0>(a.x + k0 + (FAR ? (uint64_t)off * (uint32_t)len + c16 : (uint64_t)off), dst);
        } else {
            uint64_t p = reinterpret_cast<uint64_t>(a.x + k0 + (FAR ? (uint64_t)off * (uint32_t)len + c16 : (uint64_t)off));
            p = k0 + c16 < len ? p : reinterpret_cast<uint64_t>(&fp8_zero_chunk);
            __asm__ volatile("" : "+v"(p));   // not computed where the tail is not
            copy16_to_lds<0>((const void*)p, dst);
        }
    };
    auto load_s = [&](float* ds, int b) __attribute__((always_inline)) {
        const uint32_t off = fresh(s_off);
        if (wv < 4) {
            const float* p = FAR ? a.x_scale + b + (uint64_t)off * (uint32_t)nb : a.x_scale + b + off;
            __builtin_amdgcn_global_load_lds((fp8_glb_t*)p, (fp8_lds_t*)(ds + 64 * wv), 4, 0, 0);
        } else {
            const float* p = ws_base + (size_t)b * (KN ? cb : 1);
            __builtin_amdgcn_global_load_lds((fp8_glb_t*)p, (fp8_lds_t*)(ds + 64 * wv), 4, 0, 0);
        }
    };
    // load number i of each part
    auto first_part = [&](int i, uint8_t* da, uint8_t* db, int b) __attribute__((always_inline)) {
        if (i < 4) load_a(i, da, b);
        else load_b(i - 4, db, b);
    };
    auto second_part = [&](int i, uint8_t* db, float* ds, int b) __attribute__((always_inline)) {
        if (i == 0) load_s(ds, b);
        else load_b(BH + i - 1, db, b);
    };
    // what a tile's K loop finds on its way
    auto issue_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FIRST; ++i) first_part(i, sa0, sb0, 0);
#pragma unroll
        for (int i = 0; i < SECOND; ++i) second_part(i, sb0, ss0, 0);
        if (nb > 1)
#pragma unroll
            for (int i = 0; i < FIRST; ++i) first_part(i, sa1, sb1, 1);
    };

    // ---- fragments -----------------------------------------------------------------
    const int at0 = (g ^ (rl & 7)) << 4, at1 = ((4 + g) ^ (rl & 7)) << 4;   // places of chunks g and 4 + g
    const int a_row = (wn0 + rl) * kQBlock, b_row = (16 * wm + rl) * kQBlock;
    // input gradient: lane 2 j + h of 16 addresses half h of the 16 columns' chunk in
    // reduction row j of eight; the transposing read hands lane c the eight rows of column c
    const int tr_sz = (rl >> 1) | ((g & 1) << 3);
    const int tr_at = (16 * g + (rl >> 1)) * 256 + (((wn0 >> 4) ^ tr_sz) << 4) + (rl & 1) * 8;
    auto read_a = [&](const uint8_t* __restrict__ st, int i) __attribute__((always_inline)) {
        Frag f;
        if constexpr (KN) {
            const uint8_t* p = st + ((int)fresh((uint32_t)tr_at) ^ (i << 4));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                f.quarter[q] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (fp8_lds_i32x2_t*)(p + ((q & 1) * 8 + (q >> 1) * 64) * 256));
        } else {
            f.half[0] = *reinterpret_cast<const i32x4_t*>(st + a_row + i * 16 * kQBlock + at0);
            f.half[1] = *reinterpret_cast<const i32x4_t*>(st + a_row + i * 16 * kQBlock + at1);
        }
        return f;
    };
    auto read_b = [&](const uint8_t* __restrict__ st, int j) __attribute__((always_inline)) {
        Frag f;
        f.half[0] = *reinterpret_cast<const i32x4_t*>(st + b_row + j * 32 * kQBlock + at0);
        f.half[1] = *reinterpret_cast<const i32x4_t*>(st + b_row + j * 32 * kQBlock + at1);
        return f;
    };

    f32x4_t acc[FN][FM];

    // NJ: 16-row blocks of the wave that are multiplied (the others hold no rows).
    //
    // A stage takes a step a row block: the LDS reads of the next step, the block's four
    // products, and their sums (by the time the last product is issued the first is done).  All waves meet twice a stage:
    //   P0(b), before the products of the last two steps of stage b - 1 (all its reads
    //     done): the weights, the first half of the rows and the scales of b are there; the
    //     second half and the scales of b + 1 may be loaded where b - 1 had them;
    //   P1(b), once the weights (read into registers at once) and the first half of b are
    //     read: its second half is there; the weights and the first half of b + 2 may be
    //     loaded in their place.
    // So everything is on its way for a stage and a half, in two stages' buffers.  The
    // loads are spread over the steps after each meeting: all at once they would hold up
    // every wave.
    auto kloop = [&](auto NJ_, const Fp8Tile& t) __attribute__((always_inline)) {
        constexpr int NJ = decltype(NJ_)::value;
        // steps before the last two; the one of them that P1 is in (none: it is with P0)
        constexpr int HALF = FM / 2, EARLY = NJ - 2, MEET = NJ > HALF ? HALF - 1 : EARLY;
        constexpr int PER2 = MEET > 0 ? (SECOND + MEET - 1) / MEET : SECOND;
        constexpr int PER1 = MEET < EARLY ? (FIRST + EARLY - MEET - 1) / (EARLY - MEET) : FIRST;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        Frag fa[FN], fb[2];
        float sc[2], ws;       // row scales, the weights' scale
        // Products whose sums are not taken yet, two and two: while two are multiplied, the
        // two before are added, so that neither waits for the other.  p[2] and p[3] are
        // left over at the end of a step, with their factors g0 and g1.
        f32x4_t p[4] = {};
        float g0 = 0.f, g1 = 0.f;
        auto meet0 = [&](int b) __attribute__((always_inline)) {
            if (b + 1 < nb) wait_loads<BH + FIRST>();   // after the scales of b: its second half, the first part of b + 1
            else wait_loads<0>();
            barrier_only();
        };
        auto meet1 = [&](int b) __attribute__((always_inline)) {
            if (b + 1 < nb) wait_loads<FIRST + SECOND>();   // both parts of b + 1
            else wait_loads<0>();
            barrier_only();
        };
        meet0(0);
#pragma unroll
        for (int i = 0; i < FN; ++i) fa[i] = read_a(sa0, i);
        fb[0] = read_b(sb0, 0);
        sc[0] = ss0[16 * wm + rl];
        ws = ss0[256 + 64 * (wv % WN) + lane];
        // (turns of the double buffers: NJ is even)
        auto stage = [&](uint8_t* __restrict__ ca, uint8_t* __restrict__ cbuf, float* __restrict__ cs,
                         uint8_t* __restrict__ na, uint8_t* __restrict__ nbuf, float* __restrict__ ns,
                         int b) __attribute__((always_inline)) {
            const bool more = b + 1 < nb;
            const float w = ws;
            auto next_reads = [&](int j) __attribute__((always_inline)) {
                fb[j & 1] = read_b(cbuf, j);
                sc[j & 1] = cs[16 * (2 * j + wm) + rl];
            };
            auto add = [&](f32x4_t& sum, const f32x4_t& v, float f) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[r] = __builtin_fmaf(v[r], f, sum[r]);
                __asm__("" : "+v"(sum));   // here, not where the sum is next read
            };
            auto loads_second = [&](int from, int to) __attribute__((always_inline)) {
                if (more)
#pragma unroll
                    for (int i = from; i < SECOND && i < to; ++i) second_part(i, nbuf, ns, b + 1);
            };
            auto loads_first = [&](int from, int to) __attribute__((always_inline)) {
                if (b + 2 < nb)
#pragma unroll
                    for (int i = from; i < FIRST && i < to; ++i) first_part(i, ca, cbuf, b + 2);
            };
            static_for8<0, EARLY>([&](auto J_) __attribute__((always_inline)) {
                constexpr int j = decltype(J_)::value, cur = j & 1;
                // this step's reads, issued a step ago (waited for by themselves: with loads
                // into LDS in between, the compiler would wait for the next ones too)
                wait_lds();
                if constexpr (j == MEET) {
                    if constexpr (MEET == 0) loads_second(0, SECOND);
                    meet1(b);
                }
                __builtin_amdgcn_sched_barrier(0);
                next_reads(j + 1);
                if constexpr (j < MEET) loads_second(j * PER2, (j + 1) * PER2);
                else loads_first((j - MEET) * PER1, (j - MEET + 1) * PER1);
                const float f = sc[cur] * w;
                __builtin_amdgcn_sched_barrier(0);
                p[0] = block_product<EXACT>(fa[0], fb[cur]);
                p[1] = block_product<EXACT>(fa[1], fb[cur]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (j == 0) {
                    add(acc[3][NJ - 2], p[2], g0);
                    add(acc[3][NJ - 1], p[3], g1);
                } else {
                    add(acc[2][j - 1], p[2], g0);
                    add(acc[3][j - 1], p[3], g0);
                }
                __builtin_amdgcn_sched_barrier(0);
                p[2] = block_product<EXACT>(fa[2], fb[cur]);
                p[3] = block_product<EXACT>(fa[3], fb[cur]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (j + 1 == EARLY) next_reads(NJ - 1);
                add(acc[0][j], p[0], f);
                add(acc[1][j], p[1], f);
                g0 = f;
                __builtin_amdgcn_sched_barrier(0);
            });
            // The last two steps together, by weight rows: as soon as a fragment of the
            // weights has met both, the next stage's is read in its place, beside the
            // products that follow.
            if constexpr (EARLY == 0) next_reads(NJ - 1);
            if constexpr (MEET == EARLY && MEET == 0) loads_second(0, SECOND);
            wait_lds();
            if constexpr (MEET == EARLY) {
                meet1(b);
                loads_first(0, FIRST);
            }
            if (more) meet0(b + 1);
            const float f0 = sc[0] * w, f1 = sc[1] * w;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                p[2 * (i & 1)] = block_product<EXACT>(fa[i], fb[0]);
                p[2 * (i & 1) + 1] = block_product<EXACT>(fa[i], fb[1]);
                __builtin_amdgcn_sched_barrier(0);
                if (more) fa[i] = read_a(na, i);
                if (i > 0) {
                    add(acc[i - 1][NJ - 2], p[2 * (1 - (i & 1))], f0);
                    add(acc[i - 1][NJ - 1], p[2 * (1 - (i & 1)) + 1], f1);
                } else if constexpr (EARLY > 0) {
                    add(acc[2][EARLY - 1], p[2], g0);
                    add(acc[3][EARLY - 1], p[3], g0);
                } else {
                    add(acc[3][NJ - 2], p[2], g0);
                    add(acc[3][NJ - 1], p[3], g1);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            g0 = f0;
            g1 = f1;
            if (more) {
                fb[0] = read_b(nbuf, 0);
                sc[0] = ns[16 * wm + rl];
                ws = ns[256 + 64 * (wv % WN) + lane];
            }
        };
        for (int b = 0; b < nb; b += 2) {
            stage(sa0, sb0, ss0, sa1, sb1, ss1, b);
            if (b + 1 < nb) stage(sa1, sb1, ss1, sa0, sb0, ss0, b + 1);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            acc[3][NJ - 2][r] = __builtin_fmaf(p[2][r], g0, acc[3][NJ - 2][r]);
            acc[3][NJ - 1][r] = __builtin_fmaf(p[3][r], g1, acc[3][NJ - 1][r]);
        }
    };

    Fp8Tile cur = decode(L);
    setup(cur);
    issue_tile();
    while (true) {
        // 16-row blocks wm, wm + 2, .. of the tile that hold rows
        const int blocks = (cur.valid + 15) >> 4, mine = max(0, (blocks - wm + 1) / 2);
        // a wave without rows still takes part in the loads and barriers
        static_for8<1, FM / 2 + 1>([&](auto H_) __attribute__((always_inline)) {
            constexpr int h = decltype(H_)::value;
            if (max(1, (mine + 1) / 2) == h) kloop(std::integral_constant<int, 2 * h>{}, cur);
        });

        L += nloc;
        const bool has_next = L < L_end;
        wait_lds();
        barrier_only();   // all waves have read the last stages
        Fp8Tile nxt = cur;
        if (has_next) {
            nxt = decode(L);
            setup(nxt);
            issue_tile();
        }
        // ---- results: 16 rows of 64 columns at a time through the wave's LDS, so that a
        // store covers whole runs of a row.  A wave's LDS operations complete in order.
        // (places from the lane number are made anew for every tile: kept over the K loop,
        // they would take registers that it needs)
        int ln = lane;
        __asm__ volatile("" : "+v"(ln));
        const int el = ln & 15, eg = ln >> 4;
        uint8_t* __restrict__ ep = ep_lds + wv * 16 * kEpRow;
        const int n0 = cur.n0 + wn0;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int mb = 16 * (2 * j + wm);
            if (mb >= cur.valid || n0 >= cols) continue;
            const size_t row0 = (size_t)cur.row0 + mb;
            if (a.out_bf16) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
                    *reinterpret_cast<uint2*>(ep + el * kEpRow + (16 * i + 4 * eg) * 2) =
                        make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int c = ln + 64 * s, r = c >> 3, q = c & 7;
                    const i32x4_t d = *reinterpret_cast<const i32x4_t*>(ep + r * kEpRow + q * 16);
                    if (mb + r < cur.valid && n0 + 8 * q < cols)
                        __builtin_nontemporal_store(
                            d, reinterpret_cast<i32x4_t*>(static_cast<bf16_t*>(a.out) + (row0 + r) * cols + n0 + 8 * q));
                }
            } else {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int i = 2 * hh; i < 2 * hh + 2; ++i)
                        *reinterpret_cast<f32x4_t*>(ep + el * kEpRow + ((i - 2 * hh) * 16 + 4 * eg) * 4) = acc[i][j];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = ln + 64 * s, r = c >> 3, q = c & 7, n = n0 + 32 * hh + 4 * q;
                        const f32x4_t d = *reinterpret_cast<const f32x4_t*>(ep + r * kEpRow + q * 16);
                        if (mb + r < cur.valid && n < cols)
                            __builtin_nontemporal_store(
                                d, reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (row0 + r) * cols + n));
                    }
                }
            }
        }
        if (!has_next) break;
        cur = nxt;
    }
}

}  // namespace

}  // namespace inkling
