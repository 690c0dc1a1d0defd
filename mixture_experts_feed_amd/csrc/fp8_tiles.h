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
#pragma once

#include "fp8_common.h"

namespace inkling {

namespace {

constexpr int kTileThreads = 512;

struct Fp8Tile {
    int e, row0, valid, n0;   // expert; first row and rows of the tile; first output column
};

// KN: the input gradient (weights read as [reduction][column])
template <bool KN, bool EXACT>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_tile_kernel(const Fp8Args a) {
    constexpr int BN = 256, BM = 256, WN = 4, NW = 8, FN = 4, FM = 8;
    constexpr int STAGE = 256 * kQBlock;
    // each stage its own object: the compiler then needs no wait for the loads into one
    // before reads of the other
    __shared__ __attribute__((aligned(16))) uint8_t sa0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t sa1[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t sb0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t sb1[STAGE];
    __shared__ __attribute__((aligned(16))) float ss0[BM];
    __shared__ __attribute__((aligned(16))) float ss1[BM];
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
    plan_experts<kTileThreads, BM>(a, offs, first);
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
        t.row0 = __builtin_amdgcn_readfirstlane(offs[t.e] + mt * BM);
        t.valid = __builtin_amdgcn_readfirstlane(min(BM, offs[t.e + 1] - t.row0));
        t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
        return t;
    };

    // ---- loads -------------------------------------------------------------------
    // 128-byte rows (token rows; weights of the forward): the 16-byte chunk c of row r
    // sits at chunk place c ^ (r & 7); 256-byte rows (weights of the input gradient, a
    // row of the reduction each): at c ^ swk(r).  Both keep the reads below spread over
    // the banks.
    auto swk = [](int r) { return (r & 7) | ((r >> 1) & 8); };
    // a wave load is 1 KB: eight 128-byte rows (lane / 8 of them; chunk place lane % 8)
    // or four 256-byte rows
    const int c16 = 16 * ((lane & 7) ^ (lane >> 3));   // the lane's chunk of its 128-byte rows
    const uint8_t* a_base = nullptr;    // this expert's weights, from the tile's first row
    uint32_t a_off[4];                  // the lane's four chunks of a stage, from a_base
    const uint8_t* b_src[4];
    const float* s_src = nullptr;
    int ld_block = 0, ld_valid = 1;
    auto setup = [&](const Fp8Tile& t) __attribute__((always_inline)) {
        a_base = a.weight + (size_t)t.e * a.N * a.K + (KN ? 0 : (size_t)t.n0 * a.K);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (KN) {
                const int r = 4 * (wv + NW * q) + (lane >> 4);
                const int c = (lane & 15) ^ swk(r);
                a_off[q] = (uint32_t)r * a.K + min(t.n0 + 16 * c, a.K - 16);   // columns past the end: the last chunk
            } else {
                const int r = 8 * (wv + NW * q) + (lane >> 3);
                a_off[q] = (uint32_t)min(r, a.N - 1 - t.n0) * a.K + c16;       // rows past the end: the last row
            }
            int row = t.row0 + min(8 * (wv + NW * q) + (lane >> 3), t.valid - 1);
            if (!KN && a.row_index != nullptr) row = max(0, min(a.row_index[row], a.x_rows - 1));
            b_src[q] = a.x + (size_t)row * len + c16;
        }
        if (wv < 4) {
            int row = t.row0 + min(64 * wv + lane, t.valid - 1);
            if (!KN && a.row_index != nullptr) row = max(0, min(a.row_index[row], a.x_rows - 1));
            s_src = a.x_scale + (size_t)row * nb;
        }
        ld_block = 0;
        ld_valid = t.valid;
    };
    auto issue = [&](uint8_t* da, uint8_t* db, float* ds) __attribute__((always_inline)) {
        const int k0 = ld_block * kQBlock;
        if (wv < 4)
            __builtin_amdgcn_global_load_lds((fp8_glb_t*)(s_src + ld_block), (fp8_lds_t*)(ds + 64 * wv), 4, 0, 0);
        const uint8_t* ab = a_base + (KN ? (size_t)k0 * a.K : (size_t)k0);
        if (k0 + kQBlock <= len) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (8 * (wv + NW * q) < ld_valid) copy16_to_lds<0>(b_src[q] + k0, db + (wv + NW * q) * 1024);
#pragma unroll
            for (int q = 0; q < 4; ++q) copy16_to_lds<0>(ab + a_off[q], da + (wv + NW * q) * 1024);
        } else {
            // the stage of the tail: what lies past it reads zeros
            const uint8_t* zero = reinterpret_cast<const uint8_t*>(&fp8_zero_chunk);
            const bool in = c16 < len - k0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (8 * (wv + NW * q) < ld_valid)
                    copy16_to_lds<0>(in ? b_src[q] + k0 : zero, db + (wv + NW * q) * 1024);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool there = KN ? 4 * (wv + NW * q) + (lane >> 4) < len - k0 : in;
                copy16_to_lds<0>(there ? ab + a_off[q] : zero, da + (wv + NW * q) * 1024);
            }
        }
        ++ld_block;
    };

    // ---- fragments -----------------------------------------------------------------
    const int p0 = (g ^ (rl & 7)) << 4, p1 = ((4 + g) ^ (rl & 7)) << 4;   // places of chunks g and 4 + g
    const int a_row = (wn0 + rl) * kQBlock, b_row = (16 * wm + rl) * kQBlock;
    // input gradient: lane 2 j + h of 16 addresses half h of the 16 columns' chunk in
    // reduction row j of eight; the transposing read hands lane c the eight rows of column c
    const int tr_sz = (rl >> 1) | ((g & 1) << 3);
    const int tr_at = (16 * g + (rl >> 1)) * 256 + (((wn0 >> 4) ^ tr_sz) << 4) + (rl & 1) * 8;
    auto read_a = [&](const uint8_t* __restrict__ st, int i) __attribute__((always_inline)) {
        Frag f;
        if constexpr (KN) {
            const uint8_t* p = st + (tr_at ^ (i << 4));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                f.quarter[q] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (fp8_lds_i32x2_t*)(p + ((q & 1) * 8 + (q >> 1) * 64) * 256));
        } else {
            f.half[0] = *reinterpret_cast<const i32x4_t*>(st + a_row + i * 16 * kQBlock + p0);
            f.half[1] = *reinterpret_cast<const i32x4_t*>(st + a_row + i * 16 * kQBlock + p1);
        }
        return f;
    };
    auto read_b = [&](const uint8_t* __restrict__ st, int j) __attribute__((always_inline)) {
        Frag f;
        f.half[0] = *reinterpret_cast<const i32x4_t*>(st + b_row + j * 32 * kQBlock + p0);
        f.half[1] = *reinterpret_cast<const i32x4_t*>(st + b_row + j * 32 * kQBlock + p1);
        return f;
    };

    f32x4_t acc[FN][FM];
    // weight scale of block b for this wave's columns
    auto weight_scale = [&](const Fp8Tile& t, int b) __attribute__((always_inline)) {
        const int c = min((t.n0 + wn0) / kQBlock, cb - 1);
        const int kb = (a.K + kQBlock - 1) / kQBlock;
        const int at = KN ? b * kb + c : c * kb + b;
        return scalar_load(a.weight_scale + (size_t)t.e * cb * nb + at);
    };

    // NJ: 16-row blocks of the wave that are multiplied (the others hold no rows).
    //
    // A stage takes a step a row block: its four products, the sums of the step before,
    // and the LDS reads of the next step.  Before the last step, all of whose reads are
    // done: wait for the next stage's loads, meet, load the stage after it into the
    // buffers just read; the next stage's first reads run beside the last products.
    auto kloop = [&](auto NJ_, const Fp8Tile& t) __attribute__((always_inline)) {
        constexpr int NJ = decltype(NJ_)::value;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        Frag fa[FN], fb[2];
        f32x4_t p[2][FN];      // products of a step
        float f[2], sc[2];     // their factor; row scales
        float ws = weight_scale(t, 0);
        // add the products of step (row block) j
        auto add = [&](auto J_, int turn) __attribute__((always_inline)) {
            constexpr int j = decltype(J_)::value;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[turn][i][r], f[turn], acc[i][j][r]);
                __asm__("" : "+v"(acc[i][j]));   // here, not where the sum is next read
            }
        };
        wait_loads<0>();
        barrier_only();
        if (nb > 1) issue(sa1, sb1, ss1);
#pragma unroll
        for (int i = 0; i < FN; ++i) fa[i] = read_a(sa0, i);
        fb[0] = read_b(sb0, 0);
        sc[0] = ss0[16 * wm + rl];
        // (turns of the double buffers: NJ is even)
        auto stage = [&](const uint8_t* __restrict__ ca, const uint8_t* __restrict__ cbuf, const float* __restrict__ cs,
                         const uint8_t* __restrict__ na, const uint8_t* __restrict__ nbuf,
                         const float* __restrict__ ns, uint8_t* wa, uint8_t* wb, float* wsc,
                         int b) __attribute__((always_inline)) {
            const bool more = b + 1 < nb;
            const float w = ws;
            if (more) ws = weight_scale(t, b + 1);
            static_for8<0, NJ>([&](auto J_) __attribute__((always_inline)) {
                constexpr int j = decltype(J_)::value, cur = j & 1;
                if constexpr (j + 1 < NJ) {
                    fb[cur ^ 1] = read_b(cbuf, j + 1);
                    sc[cur ^ 1] = cs[16 * (2 * (j + 1) + wm) + rl];
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < FN; ++i) p[cur][i] = block_product<EXACT>(fa[i], fb[cur]);
                } else {
                    if (more) {
                        wait_lds();
                        wait_loads<0>();
                        barrier_only();
                        if (b + 2 < nb) issue(wa, wb, wsc);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < FN; ++i) p[cur][i] = block_product<EXACT>(fa[i], fb[cur]);
                }
                f[cur] = sc[cur] * w;
                if constexpr (j > 0) add(std::integral_constant<int, j - 1>{}, cur ^ 1);
                else if (b > 0) add(std::integral_constant<int, NJ - 1>{}, cur ^ 1);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (j + 1 == NJ) {
                    if (more) {
#pragma unroll
                        for (int i = 0; i < FN; ++i) fa[i] = read_a(na, i);
                        fb[0] = read_b(nbuf, 0);
                        sc[0] = ns[16 * wm + rl];
                    }
                }
            });
        };
        for (int b = 0; b < nb; b += 2) {
            stage(sa0, sb0, ss0, sa1, sb1, ss1, sa0, sb0, ss0, b);
            if (b + 1 < nb) stage(sa1, sb1, ss1, sa0, sb0, ss0, sa1, sb1, ss1, b + 1);
        }
        add(std::integral_constant<int, NJ - 1>{}, 1);
    };

    Fp8Tile cur = decode(L);
    setup(cur);
    issue(sa0, sb0, ss0);
    while (true) {
        // 16-row blocks wm, wm + 2, .. of the tile that hold rows
        const int blocks = (cur.valid + 15) >> 4, mine = max(0, (blocks - wm + 1) / 2);
        // a wave without rows still takes part in the loads and barriers
        if (mine > 6) kloop(std::integral_constant<int, 8>{}, cur);
        else if (mine > 4) kloop(std::integral_constant<int, 6>{}, cur);
        else if (mine > 2) kloop(std::integral_constant<int, 4>{}, cur);
        else kloop(std::integral_constant<int, 2>{}, cur);

        L += nloc;
        const bool has_next = L < L_end;
        wait_lds();
        barrier_only();   // all waves have read the last stages
        Fp8Tile nxt = cur;
        if (has_next) {
            nxt = decode(L);
            setup(nxt);
            issue(sa0, sb0, ss0);
        }
        // ---- results: 16 rows of 64 columns at a time through the wave's LDS, so that a
        // store covers whole runs of a row.  A wave's LDS operations complete in order.
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
                    *reinterpret_cast<uint2*>(ep + rl * kEpRow + (16 * i + 4 * g) * 2) =
                        make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int c = lane + 64 * s, r = c >> 3, q = c & 7;
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
                        *reinterpret_cast<f32x4_t*>(ep + rl * kEpRow + ((i - 2 * hh) * 16 + 4 * g) * 4) = acc[i][j];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = lane + 64 * s, r = c >> 3, q = c & 7, n = n0 + 32 * hh + 4 * q;
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
