// Grouped matrix products on 64 x 64 tiles, one tile a workgroup: fp32 products, and
// bf16 ones with too few large tiles to fill the card, or few rows an expert against
// small weights (gfx950; the rules and both sides' times are in grouped.hip).
//
//   out[m][n] = sum_k B[m][k] A[n][k] over the rows m of one expert, as
//   kProdRows   A = weight [n][k], B = rows (gathered through row_index), K = in_features
//   kProdDx     A = weight read as [k][n], B = rows,                    K = out_features
//   kProdWgrad  A = x and B = dout, both read as [k][...],              K = the expert's rows
//
// A short call is latency: one launch, no plan before it (each wave finds its
// tile in the caller's offsets with a scan over lanes), and a K loop whose four
// stages ahead wait in registers, so that HBM's latency is paid about once.  A
// stage is 128 bytes of K a row (64 bf16, 32 fp32), written to one of two LDS
// buffers with rows padded by 16 bytes; four waves hold 32 x 32 each.
#pragma once

#include "gemm_kernel.h"

namespace inkling {

namespace {

enum { kProdRows = 0, kProdDx = 1, kProdWgrad = 2 };

struct SmallArgs {
    const void* A;              // weights [E][N][K] or [E][K][N]; kProdWgrad: x rows [..][N]
    const void* B;              // rows [..][K]; kProdWgrad: dout rows [rows][M]
    const int32_t* offsets;     // [E + 1], the caller's
    const int32_t* row_index;   // row r of the rows (kProdWgrad: of x) is row row_index[r] (NULL: r)
    int src_rows;
    int rows, E, K, N, M;       // N: columns of out; M: kProdWgrad, rows of out
    int ntn, ntm;               // column tiles; kProdWgrad: row tiles
    void* out;                  // [rows][N]; kProdWgrad: [E][M][N]
    int out_bf16;
};

// The rows [begin, end) of expert e, with the caller's offsets clamped to the
// rows and raised to the largest before them.
struct Span {
    int begin, end;
};
__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v = max(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ Span expert_span(const SmallArgs& a, int e) {
    int v = 0;
    for (int i = lane_id(); i <= e; i += kWave) v = max(v, min(a.offsets[i], a.rows));
    const int begin = wave_max(v);
    return {begin, max(begin, min(a.offsets[e + 1], a.rows))};
}

// The expert and first row of row tile `tile` (tiles of 64 rows in expert
// order); expert -1 past the last.  Lane l scans experts l C .. l C + C - 1.
struct RowTile {
    int expert, row0, end;
};
__device__ __forceinline__ RowTile find_row_tile(const SmallArgs& a, int tile) {
    const int lane = lane_id(), C = (a.E + kWave - 1) / kWave, e0 = lane * C;
    const int first = max(0, min(a.offsets[0], a.rows));
    int top = first;
    for (int c = 0; c < C; ++c)
        if (e0 + c < a.E) top = max(top, min(a.offsets[e0 + c + 1], a.rows));
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(top, d);
        if (lane >= d) top = max(top, o);
    }
    int start = __shfl_up(top, 1);   // end of the expert before this lane's first
    if (lane == 0) start = first;
    int cur = start, n = 0;
    for (int c = 0; c < C; ++c)
        if (e0 + c < a.E) {
            const int end = max(cur, min(a.offsets[e0 + c + 1], a.rows));
            n += (end - cur + 63) >> 6;
            cur = end;
        }
    int incl = n;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    RowTile t = {-1, 0, 0};
    int before = incl - n;
    if (before <= tile && tile < incl) {   // one lane, or none past the last tile
        cur = start;
        for (int c = 0; c < C; ++c)
            if (e0 + c < a.E) {
                const int end = max(cur, min(a.offsets[e0 + c + 1], a.rows)), k = (end - cur + 63) >> 6;
                if (t.expert < 0 && tile < before + k) t = {e0 + c, cur + ((tile - before) << 6), end};
                before += k;
                cur = end;
            }
    }
    const unsigned long long has = __ballot(t.expert >= 0);
    if (has == 0) return {-1, 0, 0};
    const int src = __ffsll(has) - 1;
    return {__shfl(t.expert, src), __shfl(t.row0, src), __shfl(t.end, src)};
}

template <typename TE, int MODE>
__global__ __launch_bounds__(256) void small_product_kernel(const SmallArgs a) {
    constexpr bool AKN = MODE != kProdRows, BKN = MODE == kProdWgrad;
    constexpr int ES = sizeof(TE), EPC = 16 / ES;       // values of a 16-byte chunk
    constexpr int BK = 128 / ES;                        // K of a stage
    constexpr int D = 4;                                // stages in registers
    // K-major: 64 rows of 128 bytes; [K][...]: BK rows of 64 values
    constexpr int KN_PITCH = 64 * ES + 16, PITCH_A = AKN ? KN_PITCH : 144, PITCH_B = BKN ? KN_PITCH : 144;
    constexpr int SIZE_A = AKN ? BK * KN_PITCH : 64 * 144, SIZE_B = BKN ? BK * KN_PITCH : 64 * 144;
    __shared__ __attribute__((aligned(16))) uint8_t sa[2][SIZE_A];
    __shared__ __attribute__((aligned(16))) uint8_t sb[2][SIZE_B];
    const TE* A = static_cast<const TE*>(a.A);
    const TE* B = static_cast<const TE*>(a.B);
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- tile --------------------------------------------------------------------
    int n0, m0, rows, K;    // first column, first row of out, rows of the tile
    char* out = static_cast<char*>(a.out);
    const int ob = a.out_bf16 ? 2 : 4;
    int r0 = 0;             // kProdWgrad: the expert's first row
    if constexpr (MODE == kProdWgrad) {
        const int per = a.ntm * a.ntn, e = blockIdx.x / per, l = blockIdx.x - e * per;
        const Span s = expert_span(a, e);
        r0 = s.begin;
        K = s.end - s.begin;
        m0 = l / a.ntn * 64;
        n0 = l % a.ntn * 64;
        rows = min(64, a.M - m0);
        B += (size_t)r0 * a.M;
        out += (size_t)e * a.M * a.N * ob;
    } else {
        const RowTile t = find_row_tile(a, blockIdx.x / a.ntn);
        if (t.expert < 0) return;   // the whole workgroup
        K = a.K;
        m0 = t.row0;
        n0 = blockIdx.x % a.ntn * 64;
        rows = min(64, t.end - t.row0);
        A += (size_t)t.expert * a.N * a.K;
    }

    // ---- loads: two chunks of each operand a stage and thread -----------------------
    // K-major: rows tid / 8 and + 32, chunk tid % 8; [K][...]: K rows of 64 values
    constexpr int CPR = 64 * ES / 16, RPP = 256 / CPR;   // chunks of a [K][...] row, rows of a pass
    const int kr = AKN || BKN ? tid / CPR : 0, kc = AKN || BKN ? tid % CPR : 0;
    const int mr = tid >> 3, mc = tid & 7;
    const TE* a_src[2];
    const TE* b_src[2];
    bool a_ok[2], b_ok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (AKN) {
            a_ok[i] = n0 + kc * EPC < a.N;
            a_src[i] = A + n0 + kc * EPC;       // + the K row
        } else {
            a_ok[i] = n0 + mr + 32 * i < a.N;
            a_src[i] = A + (size_t)(n0 + mr + 32 * i) * a.K + mc * EPC;
        }
        if constexpr (BKN) {
            b_ok[i] = m0 + kc * EPC < a.M;
            b_src[i] = B + m0 + kc * EPC;
        } else {
            const int r = mr + 32 * i;
            b_ok[i] = r < rows;
            size_t row = (size_t)m0 + r;
            if (MODE == kProdRows && a.row_index != nullptr && b_ok[i])   // an index out of range reads a row in it
                row = (size_t)max(0, min(a.row_index[m0 + r], a.src_rows - 1));
            b_src[i] = B + row * a.K + mc * EPC;
        }
    }
    uint4 ra[D][2], rb[D][2];
    auto load = [&](auto S_, int k0) __attribute__((always_inline)) {
        constexpr int s = decltype(S_)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ra[s][i] = make_uint4(0, 0, 0, 0);
            rb[s][i] = make_uint4(0, 0, 0, 0);
            const int k = k0 + kr + RPP * i;   // K row of a [K][...] stage
            if constexpr (AKN) {
                if (a_ok[i] && k < K) {
                    size_t row = (size_t)k;
                    if constexpr (MODE == kProdWgrad) {
                        row = (size_t)r0 + k;
                        if (a.row_index != nullptr) row = (size_t)max(0, min(a.row_index[r0 + k], a.src_rows - 1));
                    }
                    ra[s][i] = *reinterpret_cast<const uint4*>(a_src[i] + row * a.N);
                }
            } else if (a_ok[i] && k0 + mc * EPC < K) {
                ra[s][i] = *reinterpret_cast<const uint4*>(a_src[i] + k0);
            }
            if constexpr (BKN) {
                if (b_ok[i] && k < K) rb[s][i] = *reinterpret_cast<const uint4*>(b_src[i] + (size_t)k * a.M);
            } else if (b_ok[i] && k0 + mc * EPC < K) {
                rb[s][i] = *reinterpret_cast<const uint4*>(b_src[i] + k0);
            }
        }
    };
    auto put = [&](auto S_, int buf) __attribute__((always_inline)) {
        constexpr int s = decltype(S_)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pa = AKN ? (kr + RPP * i) * PITCH_A + kc * 16 : (mr + 32 * i) * PITCH_A + mc * 16;
            const int pb = BKN ? (kr + RPP * i) * PITCH_B + kc * 16 : (mr + 32 * i) * PITCH_B + mc * 16;
            *reinterpret_cast<uint4*>(sa[buf] + pa) = ra[s][i];
            *reinterpret_cast<uint4*>(sb[buf] + pb) = rb[s][i];
        }
    };

    // ---- fragments: 64 bytes of K a k-step (32 bf16, 16 fp32) ------------------------
    const int an = 32 * (wv & 1), bm = 32 * (wv >> 1), rl = lane & 15, g = lane >> 4;
    auto frag = [&](const uint8_t* st, auto KN_, int pitch, int r, int ks) __attribute__((always_inline)) -> uint4 {
        if constexpr (!decltype(KN_)::value) {
            return *reinterpret_cast<const uint4*>(st + (r + rl) * pitch + (4 * ks + g) * 16);
        } else if constexpr (ES == 2) {
            // lane addresses 4 columns of K row 8 g + (lane / 4) % 4 (see read_tr16_frag)
            return read_tr16_frag(st + (32 * ks + 8 * g + ((lane >> 2) & 3)) * pitch + (r + 4 * (lane & 3)) * 2, pitch);
        } else {
            const uint8_t* p = st + (16 * ks + 4 * g) * pitch + (r + rl) * 4;
            uint4 v;
            v.x = *reinterpret_cast<const uint32_t*>(p);
            v.y = *reinterpret_cast<const uint32_t*>(p + pitch);
            v.z = *reinterpret_cast<const uint32_t*>(p + 2 * pitch);
            v.w = *reinterpret_cast<const uint32_t*>(p + 3 * pitch);
            return v;
        }
    };
    // 16-blocks of the wave that hold columns and rows: the others are skipped (an
    // fp32 tile of few rows would be bound by the products of its empty ones)
    const int nvi = (a.N - n0 - an + 15) >> 4, nvj = (rows - bm + 15) >> 4;
    f32x4_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int ns = (K + BK - 1) / BK;
    static_for<0, D>([&](auto S_) { load(S_, decltype(S_)::value * BK); });   // past K: zeros, nothing read
    for (int s0 = 0; s0 < ns; s0 += D)
        static_for<0, D>([&](auto S_) __attribute__((always_inline)) {
            constexpr int s = decltype(S_)::value, buf = s & 1;
            if (s0 + s < ns) {
                // this buffer was last read two stages ago, before the barrier of the stage between
                put(S_, buf);
                load(S_, (s0 + s + D) * BK);
                wait_lgkmcnt0();
                barrier_keep_loads();
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    uint4 fa[2], fb[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        fa[i] = frag(sa[buf], std::integral_constant<bool, AKN>{}, PITCH_A, an + 16 * i, ks);
                        fb[i] = frag(sb[buf], std::integral_constant<bool, BKN>{}, PITCH_B, bm + 16 * i, ks);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (i < nvi && j < nvj) mma16<TE>(acc[i][j], fa[i], fb[j]);
                }
            }
        });

    // acc[i][j][r]: column an + 16 i + 4 (lane / 16) + r of row bm + 16 j + lane % 16
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = bm + 16 * j + rl, n = n0 + an + 16 * i + 4 * g;
            if (m < rows && n < a.N) {
                const size_t at = (size_t)(m0 + m) * a.N + n;
                if (a.out_bf16) *reinterpret_cast<uint2*>(out + 2 * at) = pack_bf16x4(acc[i][j]);
                else *reinterpret_cast<f32x4_t*>(out + 4 * at) = acc[i][j];
            }
        }
}

}  // namespace

}  // namespace inkling
