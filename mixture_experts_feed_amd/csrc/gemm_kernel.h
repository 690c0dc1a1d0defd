// Grouped expert GEMM kernel of the Inkling MoE on gfx950 matrix cores, and its
// device helpers (launched from gemm.hip).
//
// Every expert product here is out[row][n] = sum_k W[n][k] * X[row][k] with
// both operands K-contiguous (nn.Linear weights [out, in] and row-major token
// rows).  The weights are the MFMA A operand (MFMA rows = output columns n) and
// the token rows the B operand (MFMA columns = tokens), so each lane's 16x16
// accumulator holds four consecutive output columns of one token.  For the
// gate_up projection those four columns are [g_j, u_j, g_j+1, u_j+1] of the
// interleaved layout (inkling_swiglu on the Inkling layers page: ::2 gate,
// 1::2 up), so SwiGLU and the routing-weight scale are applied in registers.
//
// Launches per forward:
//   gate_up  routed tiles (rows gathered through the expert-sorted token list,
//            scaled by that slot's gamma) and shared tiles (all tokens against
//            the S shared experts concatenated along N, scaled by the token's
//            shared gamma) -> act_r, act_sh (fp16 for bf16 layers, see ActOf);
//   down     routed: act_r rows of each expert -> y, one fp32 row per routed
//            slot t*k + i (rows of a token are adjacent);
//   down_out shared: act_sh [T][S*I] against the shared down weights
//            concatenated along K, so the sum over shared experts happens
//            inside the reduction; the epilogue adds the token's k routed y
//            rows and rounds once: out[t] = shared + sum_i y[t*k + i].  (Two
//            launches: a token's y rows come from tiles on every XCD, and the
//            launch boundary is what makes them visible to the other XCDs' L2.)
//   combine  only without shared experts: out[t] = sum_i y[t*k + i].
// The backward reuses the same kernel with other epilogues and operands (see
// the modes below and backward.hip).  Its products contract over the other
// index of a stored matrix (the down weights over H, the gate_up weights over
// 2I, activations over their rows), so those operands are read in their
// stored [K][N] layout: K rows of N contiguous elements are copied to LDS as
// they are, and the CDNA4 transposing LDS read (ds_read_b64_tr_b16) turns four
// K rows of a column block into the per-lane K runs the MFMA takes.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "tile_ranges.h"

namespace inkling {

namespace {

// kModeGateUp: SwiGLU * gamma epilogue -> activation rows (TE)
// kModeDown: fp32 rows (routed rows go to their slot row)
// kModeGateUpRaw: the gate_up projection itself -> h rows (fp32) (backward recompute)
// kModeDAct: backward through down and SwiGLU: acc = dact; epilogue writes
//            dh = d[gate, up] (TE), a = gamma * silu(g) * u (TE) and per-64-column
//            partial sums of dact . silu(g) * u (the routing-weight gradient)
// kModeWgrad: weight gradients, one problem per expert, K = that expert's rows
// kModeDx: backward through gate_up: the down epilogue (fp32 rows)
// kModeDownOut: the shared down projection with the combine in its epilogue:
//            out[t] = (shared sum) + sum_i y[t*k + i], in fp32 in that order,
//            rounded once to the output type (shared tiles only)
// The products that callers reach on their own (grouped.hip); K and N are any
// multiples of 8 there, and a K tail reads zeros for both operands:
// kModeGroup: out[r][n] = sum_k W_e[n][k] x[row of r][k], rounded once
// kModeGroupDx: dx[r][n] = sum_k W_e[k][n] dout[r][k], rounded once
// kModeGroupWgrad: dW_e[m][n] = sum_r dout[r][m] x[r][n]
// A is read as [K][N] in kModeDAct, kModeDx, kModeGroupDx and the two
// weight-gradient modes, B in the latter.
enum { kModeGateUp = 0, kModeDown = 1, kModeGateUpRaw = 2, kModeDAct = 3, kModeWgrad = 4, kModeDx = 5,
       kModeDownOut = 6, kModeGroup = 7, kModeGroupDx = 8, kModeGroupWgrad = 9 };
template <int MODE>
constexpr bool grouped_mode() { return MODE == kModeGroup || MODE == kModeGroupDx || MODE == kModeGroupWgrad; }
template <int MODE>
constexpr bool wgrad_mode() { return MODE == kModeWgrad || MODE == kModeGroupWgrad; }
template <int MODE>
constexpr bool a_kn() { return MODE == kModeDAct || MODE == kModeDx || MODE == kModeGroupDx || wgrad_mode<MODE>(); }
template <int MODE>
constexpr bool b_kn() { return wgrad_mode<MODE>(); }
// How the workgroups of an XCD walk its range of tiles after their first:
// kSchedStride: with stride = workgroups per XCD;
// kSchedRound: the same, meeting at the end of every round of tiles (below);
// kSchedQueue: each takes the next tile of the range from the XCD's counter,
//              so the tiles in flight on an XCD stay a contiguous window of
//              the range.
// kSchedGroup: each takes the next tile from the counter once it is free, then
//              waits (at most kSpinLimit polls) until every tile of its partner
//              group (the row tiles that read its weight tile, at most
//              kGroupMax of them) has been taken, so that they start together.
enum { kSchedStride = 0, kSchedRound = 1, kSchedQueue = 2, kSchedGroup = 3 };
constexpr int kGroupMax = 8;
constexpr int kSpinLimit = 400;   // polls of a tile-round wait (about 100-400 us at most)
// Cache policy of the weight (A) loads.  Tiles of at most 16 token rows (the
// decode configuration) read each weight byte once per call: those loads carry
// the non-temporal bit, which streams the weights at about 6.7 TB/s instead of
// 5.9.  Larger tiles share weight tiles through L2 and keep the default policy
// (non-temporal weights there slowed the down projection by 6%).
constexpr int kPolicyNT = 2;      // nt bit of a global load's cache-policy operand

typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void glb_void_t;

struct GemmKArgs {
    const void* A_routed;   // [E][N_r][K_r]
    const void* A_shared;   // see seg_s
    const void* B_routed;   // x [T][H] (gate_up, gathered) or act_r [T*k][I]
    const void* B_shared;   // x [T][H] or act_sh [T][S*I]
    const RoutedTile* tiles;
    const int32_t* num_tiles;
    const int32_t* offsets;
    const int32_t* row_token;
    const int32_t* row_slot;   // sorted row -> slot t*k + i
    const float* row_gamma;
    const float* shared_g;
    void* out_routed;          // gate_up: act_r [T*k][I] (sorted rows); down: y [T*k][H] (slot rows, TA)
    void* out_shared;          // gate_up: act_sh [T][S*I]; dx: the shared rows [T][H] fp32
    int T, H, I, S, k;
    int K_r, N_r, ntn_r;    // routed problem: K, N per expert, N tiles
    int K_s, N_s, ntn_s;    // shared problem
    int seg_s;              // shared A(n, kk) = A_shared + (kk/seg)*N_s*seg + n*seg + kk%seg
    int shared_blocks, shared_mtiles;
    int has_routed;
    int32_t* round_counter;    // [8] per XCD, zero at launch: tiles finished (kSchedRound) or taken (queue, group)
    // kModeDAct
    const void* h_routed;      // [T*k][2I] sorted rows, fp32
    const void* h_shared;      // [T][S*2I] fp32
    void* a_routed;            // [T*k][I] sorted rows
    void* a_shared;            // [T][S*I]
    float* dgp_routed;         // [T*k][I/64]
    float* dgp_shared;         // [T][S*I/64]
    // kModeGateUp: optional fp32 copies of the projection (NULL: none), as
    // h_routed / h_shared above
    float* h_save_routed;
    float* h_save_shared;
    // operands read as [K][N]: row strides; the shared A of kModeDAct holds the
    // S experts side by side along N (column n at element (n / a_segn_s) *
    // a_segstride_s + n % a_segn_s of a row)
    int lda_r, lda_s, ldb_r, ldb_s;
    int a_segn_s;
    long long a_segstride_s;
    // kModeWgrad: problems e < E (routed: K = rows offsets[e].. of e, padded to
    // poff[e+1] - poff[e]) then s < S (shared: K = K_s rows of which T are
    // tokens); out[m][n] = sum_k B[k][m] A[k][n]; padding rows of B read `zero`
    const int32_t* poff;       // [E+1] prefix sums of the padded row counts
    const void* zero;          // a zero row, at least wg_M elements
    long long a_sh_stride, b_sh_stride;   // element offset of shared problem s in A / B
    int wg_E, wg_M, wg_N, wg_mtiles, wg_ntiles;
    void* w_out_routed;        // [E][M][N], fp32 or (w_out_bf16) bf16
    void* w_out_shared;        // [S][M][N]
    int w_out_bf16;
    // kModeDownOut: the routed rows of each token (slot rows t*k + i, fp16 for
    // bf16 layers, fp32 for fp32 ones), slot -> sorted row (-1 for every slot
    // of a padded token), the layer output [T][H] and its type (1: bf16)
    const void* y_rows;
    const int32_t* pos;
    void* out_final;
    int out_final_bf16;
    // kModeGroup, kModeGroupWgrad: T is the rows of x, which row_token gathers
    // from (row_token NULL: row r reads row r); kModeGroup, kModeGroupDx: out_final_bf16 is the type
    // of out_routed
};

// an int at an address that is the same for the whole wave, written by an earlier
// kernel only: a scalar load, which the waits for vector loads do not count
__device__ __forceinline__ int uniform_load(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)p;
}

// what the lanes past a K tail load (16 bytes serve every lane)
__device__ uint4 zero_chunk = {0u, 0u, 0u, 0u};

// 16 bytes of a result.  PAST: past the caches, for the grouped products, whose
// results nothing in the same launch reads again.  The operands then keep the L2,
// and a wave gets over its stores sooner: weight gradients of 64 experts of 384
// rows (2048 x 1536) 352 to 287 us in fp32 and 261 to 187 in bf16, of 16 of 512
// (2048 x 6144) 303 to 238; forward and input gradient 1 to 5% less.  Two products
// with the SwiGLU between them, which reads the first at once: 418 to 401 at 128 of
// 128 (2048 wide), 105 to 107 at the worst (16 of 512, 1024 wide).
template <bool PAST>
__device__ __forceinline__ void store16(void* p, f32x4_t v) {
    if constexpr (PAST) __builtin_nontemporal_store(v, static_cast<f32x4_t*>(p));
    else *static_cast<f32x4_t*>(p) = v;
}

typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
// four fp32 -> bf16, nearest even, NaN kept (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint2 pack_bf16x4(const f32x4_t& v) {
    return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4_t));
}

template <typename TE>
__device__ __forceinline__ void mma16(f32x4_t& acc, const uint4& a, const uint4& b);

template <>
__device__ __forceinline__ void mma16<bf16_t>(f32x4_t& acc, const uint4& a, const uint4& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                  acc, 0, 0, 0);
}

template <>
__device__ __forceinline__ void mma16<float>(f32x4_t& acc, const uint4& a, const uint4& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), acc, 0, 0, 0);
}

// The activation between the two projections of a bf16 layer is kept in fp16,
// not bf16: act = gamma silu(g) u is rounded once before the down projection,
// and fp16's 11-bit significand makes that rounding 8x smaller than bf16's.
// The routed experts' output rows y (summed per token by the combine) are
// fp16 too, which halves their round trip through HBM; with fp16 act and fp16
// y the skewed workload's error is about 5e-3 of the output RMS (bf16 y alone
// would add about 3e-2).  Both must stay below 65504 in magnitude.
// (On heavy-tailed inputs, where rows of 4x the norm give outputs far above the
// RMS, the bf16 rounding alone reaches about 2.6e-2 of the output RMS; fp16
// gives about 3e-3.)  The down weights stay bf16 in memory and are converted to
// fp16 as MFMA fragments, which is exact for every bf16 value with
// 2^-17 <= |w| < 2^16 (smaller ones truncate to the fp16 subnormal grid,
// an error below 2^-24); act must stay below 65504 in magnitude.
template <typename TE>
struct ActOf {
    using type = TE;
};
template <>
struct ActOf<bf16_t> {
    using type = f16_t;
};

__device__ __forceinline__ void mma16_f16(f32x4_t& acc, const uint4& a, const uint4& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), acc,
                                                 0, 0, 0);
}

// eight bf16 -> eight fp16 (two per v_cvt_pkrtz_f16_f32; exact in fp16's range)
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_pkrtz(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)));
}
__device__ __forceinline__ uint4 bf16x8_to_f16x8(const uint4& v) {
    return make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
}

// sigmoid through the hardware reciprocal (v_rcp_f32, 1 ulp) instead of an
// IEEE division sequence; exp overflow gives 1/inf = 0, the right limit
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;

// One bf16 MFMA fragment (8 consecutive K of one column per lane) from a
// [K][N] LDS stage: lane l of each 16-lane group addresses 4 columns of K row
// (l/4)%4 at p, and ds_read_b64_tr_b16 hands lane l the 4 rows of column l%16;
// the second read takes the next 4 rows.
__device__ __forceinline__ uint4 read_tr16_frag(const uint8_t* p, int row_bytes) {
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)p);
    const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(p + 4 * row_bytes));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return make_uint4(a.x, a.y, b.x, b.y);
}

template <typename TE>
__device__ __forceinline__ void store2(TE* p, float a, float b);
template <>
__device__ __forceinline__ void store2<float>(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
template <>
__device__ __forceinline__ void store2<f16_t>(f16_t* p, float a, float b) {
    const f16x2_t v = {(f16_t)a, (f16_t)b};   // round to nearest even (v_cvt_pk_f16_f32)
    *reinterpret_cast<f16x2_t*>(p) = v;
}

template <typename TE>
__device__ __forceinline__ void store4(TE* p, const float* v);
template <>
__device__ __forceinline__ void store4<bf16_t>(bf16_t* p, const float* v) {
    uint2 q;
    q.x = (uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
    q.y = (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
    *reinterpret_cast<uint2*>(p) = q;
}
template <>
__device__ __forceinline__ void store4<float>(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store4<f16_t>(f16_t* p, const float* v) {
    const f16x2_t lo = {(f16_t)v[0], (f16_t)v[1]}, hi = {(f16_t)v[2], (f16_t)v[3]};   // nearest even
    *reinterpret_cast<uint2*>(p) = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

// four consecutive values widened to fp32
template <typename TY>
__device__ __forceinline__ f32x4_t load4f(const TY* p);
template <>
__device__ __forceinline__ f32x4_t load4f<float>(const float* p) {
    return *reinterpret_cast<const f32x4_t*>(p);
}
template <>
__device__ __forceinline__ f32x4_t load4f<f16_t>(const f16_t* p) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    const f16x2_t lo = __builtin_bit_cast(f16x2_t, q.x), hi = __builtin_bit_cast(f16x2_t, q.y);
    return f32x4_t{(float)lo[0], (float)lo[1], (float)hi[0], (float)hi[1]};
}

template <typename TE>
__device__ __forceinline__ void load8f(const TE* p, float* v);
template <>
__device__ __forceinline__ void load8f<float>(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <typename TE>
__device__ __forceinline__ void store8(TE* p, const float* v) {
    store4<TE>(p, v);
    store4<TE>(p + 4, v + 4);
}

// s_waitcnt vmcnt(N) (gfx9 encoding: vmcnt low bits [3:0], high bits [15:14];
// expcnt and lgkmcnt left at their maxima so they are not waited on).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// s_waitcnt lgkmcnt(0) only (LDS reads); vmcnt and expcnt left at their maxima.
__device__ __forceinline__ void wait_lgkmcnt0() {
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
}

// Workgroup barrier without the implicit wait for all outstanding memory
// operations, so loads of later pipeline stages stay in flight across it.
__device__ __forceinline__ void barrier_keep_loads() {
    __asm__ volatile("s_barrier" ::: "memory");
}

// Grouped ordering of an (MT x NT) tile grid: consecutive ids cycle over up to
// GM row tiles, then advance the column tile.
template <int GM>
__device__ __forceinline__ void grouped(int L, int MT, int NT, int& mt, int& nt) {
    const int gsz = GM * NT;
    const int g = L / gsz;
    const int first = g * GM;
    const int gm = min(GM, MT - first);
    const int w = L - g * gsz;
    mt = first + w % gm;
    nt = w / gm;
}

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// One output tile: BN weight rows from n0 x up to BM token rows.
template <typename TE>
struct Tile {
    bool is_shared;
    int K, N, seg, n0, rows_valid, grow0, t0;
    int lda, ldb;        // row strides of A and B (elements)
    int cnt;             // operands read as [K][N]: K rows that exist (K unless padded)
    int segn;            // ... A column segments (see GemmKArgs::a_segn_s)
    long long segstride;
    const TE* A;
    const TE* B;
    void* out;           // kModeWgrad: this problem's gradient [M][N] (fp32 or bf16)
    int gend;            // end of the tile's partner group (tiles gend - n .. gend - 1)
};

template <typename TE, int BM, int GM, int MODE>
__device__ __forceinline__ Tile<TE> decode_tile(const GemmKArgs& a, int L, int BN) {
    Tile<TE> t;
    t.gend = L + 1;
    t.grow0 = 0;
    t.t0 = 0;
    t.out = nullptr;
    t.segn = 1;
    t.segstride = 0;
    if constexpr (wgrad_mode<MODE>()) {
        const int per_p = a.wg_mtiles * a.wg_ntiles;
        const int pr = L / per_p;
        int mt, nt;
        grouped<GM>(L - pr * per_p, a.wg_mtiles, a.wg_ntiles, mt, nt);
        t.is_shared = pr >= a.wg_E;
        t.t0 = mt * BM;
        t.rows_valid = min(BM, a.wg_M - t.t0);
        t.n0 = nt * BN;
        t.N = a.wg_N;
        if (!t.is_shared) {
            const int r0 = a.offsets[pr];
            t.grow0 = r0;
            if constexpr (MODE == kModeGroupWgrad) {
                constexpr int kStage = 64 / (int)sizeof(TE);   // whole stages of 64 bytes of K
                t.K = (a.offsets[pr + 1] - r0 + kStage - 1) / kStage * kStage;
            } else {
                t.K = a.poff[pr + 1] - a.poff[pr];
            }
            t.cnt = a.offsets[pr + 1] - r0;
            t.A = reinterpret_cast<const TE*>(a.A_routed) + (size_t)r0 * a.lda_r;
            t.B = reinterpret_cast<const TE*>(a.B_routed) + (size_t)r0 * a.ldb_r;
            t.lda = a.lda_r;
            t.ldb = a.ldb_r;
            t.out = static_cast<char*>(a.w_out_routed) + (size_t)pr * a.wg_M * a.wg_N * (a.w_out_bf16 ? 2 : 4);
        } else {
            const int sx = pr - a.wg_E;
            t.K = a.K_s;
            t.cnt = a.T;
            t.A = reinterpret_cast<const TE*>(a.A_shared) + sx * a.a_sh_stride;
            t.B = reinterpret_cast<const TE*>(a.B_shared) + sx * a.b_sh_stride;
            t.lda = a.lda_s;
            t.ldb = a.ldb_s;
            t.out = static_cast<char*>(a.w_out_shared) + (size_t)sx * a.wg_M * a.wg_N * (a.w_out_bf16 ? 2 : 4);
        }
        t.seg = max(t.K, 1);
        t.segn = t.N;
        return t;
    }
    t.is_shared = L < a.shared_blocks;
    if (t.is_shared) {
        int mt, nt;
        grouped<GM>(L, a.shared_mtiles, a.ntn_s, mt, nt);
        {
            // partners: the row tiles of this column tile in its group of GM
            const int first = (mt / GM) * GM, gm = min(GM, a.shared_mtiles - first);
            t.gend = L - (mt - first) + min(gm, kGroupMax);
        }
        t.t0 = mt * BM;
        t.rows_valid = min(BM, a.T - t.t0);
        t.n0 = nt * BN;
        t.K = a.K_s;
        t.N = a.N_s;
        t.seg = a.seg_s;
        t.lda = a.seg_s;
        t.ldb = a.K_s;
        t.A = reinterpret_cast<const TE*>(a.A_shared);
        t.B = reinterpret_cast<const TE*>(a.B_shared);
        if constexpr (a_kn<MODE>()) {
            t.lda = a.lda_s;
            t.segn = a.a_segn_s;
            t.segstride = a.a_segstride_s;
        }
    } else {
        // The blocks of expert e are [first tile of e, last + 1) x ntn_r; they are
        // walked column-major (all row tiles of e for weight tile 0, then 1, ...)
        // so the workgroups side by side on an XCD read each weight tile once.
        const int l0 = L - a.shared_blocks;
        const RoutedTile tl0 = a.tiles[l0 / a.ntn_r];
        const int tb = l0 / a.ntn_r - tl0.row_start / BM;   // first tile of the expert
        const int base = a.offsets[tl0.expert];
        const int cnt = a.offsets[tl0.expert + 1] - base;
        const int c = (cnt + BM - 1) / BM;                  // row tiles of the expert
        const int l = l0 - tb * a.ntn_r;
        const int nt = l / c;
        const int row_start = (l - nt * c) * BM;
        {
            // partners: the expert's row tiles for weight tile nt, in runs of
            // at most kGroupMax
            const int j = l - nt * c, run0 = L - j + kGroupMax * (j / kGroupMax);
            t.gend = min(L - j + c, run0 + kGroupMax);
        }
        const RoutedTile tl = {tl0.expert, row_start};
        t.rows_valid = min(BM, cnt - row_start);
        t.grow0 = base + row_start;
        t.n0 = nt * BN;
        t.K = a.K_r;
        t.N = a.N_r;
        t.seg = a.K_r;
        t.lda = a.K_r;
        t.ldb = a.K_r;
        t.A = reinterpret_cast<const TE*>(a.A_routed) + (size_t)tl.expert * a.N_r * a.K_r;
        t.B = reinterpret_cast<const TE*>(a.B_routed);
        if constexpr (a_kn<MODE>()) {
            t.lda = a.lda_r;
            t.segn = a.N_r;
        }
    }
    t.cnt = t.K;
    return t;
}

// Persistent grouped GEMM.  A workgroup owns a contiguous range of grouped
// tiles on its XCD (blocks are dealt to the 8 XCDs round-robin, so workgroups
// that run side by side on one XCD share that range's operands through its L2)
// and walks the range as SCHED says (kSchedStride, kSchedRound, kSchedQueue,
// kSchedGroup).  BN weight rows x BM
// token rows per tile; WN x WM waves (8, two per SIMD; or 4 with two workgroups
// per CU); SA weight and SB token
// LDS pipeline stages of ROWB bytes of K per row, filled by direct global->LDS
// loads.  TE: operand and intermediate type.
//
// Each stage is its own __shared__ array and the K loop is unrolled by
// lcm(SA, SB),
// so every LDS read and every LDS-DMA target is a distinct, statically known
// object: the compiler then needs no wait on in-flight DMA before reading a
// stage that is already complete.  The first stages of the next tile are
// loaded before the epilogue of the current one, so the epilogue's stores and
// SwiGLU arithmetic overlap the next tile's load latency.
template <typename TE, int BN, int BM, int WN, int WM, int SA, int SB, int ROWB, int GM, int SCHED, int MODE>
__global__ __launch_bounds__(WN * WM * 64, 512 / (WN * WM * 64)) void moe_gemm_kernel(const GemmKArgs a) {
    constexpr int NW = WN * WM;                     // waves per workgroup
    static_assert(SCHED != kSchedGroup || !wgrad_mode<MODE>(), "one slot for the next tile: every tile has a K loop");
    static_assert(NW == 8 || NW == 4, "eight waves (two per SIMD), or four (two workgroups per CU)");
    static_assert(SB >= 2 && SA <= 8 && (SA == SB || SA == SB + 1), "weight stages = token stages (+1)");
    // stages unrolled per K-loop iteration: every weight and token buffer index
    // repeats, and the fragment double buffers keep a compile-time parity
    constexpr int U = SA == SB ? SA : SA * SB;
    static_assert(U % 2 == 0, "even unroll");
    static_assert(ROWB == 64 || ROWB == 128 || ROWB == 256, "64, 128 or 256 bytes of K per row and stage");
    constexpr int CH = ROWB / 16;                   // 16-byte chunks per row and stage
    constexpr int KS = ROWB / 64;                   // MFMA k-steps per stage (64 bytes of K each)
    constexpr int EPC = 16 / sizeof(TE);            // elements per 16-byte chunk
    constexpr int BK = ROWB / sizeof(TE);           // K elements per stage
    constexpr int WTN = BN / WN, WTM = BM / WM;     // wave tile
    constexpr int FN = WTN / 16, FM = WTM / 16;     // 16-row blocks per wave (token blocks interleaved by WM)
    static_assert(FN >= 1 && FM >= 1, "wave tile at least 16x16");
    static_assert(BN % 64 == 0 && BM % 16 == 0, "tile shape");
    constexpr int RPL = 1024 / ROWB;                // rows per 1 KB wave load
    constexpr int A_BYTES = BN * ROWB, B_BYTES = BM * ROWB;
    constexpr int A_INS = BN / RPL, B_INS = BM / RPL;   // 1 KB wave loads per stage
    constexpr int A_PW = A_INS / NW, B_PW = (B_INS + NW - 1) / NW;
    static_assert(A_INS % NW == 0, "A loads spread evenly over the waves");
    constexpr int SMALL = 16;
    // operands read as [K][N]: a stage holds BK rows of K, each the tile's BN
    // (A) or BM (B) columns, filled by the same number of 1 KB wave loads
    constexpr bool AKN = a_kn<MODE>(), BKN = b_kn<MODE>();
    constexpr bool GRP = grouped_mode<MODE>(), WG = wgrad_mode<MODE>();
    constexpr int KUP = GRP ? BK - 1 : 0;           // a K tail is a stage of its own
    static_assert(MODE != kModeGroupWgrad || ROWB == 64, "decode_tile pads K to stages of 64 bytes");
    // activation rows (written by gate_up, read by down): fp16 for bf16 layers,
    // so the bf16 down weights are converted to fp16 fragments (f16 MFMA)
    using TA = typename ActOf<TE>::type;
    constexpr bool CVT = (MODE == kModeDown || MODE == kModeDownOut) && std::is_same<TE, bf16_t>::value;
    constexpr int RBA = BN * (int)sizeof(TE), RBB = BM * (int)sizeof(TE);   // bytes per K row
    constexpr int CHA = RBA / 16, CHB = RBB / 16;                           // 16-byte chunks per K row
    constexpr int RPIA = 1024 / RBA, RPIB = 1024 / RBB;                     // K rows per wave load
    static_assert(!AKN || (RBA >= 256 && RBA <= 1024 && BK / RPIA == A_INS), "[K][N] A stage shape");
    static_assert(!BKN || (RBB >= 256 && RBB <= 1024 && BK / RPIB == B_INS), "[K][N] B stage shape");
    // distinct LDS objects per weight stage and per token stage (unused ones
    // shrink to SMALL bytes)
    __shared__ __attribute__((aligned(16))) uint8_t sa0[A_BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t sa1[A_BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t sa2[SA > 2 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sa3[SA > 3 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sa4[SA > 4 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sa5[SA > 5 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sa6[SA > 6 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sa7[SA > 7 ? A_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb0[B_BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t sb1[B_BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t sb2[SB > 2 ? B_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb3[SB > 3 ? B_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb4[SB > 4 ? B_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb5[SB > 5 ? B_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb6[SB > 6 ? B_BYTES : SMALL];
    __shared__ __attribute__((aligned(16))) uint8_t sb7[SB > 7 ? B_BYTES : SMALL];
    // epilogue staging (256 x 256 tiles): per wave 16 rows of kEpRowB bytes
    constexpr int kEpRowB = 144;   // 128 bytes of a row + 16 of padding
    constexpr bool kEpLds = FN == 4 && MODE != kModeDAct;
    __shared__ __attribute__((aligned(16))) uint8_t ep_lds[kEpLds ? NW * 16 * kEpRowB : SMALL];
    auto stage_a = [&](auto S_) -> uint8_t* {
        constexpr int i = decltype(S_)::value % SA;
        if constexpr (i == 0) return sa0;
        else if constexpr (i == 1) return sa1;
        else if constexpr (i == 2) return sa2;
        else if constexpr (i == 3) return sa3;
        else if constexpr (i == 4) return sa4;
        else if constexpr (i == 5) return sa5;
        else if constexpr (i == 6) return sa6;
        else return sa7;
    };
    auto stage_b = [&](auto S_) -> uint8_t* {
        constexpr int i = decltype(S_)::value % SB;
        if constexpr (i == 0) return sb0;
        else if constexpr (i == 1) return sb1;
        else if constexpr (i == 2) return sb2;
        else if constexpr (i == 3) return sb3;
        else if constexpr (i == 4) return sb4;
        else if constexpr (i == 5) return sb5;
        else if constexpr (i == 6) return sb6;
        else return sb7;
    };

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform (scalar) wave index
    const int wn0 = (wv % WN) * WTN, wm = wv / WN;              // token blocks wm, wm+WM, ...
    const int rl = lane & 15;

    // ---- this workgroup's tiles ---------------------------------------------
    // Each XCD takes a contiguous range of blocks holding an eighth of the K
    // stages (shared and routed blocks differ in K when S*I is concatenated).
    // (weight gradients: one tile per workgroup, ranges by count)
    const int nb_routed = WG ? 0 : a.has_routed ? (*a.num_tiles) * a.ntn_r : 0;
    const int nb_real = WG ? (a.wg_E + a.S) * a.wg_mtiles * a.wg_ntiles
                           : a.shared_blocks + nb_routed;
    const long long cost_s = (long long)a.shared_blocks * a.K_s;
    const long long cost_all = cost_s + (long long)nb_routed * a.K_r;
    auto range_start = [&](int x) -> int {
        if (x >= 8) return nb_real;
        if constexpr (WG) {
            // by cost: the layer's padded row counts, or the caller's row offsets
            return wgrad_range_start<MODE == kModeGroupWgrad>(x, a.poff, a.wg_E, a.S, a.wg_mtiles * a.wg_ntiles, a.K_s,
                                                              nb_real);
        }
        const long long c = cost_all * x / 8;
        if (c <= 0) return 0;                                   // also K_s == 0 (no shared blocks)
        if (c <= cost_s) return (int)((c + a.K_s - 1) / a.K_s);
        return min(nb_real, a.shared_blocks + (int)((c - cost_s + a.K_r - 1) / a.K_r));
    };
    const int xcd = blockIdx.x & 7;
    const int nloc = gridDim.x >> 3;
    const int L_beg = range_start(xcd);
    const int L_end = range_start(xcd + 1);
    int L = L_beg + (blockIdx.x >> 3);
    if (L >= L_end) return;
    // kSchedQueue: tiles L_beg + nloc + q for q = 0, 1, ... of the XCD's counter
    // (zero at launch); thread 0 draws the next one while the current tile
    // runs and hands it to the workgroup through LDS (next_slot; tiles that always
    // have a K loop, whose barriers keep the turns apart, take one slot)
    __shared__ int q_next[WG ? kNextSlots : 1];
    int q_val = 0, turn = 0;
    auto draw = [&]() __attribute__((always_inline)) {
        if constexpr (SCHED == kSchedQueue)
            if (tid == 0)
                q_val = __hip_atomic_fetch_add(a.round_counter + xcd, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    // kSchedGroup: before a tile's K loop, thread 0 waits until the counter
    // has handed out every partner tile of its range (the K loop's first
    // barrier holds the other threads).  Partners beyond L + nloc - 1 are not
    // waited for: with at most nloc workgroups, a wait for more could only end
    // at the poll limit, while up to L + nloc - 1 the tiles held by waiting
    // workgroups always cover it.
    auto group_wait = [&](const Tile<TE>& t) __attribute__((always_inline)) {
        if constexpr (SCHED == kSchedGroup) {
            const int need = min(min(t.gend, L_end), L + nloc) - (L_beg + nloc);   // counter value that covers it
            if (tid == 0 && need > 0)
                for (int it = 0; it < kSpinLimit; ++it) {
                    if (__hip_atomic_load(a.round_counter + xcd, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= need)
                        break;
                    __builtin_amdgcn_s_sleep(1);
                }
        }
    };

    // ---- load sources and the stage issue -------------------------------------
    // LDS rows are ROWB bytes; the 16-byte chunk c of row r sits at chunk
    // position c ^ sw(r), which makes the fragment reads below conflict-free.
    // A wave load fills RPL rows: lane -> row lane / CH, chunk position lane % CH.
    auto sw = [](int r) { return CH == 4 ? ((r >> 1) & 3) : CH == 8 ? (r & 7) : (r & 15); };
    // [K][N] stages: the 16-byte chunk c of K row r sits at chunk position
    // c ^ swk(r); the rows that one transposing read touches differ in bits 0,
    // 1 and 3, so their column blocks land on different banks.  (fp32 stages
    // are not swizzled.)
    auto swk = [](int r) { return sizeof(TE) == 2 ? ((r & 3) | ((r >> 1) & 4)) << 1 : 0; };
    const int lr = lane / CH, lp = lane % CH;
    const TE* a_src[A_PW];
    const TE* b_src[B_PW];
    int a_k = 0, b_k = 0, rows_valid_ld = 1, seg_ld = 1, cnt_ld = 0, lda_ld = 0, ldb_ld = 0, m0_ld = 0;
    size_t a_seg = 0, a_seg_step = 0;
    // kModeGroupWgrad with gathered rows of x: the row numbers of the K rows that
    // this wave loads, for the next two stages, in scalar registers (they are the
    // same for the 16 lanes of a K row): the loads of a stage find them there
    constexpr bool GATHER_A = MODE == kModeGroupWgrad;
    static_assert(!GATHER_A || SA == 2, "row numbers two stages ahead");
    int a_idx[GATHER_A ? 2 : 1][GATHER_A ? A_PW : 1][GATHER_A ? RPIA : 1];
    int r0_ld = 0;
    auto row_numbers = [&](auto S_, int k) __attribute__((always_inline)) {
        if constexpr (GATHER_A) {
#pragma unroll
            for (int q = 0; q < A_PW; ++q)
#pragma unroll
                for (int i = 0; i < RPIA; ++i) {
                    const int r = __builtin_amdgcn_readfirstlane(r0_ld + min(k + RPIA * (wv + NW * q) + i, cnt_ld - 1));
                    a_idx[decltype(S_)::value & 1][q][i] = uniform_load(a.row_token + r);
                }
        }
    };
    auto setup = [&](const Tile<TE>& t) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < A_PW; ++q) {
            if constexpr (AKN) {
                const int r = RPIA * (wv + NW * q) + lane / CHA;   // K row within a stage
                const int c = (lane % CHA) ^ swk(r);                // chunk this lane's LDS position holds
                const int n = min(t.n0 + c * EPC, t.N - EPC);      // columns past N re-read the last chunk
                if (GATHER_A && a.row_token != nullptr) a_src[q] = reinterpret_cast<const TE*>(a.A_routed) + n;
                else a_src[q] = t.A + (long long)(n / t.segn) * t.segstride + n % t.segn + (size_t)r * t.lda;
            } else {
                const int r = RPL * (wv + NW * q) + lr;
                a_src[q] = t.A + (size_t)min(t.n0 + r, t.N - 1) * t.lda + (lp ^ sw(r)) * EPC;   // rows past N re-read N-1
            }
        }
#pragma unroll
        for (int q = 0; q < B_PW; ++q) {
            if constexpr (BKN) {
                const int r = RPIB * (wv + NW * q) + lane / CHB;
                const int c = (lane % CHB) ^ swk(r);
                b_src[q] = t.B + min(t.t0 + c * EPC, a.wg_M - EPC) + (size_t)r * t.ldb;
            } else {
                const int r = RPL * (wv + NW * q) + lr;
                const int rr = min(r, t.rows_valid - 1);   // rows past the end re-read the last valid row
                size_t row;
                if constexpr (GRP) {
                    row = (size_t)(t.grow0 + rr);
                    if (MODE == kModeGroup && a.row_token != nullptr)   // gathered; an index out of range reads a row in it
                        row = (size_t)max(0, min(a.row_token[t.grow0 + rr], a.T - 1));
                } else if (t.is_shared || MODE == kModeWgrad) row = (size_t)(t.t0 + rr);
                else if (MODE == kModeGateUp || MODE == kModeGateUpRaw || MODE == kModeDAct)
                    row = (size_t)a.row_token[t.grow0 + rr];   // routed token rows, gathered
                else row = (size_t)(t.grow0 + rr);
                b_src[q] = t.B + row * t.ldb + (lp ^ sw(r)) * EPC;
            }
        }
        a_k = 0;
        b_k = 0;
        a_seg = 0;
        a_seg_step = (size_t)t.N * t.seg;
        seg_ld = t.seg;
        rows_valid_ld = t.rows_valid;
        cnt_ld = t.cnt;
        lda_ld = t.lda;
        ldb_ld = t.ldb;
        m0_ld = t.t0;
        if (GATHER_A && a.row_token != nullptr && t.cnt > 0) {
            r0_ld = t.grow0;
            row_numbers(std::integral_constant<int, 0>{}, 0);
            row_numbers(std::integral_constant<int, 1>{}, BK);
        }
    };
    // Weight stage j is issued SA stage boundaries ahead of its use, token stage
    // j SB ahead (tokens first within a boundary).  A wave's weight loads per
    // stage are a fixed A_PW; its token loads vary (rows past a ragged tile's
    // end are not loaded), so every wait counts weight loads only: waiting
    // until at most n*A_PW loads are outstanding completes everything issued
    // before the n youngest weight stages.
    // K offset of A at the next weight stage to issue: A rows are read in
    // segments of `seg` columns (the shared down projection concatenates S
    // experts along K).
    auto issue_a = [&](auto S_) __attribute__((always_inline)) {
        uint8_t* __restrict__ dst = stage_a(S_);
        if constexpr (GATHER_A) {
            if (a.row_token != nullptr) {
#pragma unroll
                for (int q = 0; q < A_PW; ++q) {
                    const int i = lane / CHA;   // of the wave load's RPIA K rows
                    int row = 0;
#pragma unroll
                    for (int j = 0; j < RPIA; ++j) {
                        // (a select of values: seen as one of an array's elements, the compiler
                        // puts the array into LDS, 24 us of 285 at 64 experts of 384 rows)
                        int v = a_idx[decltype(S_)::value & 1][q][j];
                        __asm__("" : "+s"(v));
                        row = i == j ? v : row;
                    }
                    row = max(0, min(row, a.T - 1));   // an index out of range reads a row in it
                    const TE* src = a_src[q] + (size_t)row * lda_ld;
                    if (a_k + RPIA * (wv + NW * q) + i >= cnt_ld) src = reinterpret_cast<const TE*>(&zero_chunk);
                    __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + (wv + NW * q) * 1024), 16, 0,
                                                     0);
                }
                a_k += BK;
                row_numbers(S_, a_k + BK);
                return;
            }
        }
        if constexpr (GRP) {
            // the stage that holds the K tail: rows (AKN) or chunks past it load zeros
            if (a_k + BK > cnt_ld) {
                const size_t off = AKN ? (size_t)a_k * lda_ld : (size_t)a_k;
#pragma unroll
                for (int q = 0; q < A_PW; ++q) {
                    const int r = AKN ? RPIA * (wv + NW * q) + lane / CHA : (lp ^ sw(RPL * (wv + NW * q) + lr)) * EPC;
                    const TE* src = a_k + r < cnt_ld ? a_src[q] + off : reinterpret_cast<const TE*>(&zero_chunk);
                    __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + (wv + NW * q) * 1024), 16, 0,
                                                     0);
                }
                a_k += BK;
                return;
            }
        }
        if constexpr (AKN) {
            const size_t off = (size_t)a_k * lda_ld;
            if (MODE == kModeWgrad && a_k + BK > cnt_ld) {
                // the stage that holds the tile's padding rows: rows past the
                // count re-read its last row (B reads zeros there)
#pragma unroll
                for (int q = 0; q < A_PW; ++q) {
                    const int r = RPIA * (wv + NW * q) + lane / CHA;
                    const long long rel = a_k + r < cnt_ld ? a_k : cnt_ld - 1 - r;
                    __builtin_amdgcn_global_load_lds((glb_void_t*)(a_src[q] + rel * lda_ld),
                                                     (lds_void_t*)(dst + (wv + NW * q) * 1024), 16, 0, 0);
                }
            } else {
#pragma unroll
                for (int q = 0; q < A_PW; ++q)
                    __builtin_amdgcn_global_load_lds((glb_void_t*)(a_src[q] + off),
                                                     (lds_void_t*)(dst + (wv + NW * q) * 1024), 16, 0, 0);
            }
            a_k += BK;
            return;
        }
        const size_t aoff = a_seg + a_k;
#pragma unroll
        for (int q = 0; q < A_PW; ++q)
            __builtin_amdgcn_global_load_lds((glb_void_t*)(a_src[q] + aoff), (lds_void_t*)(dst + (wv + NW * q) * 1024),
                                             16, 0, BM <= 16 ? kPolicyNT : 0);
        a_k += BK;
        if (a_k == seg_ld) {
            a_k = 0;
            a_seg += a_seg_step;
        }
    };
    auto issue_b = [&](auto S_) __attribute__((always_inline)) {
        uint8_t* __restrict__ dst = stage_b(S_);
        if constexpr (GRP) {
            if (b_k + BK > cnt_ld) {
                const size_t off = BKN ? (size_t)b_k * ldb_ld : (size_t)b_k;
#pragma unroll
                for (int q = 0; q < B_PW; ++q) {
                    const int qi = wv + NW * q;
                    const int r = BKN ? RPIB * qi + lane / CHB : (lp ^ sw(RPL * qi + lr)) * EPC;
                    const TE* src = b_k + r < cnt_ld ? b_src[q] + off : reinterpret_cast<const TE*>(&zero_chunk);
                    if (qi < B_INS && (BKN || RPL * qi < rows_valid_ld))
                        __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + qi * 1024), 16, 0, 0);
                }
                b_k += BK;
                return;
            }
        }
        if constexpr (BKN) {
            const size_t off = (size_t)b_k * ldb_ld;
            if (!GRP && b_k + BK > cnt_ld) {
                // rows past the tile's count read the zero row (same columns)
#pragma unroll
                for (int q = 0; q < B_PW; ++q) {
                    const int qi = wv + NW * q;
                    const int r = RPIB * qi + lane / CHB;
                    const int m = min(m0_ld + ((lane % CHB) ^ swk(r)) * EPC, a.wg_M - EPC);
                    const TE* src = b_k + r < cnt_ld ? b_src[q] + off : reinterpret_cast<const TE*>(a.zero) + m;
                    if (qi < B_INS)
                        __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + qi * 1024), 16, 0, 0);
                }
            } else {
#pragma unroll
                for (int q = 0; q < B_PW; ++q) {
                    const int qi = wv + NW * q;
                    if (qi < B_INS)
                        __builtin_amdgcn_global_load_lds((glb_void_t*)(b_src[q] + off), (lds_void_t*)(dst + qi * 1024),
                                                         16, 0, 0);
                }
            }
            b_k += BK;
            return;
        }
#pragma unroll
        for (int q = 0; q < B_PW; ++q) {
            const int qi = wv + NW * q;
            if (qi < B_INS && RPL * qi < rows_valid_ld)
                __builtin_amdgcn_global_load_lds((glb_void_t*)(b_src[q] + b_k), (lds_void_t*)(dst + qi * 1024), 16, 0,
                                                 0);
        }
        b_k += BK;
    };
    auto issue_first = [&](int nk) __attribute__((always_inline)) {
        static_for<0, SA>([&](auto S_) {
            constexpr int j = decltype(S_)::value;
            if (j < SB && j < nk) issue_b(S_);
            if (j < nk) issue_a(S_);
        });
    };

    // per-row epilogue data, loaded when a tile starts (used after its K loop)
    float ep_g0[FM], ep_g1[FM];   // gate_up: gamma of the row (routed) / of the wave's first and last shared expert
    int ep_row[FM];               // down: output row (slot for routed tiles, token for shared tiles);
                                  // down_out: 1 if the row's token has routed rows
    int ep_s0 = 0;                // gate_up shared: expert of the wave's first weight row
    auto prefetch_epilogue = [&](const Tile<TE>& t) __attribute__((always_inline)) {
        if constexpr (MODE == kModeGateUpRaw || WG || GRP) return;
        // columns of shared expert s: [s*2I, (s+1)*2I) in gate_up, [s*I, (s+1)*I) in dact
        const int width = MODE == kModeDAct ? a.I : 2 * a.I;
        const int s0 = min((t.n0 + wn0) / width, max(a.S - 1, 0));
        const int s1 = min((t.n0 + wn0 + WTN - 1) / width, max(a.S - 1, 0));
        ep_s0 = s0;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = min(16 * (WM * j + wm) + rl, t.rows_valid - 1);
            if (MODE == kModeGateUp || MODE == kModeDAct) {
                if (t.is_shared) {
                    ep_g0[j] = a.shared_g[(size_t)(t.t0 + m) * a.S + s0];
                    ep_g1[j] = a.shared_g[(size_t)(t.t0 + m) * a.S + s1];
                } else {
                    ep_g0[j] = a.row_gamma[t.grow0 + m];
                    ep_g1[j] = 0.f;
                }
            } else if (MODE == kModeDownOut) {
                ep_row[j] = a.k > 0 && a.pos[(size_t)(t.t0 + m) * a.k] >= 0;   // the token has routed rows
            } else {
                ep_row[j] = t.is_shared ? t.t0 + m : a.row_slot[t.grow0 + m];
            }
        }
    };

    f32x4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // fragment rows: A rows wn0 + 16i + rl, B rows 16*(WM*j + wm) + rl; 16-row
    // blocks start at multiples of 8 rows, so sw(row) = sw(rl) throughout.
    // In k-step s a lane feeds logical chunk 4s + lane/16 to the MFMA.
    int a_rd[KS], b_rd[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int cpos = ((4 * s + (lane >> 4)) ^ sw(rl)) << 4;
        a_rd[s] = (wn0 + rl) * ROWB + cpos;
        b_rd[s] = (16 * wm + rl) * ROWB + cpos;
    }
    constexpr int A_STEP = 16 * ROWB;               // bytes between a wave's weight-row blocks
    constexpr int B_STEP = 16 * WM * ROWB;          // bytes between a wave's token blocks

    // [K][N] stages, bf16: lane l of 16-lane group g = l/16 addresses K row
    // 8g + (l/4)%4 (+ 32 per k-step, + 4 for the second read) at columns
    // 4(l%4).. of its 16-column block; swk of all those rows is the same.
    // The chunk of fragment i (A) is ((wn0 + 16i)/8 + (l%4)/2) ^ sz, whose
    // bits 1-2 (2i, i < 4) meet sz there: its byte offset is a lane constant
    // XOR 32i.  For B, chunk (16(WM j + wm))/8 + (l%4)/2 = 4j + 2wm + ..:
    // a lane constant XOR 64j.
    int a_kn0 = 0, b_kn0 = 0;
    if constexpr (sizeof(TE) == 2 && (AKN || BKN)) {
        static_assert(!AKN || (FN <= 4 && WTN % 64 == 0), "A fragment offsets: 2i in chunk bits 1-2");
        static_assert(!BKN || (WM == 2 && FM <= 8), "B fragment offsets: 4j in chunk bits 2-4");
        const int g = lane >> 4, j4 = (lane >> 2) & 3, q4 = lane & 3;
        const int sz = (j4 | ((g & 1) << 2)) << 1;
        a_kn0 = (8 * g + j4) * RBA + ((((wn0 >> 3) + (q4 >> 1)) ^ sz) << 4) + (q4 & 1) * 8;
        b_kn0 = (8 * g + j4) * RBB + (((2 * wm + (q4 >> 1)) ^ sz) << 4) + (q4 & 1) * 8;
    }
    // [K][N] stages, fp32: element k = 16 ks + 4(l/16) + c of column cb + l%16
    // for c < 4 (the K order of the K-major fragments)
    auto read_kn32 = [&](const uint8_t* __restrict__ st, int ks, int cb, int rb) __attribute__((always_inline)) {
        float v[4];
        const uint8_t* p = st + (4 * (lane >> 4)) * rb + (cb + (lane & 15)) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const float*>(p + (16 * ks + c) * rb);
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    };
    // fragment i (A: weight rows wn0 + 16i..) / j (B: token block WM*j + wm) of k-step ks
    auto read_a = [&](const uint8_t* __restrict__ st, int ks, int i) __attribute__((always_inline)) -> uint4 {
        if constexpr (!AKN) return *reinterpret_cast<const uint4*>(st + a_rd[ks] + i * A_STEP);
        else if constexpr (sizeof(TE) == 2) return read_tr16_frag(st + (a_kn0 ^ (32 * i)) + ks * 32 * RBA, RBA);
        else return read_kn32(st, ks, wn0 + 16 * i, RBA);
    };
    auto read_b = [&](const uint8_t* __restrict__ st, int ks, int j) __attribute__((always_inline)) -> uint4 {
        if constexpr (!BKN) return *reinterpret_cast<const uint4*>(st + b_rd[ks] + j * B_STEP);
        else if constexpr (sizeof(TE) == 2) return read_tr16_frag(st + (b_kn0 ^ (64 * j)) + ks * 32 * RBB, RBB);
        else return read_kn32(st, ks, 16 * (WM * j + wm), RBB);
    };

    // Tile-round rendezvous of an XCD (kSchedRound): every workgroup counts each tile
    // it finishes on its XCD's counter and waits, for at most kSpinLimit polls,
    // until every workgroup of its round has finished, so that the workgroups
    // that share tiles through L2 start the next round together.  (Meeting
    // also every 4-32 K stages inside a tile was measured slower.)
    int sync_round = 0;
    auto rendezvous = [&](long long target, bool wait) __attribute__((always_inline)) {
        if (tid == 0) {
            int32_t* ctr = a.round_counter + xcd;
            __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (wait)
                for (int it = 0; it < kSpinLimit; ++it) {
                    if (__hip_atomic_fetch_add(ctr, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= target) break;
                    __builtin_amdgcn_s_sleep(2);
                }
        }
    };

    // kModeDownOut: out[t][n..n+3] = v + y[t*k + 0][n..] + ... + y[t*k + k-1][n..]
    // (fp32, in that order, which is also the order of the combine kernel),
    // rounded once.  `routed`: the token was dispatched (a padded token has no
    // routed rows), read with the other per-row epilogue data.
    auto combine_store = [&](int t, int n, f32x4_t v, int routed) __attribute__((always_inline)) {
        if constexpr (MODE == kModeDownOut) {
            if (routed) {
                // the first 8 rows are loaded unconditionally (a smaller k
                // re-reads its last row, not added), so all 8 are in flight
                // before the first add; then the rest one by one
                const TA* yr = static_cast<const TA*>(a.y_rows) + (size_t)t * a.k * a.H + n;
                const int k8 = min(a.k, 8);
                f32x4_t u[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] = load4f<TA>(yr + (size_t)min(q, k8 - 1) * a.H);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < k8) v += u[q];
                for (int i = 8; i < a.k; ++i) v += load4f<TA>(yr + (size_t)i * a.H);
            }
            const float w[4] = {v[0], v[1], v[2], v[3]};
            if (a.out_final_bf16) store4<bf16_t>(static_cast<bf16_t*>(a.out_final) + (size_t)t * a.H + n, w);
            else store4<float>(static_cast<float*>(a.out_final) + (size_t)t * a.H + n, w);
        }
    };

    // NJ: 16-row token blocks computed (blocks past the last valid row skipped).
    //
    // Work of a stage = KS k-steps x 2 halves of the token blocks (half-steps).
    // The LDS fragments of each half-step are read during the previous one:
    //   wait for the reads issued last half-step -> issue the next half-step's
    //   reads -> MFMAs of this half-step.
    // Before the stage's last half-step (all its reads done): wait for this
    // wave's loads of stage kt+1, barrier, load weight stage kt+SA and token
    // stage kt+SB into the buffers just freed, then read the first half-step
    // of stage kt+1.  The first SA weight and SB token stages of a tile are
    // issued before its K loop.
    auto kloop = [&](auto NJ_, int nk) __attribute__((always_inline)) {
        constexpr int NJ = decltype(NJ_)::value;
        constexpr int H1 = (NJ + 1) / 2, H2 = NJ - H1;
        constexpr int HS = H2 > 0 ? 2 * KS : KS;    // half-steps per stage
        // fragments double-buffered by the parity of the global k-step (A) and
        // half-step (B) index; with U even both parities are compile-time
        uint4 fa[2][FN], fb[2][H1];
        if (SA - 1 < nk) wait_vmcnt<(SA - 1) * A_PW>();
        else wait_vmcnt<0>();
        barrier_keep_loads();
        {
            const uint8_t* __restrict__ s0a = stage_a(std::integral_constant<int, 0>{});
            const uint8_t* __restrict__ s0b = stage_b(std::integral_constant<int, 0>{});
#pragma unroll
            for (int i = 0; i < FN; ++i) fa[0][i] = read_a(s0a, 0, i);
#pragma unroll
            for (int j = 0; j < H1; ++j) fb[0][j] = read_b(s0b, 0, j);
        }
        for (int kt0 = 0; kt0 < nk; kt0 += U) {
            static_for<0, U>([&](auto S_) __attribute__((always_inline)) {
                constexpr int sidx = decltype(S_)::value;
                const int kt = kt0 + sidx;
                if (kt < nk) {
                    const uint8_t* __restrict__ sba = stage_a(S_);
                    const uint8_t* __restrict__ sbb = stage_b(S_);
                    static_for<0, HS>([&](auto H_) __attribute__((always_inline)) {
                        constexpr int h = decltype(H_)::value;
                        constexpr int ks = H2 > 0 ? h >> 1 : h;          // k-step of this half-step
                        constexpr int half = H2 > 0 ? (h & 1) : 0;       // token half
                        constexpr int bcur = (sidx * HS + h) & 1;        // B buffer of this half-step
                        constexpr int acur = (sidx * KS + ks) & 1;       // A buffer of this k-step
                        wait_lgkmcnt0();
                        if constexpr (h + 1 < HS) {
                            // read the next half-step of this stage
                            constexpr int hn = h + 1;
                            constexpr int ksn = H2 > 0 ? hn >> 1 : hn;
                            constexpr int halfn = H2 > 0 ? (hn & 1) : 0;
                            if constexpr (halfn == 0) {
#pragma unroll
                                for (int i = 0; i < FN; ++i) fa[acur ^ 1][i] = read_a(sba, ksn, i);
                            }
                            constexpr int j0 = halfn ? H1 : 0, jn = halfn ? H2 : H1;
#pragma unroll
                            for (int j = 0; j < jn; ++j) fb[bcur ^ 1][j] = read_b(sbb, ksn, j0 + j);
                        } else {
                            if (kt + 1 < nk) {
                                // all reads of this stage are done: wait for stage kt+1
                                // (SA-2 younger weight stages may stay in flight),
                                // refill this stage's buffers, start the next stage
                                if (kt + SA - 1 < nk) wait_vmcnt<(SA - 2) * A_PW>();
                                else wait_vmcnt<0>();
                                barrier_keep_loads();
                                if (kt + SB < nk) issue_b(S_);
                                if (kt + SA < nk) issue_a(S_);
                                constexpr int snext = (sidx + 1) % U;
                                const uint8_t* __restrict__ sna = stage_a(std::integral_constant<int, snext>{});
                                const uint8_t* __restrict__ snb = stage_b(std::integral_constant<int, snext>{});
                                constexpr int an = (snext * KS) & 1;     // A buffer of the next stage's k-step 0
#pragma unroll
                                for (int i = 0; i < FN; ++i) fa[an][i] = read_a(sna, 0, i);
#pragma unroll
                                for (int j = 0; j < H1; ++j) fb[bcur ^ 1][j] = read_b(snb, 0, j);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        constexpr int jbase = half ? H1 : 0, jn = half ? H2 : H1;
                        if constexpr (CVT) {
                            // bf16 weight fragments -> fp16, once per k-step (at
                            // its first half-step, after the wait above)
                            if constexpr (half == 0) {
#pragma unroll
                                for (int i = 0; i < FN; ++i) {
                                    fa[acur][i] = bf16x8_to_f16x8(fa[acur][i]);
#pragma unroll
                                    for (int j = 0; j < jn; ++j)
                                        mma16_f16(acc[i][jbase + j], fa[acur][i], fb[bcur][j]);
                                }
                                // the 12 VALU ops converting fragment i + 1 issue
                                // between the MFMAs of fragment i, which do not
                                // wait for them
                                constexpr int cv = 12 / jn;
                                __builtin_amdgcn_sched_group_barrier(0x002, 12, 0);
#pragma unroll
                                for (int g = 0; g < (FN - 1) * jn; ++g) {
                                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                                    __builtin_amdgcn_sched_group_barrier(0x002, cv, 0);
                                }
                                __builtin_amdgcn_sched_group_barrier(0x008, jn, 0);
                            } else {
#pragma unroll
                                for (int i = 0; i < FN; ++i)
#pragma unroll
                                    for (int j = 0; j < jn; ++j)
                                        mma16_f16(acc[i][jbase + j], fa[acur][i], fb[bcur][j]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < jn; ++j)
#pragma unroll
                                for (int i = 0; i < FN; ++i) mma16<TE>(acc[i][jbase + j], fa[acur][i], fb[bcur][j]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    });
                }
            });
        }
    };

    Tile<TE> cur = decode_tile<TE, BM, GM, MODE>(a, L, BN);
    setup(cur);
    issue_first((cur.K + KUP) / BK);
    prefetch_epilogue(cur);
    draw();

    while (true) {
        const int nk = (cur.K + KUP) / BK;
        if constexpr (SCHED == kSchedRound) sync_round = (L - L_beg) / nloc;
        // token blocks / weight-row blocks of this wave that hold valid rows
        const int nvb_all = (cur.rows_valid + 15) >> 4;
        const int nvb = min(FM, max(0, (nvb_all - wm + WM - 1) / WM));
        const int nvi = min(FN, max(0, (cur.N - cur.n0 - wn0 + 15) >> 4));
        if (nk > 0) {
            if constexpr (FM == 1) {
                kloop(std::integral_constant<int, 1>{}, nk);
            } else {
                // a wave without valid token rows still runs one block, to take part
                // in the loads and barriers; nothing of it is stored
                const int nvb_run = max(nvb, 1);
                static_for<1, FM + 1>([&](auto P_) {
                    if (nvb_run == decltype(P_)::value) kloop(std::integral_constant<int, decltype(P_)::value>{}, nk);
                });
            }
        }

        // all waves are done reading the stages: start loading the next tile
        if constexpr (SCHED == kSchedGroup) {
            // the next tile is taken now that this workgroup is free
            if (tid == 0)
                q_next[0] = __hip_atomic_fetch_add(a.round_counter + xcd, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            L = L_beg + nloc + q_next[0];
        } else if constexpr (SCHED == kSchedQueue) {
            // (no loads are in flight here: the last stage waited for all)
            const int slot = WG ? next_slot(turn++) : 0;
            if (tid == 0) q_next[slot] = q_val;
            __syncthreads();
            L = L_beg + nloc + q_next[slot];
        } else {
            L += nloc;
        }
        const bool has_next = L < L_end;
        if constexpr (SCHED == kSchedRound) {
            // end of the tile: round r + 1 starts once round r is done by all
            // (with a next tile, rounds 0..r are full)
            rendezvous((long long)nloc * (sync_round + 1), has_next);
        }
        if constexpr (SCHED != kSchedQueue && SCHED != kSchedGroup) {
            wait_lgkmcnt0();
            barrier_keep_loads();
        }
        Tile<TE> nxt = cur;
        if (has_next) {
            nxt = decode_tile<TE, BM, GM, MODE>(a, L, BN);
            setup(nxt);
            issue_first((nxt.K + KUP) / BK);
            draw();
        }

        // ---- epilogue of the current tile ----------------------------------
        // acc[i][j][r]: output column n = n0 + wn0 + 16i + 4*(lane/16) + r,
        // token row m = 16*(WM*j + wm) + lane%16
        if constexpr (MODE == kModeDAct) {
            // acc = dact (d of the activation the down projection saw); with
            // h = [g, u] interleaved, p = silu(g) u, a = gamma p:
            //   dgamma += dact . p,  dp = gamma dact,
            //   dg = dp u silu'(g),  du = dp silu(g)
            const int nrow = cur.N;   // I (routed) or S*I (shared) columns
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int m = 16 * (WM * j + wm) + rl;
                const bool rv = j < nvb && m < cur.rows_valid && nvi > 0;
                const size_t row = cur.is_shared ? (size_t)(cur.t0 + m) : (size_t)(cur.grow0 + m);
                const float* hrow = reinterpret_cast<const float*>(cur.is_shared ? a.h_shared : a.h_routed) + row * 2 * nrow;
                TE* dhrow = reinterpret_cast<TE*>(cur.is_shared ? a.out_shared : a.out_routed) + row * 2 * nrow;
                TE* arow = reinterpret_cast<TE*>(cur.is_shared ? a.a_shared : a.a_routed) + row * nrow;
                float part = 0.f;
                if (rv) {
#pragma unroll
                    for (int i = 0; i < FN; ++i) {
                        const int n = cur.n0 + wn0 + 16 * i + 4 * (lane >> 4);
                        if (i < nvi) {
                            const float g_ = (cur.is_shared && n / a.I != ep_s0) ? ep_g1[j] : ep_g0[j];
                            float hv[8];
                            load8f<float>(hrow + 2 * n, hv);
                            float dh[8], av[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float gg = hv[2 * r], uu = hv[2 * r + 1];
                                const float sg = sigmoid(gg);
                                const float si = gg * sg;
                                const float pp = si * uu;
                                const float da = acc[i][j][r];
                                const float dp = g_ * da;
                                part += da * pp;
                                av[r] = g_ * pp;
                                dh[2 * r] = dp * uu * sg * (1.0f + gg * (1.0f - sg));
                                dh[2 * r + 1] = dp * si;
                            }
                            store8<TE>(dhrow + 2 * n, dh);
                            store4<TE>(arow + n, av);
                        }
                    }
                }
                // row sum over the wave's 64 columns (lanes l, l^16, l^32, l^48 share the row)
                part += __shfl_xor(part, 16);
                part += __shfl_xor(part, 32);
                if (rv && (lane >> 4) == 0) {
                    float* dgp = cur.is_shared ? a.dgp_shared : a.dgp_routed;
                    dgp[row * (nrow / 64) + (cur.n0 + wn0) / 64] = part;
                }
            }
        }
        if constexpr (kEpLds) {
            // The wave's results go through its LDS block, 16 rows at a time,
            // so that a global store writes whole row segments (4 or 8 rows of
            // 128 bytes, or 16 rows of 64) instead of 16 rows of 4-16 bytes:
            // phase A writes the lane's values in the MFMA layout, phase B
            // reads 16-byte chunks of rows and stores them.  LDS operations of
            // one wave complete in order, so no barrier is needed.
            // (lane-derived offsets are recomputed for every tile: hoisted out
            // of the tile loop, the compiler would keep dozens of them live
            // across the K loop and spill them)
            int ln = lane;
            __asm__ volatile("" : "+v"(ln));
            const int g4 = ln >> 4, rw = ln & 15;
            uint8_t* __restrict__ ep = ep_lds + wv * 16 * kEpRowB;
            // fp32 columns wn0 .. wn0 + 63 of the 16 rows from mb, in two
            // halves of 32 columns; rowp(r): output row of row mb + r at
            // column n0 + wn0 (nullptr: none)
            auto flush_f32 = [&](int j, int mb, auto rowp) __attribute__((always_inline)) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int i = 2 * hh; i < 2 * hh + 2; ++i)
                        if (i < nvi)
                            *reinterpret_cast<f32x4_t*>(ep + rw * kEpRowB + ((i - 2 * hh) * 16 + 4 * g4) * 4) = acc[i][j];
#pragma unroll
                    for (int sgi = 0; sgi < 2; ++sgi) {
                        const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                        const f32x4_t d = *reinterpret_cast<const f32x4_t*>(ep + r * kEpRowB + q * 16);
                        float* o = rowp(r);
                        if (o != nullptr && mb + r < cur.rows_valid && 2 * hh + (q >> 2) < nvi &&
                            (!GRP || cur.n0 + wn0 + 32 * hh + 4 * q < cur.N))   // N a multiple of 8, not of 16
                            store16<GRP>(o + 32 * hh + 4 * q, d);
                    }
                }
            };
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                if (j >= nvb) continue;
                const int mb = 16 * (WM * j + wm);
                if constexpr (MODE == kModeGateUp) {
                    // act = gamma silu(g) u of the interleaved pairs: the wave's
                    // 64 projection columns give 32 act columns per row
                    const float g0 = ep_g0[j], g1 = ep_g1[j];
#pragma unroll
                    for (int i = 0; i < FN; ++i) {
                        if (i < nvi) {
                            const f32x4_t v = acc[i][j];
                            const int n = cur.n0 + wn0 + 16 * i + 4 * g4;
                            const float g = cur.is_shared && n / (2 * a.I) != ep_s0 ? g1 : g0;
                            store2<TA>(reinterpret_cast<TA*>(ep + rw * kEpRowB + (8 * i + 2 * g4) * sizeof(TA)),
                                       silu(v[0]) * v[1] * g, silu(v[2]) * v[3] * g);
                        }
                    }
                    constexpr int CPR = 32 * (int)sizeof(TA) / 16;   // 16-byte chunks per row
                    const int ld = cur.is_shared ? a.S * a.I : a.I;
                    TA* obase = reinterpret_cast<TA*>(cur.is_shared ? a.out_shared : a.out_routed) +
                                (size_t)(cur.is_shared ? cur.t0 : cur.grow0) * ld + ((cur.n0 + wn0) >> 1);
#pragma unroll
                    for (int sgi = 0; sgi < 16 * CPR / 64; ++sgi) {
                        const int c = ln + 64 * sgi, r = c / CPR, q = c % CPR;
                        const uint4 d = *reinterpret_cast<const uint4*>(ep + r * kEpRowB + q * 16);
                        const int col = q * (16 / (int)sizeof(TA));
                        if (mb + r < cur.rows_valid && col / 8 < nvi)
                            *reinterpret_cast<uint4*>(obase + (size_t)(mb + r) * ld + col) = d;
                    }
                    // optional fp32 copy of the projection itself (kept for the backward)
                    float* hs = cur.is_shared ? a.h_save_shared : a.h_save_routed;
                    if (hs != nullptr) {
                        float* hb = hs + (size_t)(cur.is_shared ? cur.t0 : cur.grow0) * cur.N + cur.n0 + wn0;
                        flush_f32(j, mb, [&](int r) -> float* { return hb + (size_t)(mb + r) * cur.N; });
                    }
                } else if constexpr (MODE == kModeGateUpRaw) {   // h kept in fp32 (not an MFMA operand)
                    float* hb = reinterpret_cast<float*>(cur.is_shared ? a.out_shared : a.out_routed) +
                                (size_t)(cur.is_shared ? cur.t0 : cur.grow0) * cur.N + cur.n0 + wn0;
                    flush_f32(j, mb, [&](int r) -> float* { return hb + (size_t)(mb + r) * cur.N; });
                } else if constexpr (GRP) {
                    // rows of the product (weight gradients: rows of dW_e), fp32
                    // or rounded once to bf16 (64 columns fill a 128-byte LDS row)
                    const bool to_bf16 = WG ? a.w_out_bf16 : a.out_final_bf16;
                    char* ob = static_cast<char*>(WG ? cur.out : a.out_routed);
                    const size_t row0 = (size_t)(WG ? cur.t0 : cur.grow0);
                    if (to_bf16) {
#pragma unroll
                        for (int i = 0; i < FN; ++i)
                            if (i < nvi)
                                *reinterpret_cast<uint2*>(ep + rw * kEpRowB + (16 * i + 4 * g4) * 2) =
                                    pack_bf16x4(acc[i][j]);
                        bf16_t* hb = reinterpret_cast<bf16_t*>(ob) + row0 * cur.N + cur.n0 + wn0;
#pragma unroll
                        for (int sgi = 0; sgi < 2; ++sgi) {
                            const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                            const f32x4_t d = *reinterpret_cast<const f32x4_t*>(ep + r * kEpRowB + q * 16);
                            if (mb + r < cur.rows_valid && cur.n0 + wn0 + 8 * q < cur.N)
                                store16<GRP>(hb + (size_t)(mb + r) * cur.N + 8 * q, d);
                        }
                    } else {
                        float* hb = reinterpret_cast<float*>(ob) + row0 * cur.N + cur.n0 + wn0;
                        flush_f32(j, mb, [&](int r) -> float* { return hb + (size_t)(mb + r) * cur.N; });
                    }
                } else if constexpr (MODE == kModeWgrad) {
                    if (a.w_out_bf16) {
                        // bf16 gradients: the fp32 sums rounded once; 64 columns
                        // of 2 bytes fill one 128-byte LDS row
#pragma unroll
                        for (int i = 0; i < FN; ++i)
                            if (i < nvi) {
                                const float v4[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                                store4<bf16_t>(reinterpret_cast<bf16_t*>(ep + rw * kEpRowB + (16 * i + 4 * g4) * 2), v4);
                            }
                        bf16_t* hb = static_cast<bf16_t*>(cur.out) + (size_t)cur.t0 * cur.N + cur.n0 + wn0;
#pragma unroll
                        for (int sgi = 0; sgi < 2; ++sgi) {
                            const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                            const uint4 d = *reinterpret_cast<const uint4*>(ep + r * kEpRowB + q * 16);
                            if (mb + r < cur.rows_valid && (q >> 1) < nvi)
                                *reinterpret_cast<uint4*>(hb + (size_t)(mb + r) * cur.N + 8 * q) = d;
                        }
                    } else {
                        float* hb = static_cast<float*>(cur.out) + (size_t)cur.t0 * cur.N + cur.n0 + wn0;
                        flush_f32(j, mb, [&](int r) -> float* { return hb + (size_t)(mb + r) * cur.N; });
                    }
                } else if constexpr (MODE == kModeDownOut) {
                    // the combine: each 16-byte chunk of a row (4 columns of one
                    // token) gets the token's routed rows added in slot order
                    // (8 lanes read 128 contiguous bytes of each y row), then is
                    // rounded once and stored
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                        for (int i = 2 * hh; i < 2 * hh + 2; ++i)
                            if (i < nvi)
                                *reinterpret_cast<f32x4_t*>(ep + rw * kEpRowB + ((i - 2 * hh) * 16 + 4 * g4) * 4) =
                                    acc[i][j];
                        f32x4_t d[2];
#pragma unroll
                        for (int sgi = 0; sgi < 2; ++sgi) {
                            const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                            d[sgi] = *reinterpret_cast<const f32x4_t*>(ep + r * kEpRowB + q * 16);
                        }
                        const int er = ep_row[j];
#pragma unroll
                        for (int sgi = 0; sgi < 2; ++sgi) {
                            const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                            const int routed = __shfl(er, r);
                            if (mb + r < cur.rows_valid && 2 * hh + (q >> 2) < nvi)
                                combine_store(cur.t0 + mb + r, cur.n0 + wn0 + 32 * hh + 4 * q, d[sgi], routed);
                        }
                    }
                } else if ((MODE == kModeDown || MODE == kModeDx) && sizeof(TA) == 2 && !cur.is_shared) {
                    // routed rows (down: y, dx: the routed dx rows) rounded to
                    // fp16: the wave's 64 columns of 16 rows pass through LDS as
                    // 128-byte row segments
#pragma unroll
                    for (int i = 0; i < FN; ++i)
                        if (i < nvi) {
                            const float v4[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                            store4<TA>(reinterpret_cast<TA*>(ep + rw * kEpRowB + (16 * i + 4 * g4) * 2), v4);
                        }
                    TA* o = reinterpret_cast<TA*>(a.out_routed) + cur.n0 + wn0;
                    const int er = ep_row[j];
#pragma unroll
                    for (int sgi = 0; sgi < 2; ++sgi) {
                        const int c = ln + 64 * sgi, r = c >> 3, q = c & 7;
                        const uint4 d = *reinterpret_cast<const uint4*>(ep + r * kEpRowB + q * 16);
                        const int row = __shfl(er, r);
                        if (mb + r < cur.rows_valid && (q >> 1) < nvi)
                            *reinterpret_cast<uint4*>(o + (size_t)row * a.H + 8 * q) = d;
                    }
                } else {
                    // fp32 rows (the routed rows of fp32 layers; the shared sums
                    // of a down launch and of dx)
                    float* o = reinterpret_cast<float*>(cur.is_shared ? a.out_shared : a.out_routed) + cur.n0 + wn0;
                    const int er = ep_row[j];
                    flush_f32(j, mb, [&](int r) -> float* { return o + (size_t)__shfl(er, r) * a.H; });
                }
            }
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            if constexpr (MODE == kModeDAct || kEpLds) break;
            const int m = 16 * (WM * j + wm) + rl;
            if (j < nvb && m < cur.rows_valid) {
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const int n = cur.n0 + wn0 + 16 * i + 4 * (lane >> 4);
                    if (i < nvi) {
                        const f32x4_t v = acc[i][j];
                        if constexpr (GRP) {
                            const size_t at = (size_t)((WG ? cur.t0 : cur.grow0) + m) * cur.N + n;
                            void* ob = WG ? cur.out : a.out_routed;
                            if (n < cur.N) {
                                if (WG ? a.w_out_bf16 : a.out_final_bf16)
                                    *reinterpret_cast<uint2*>(static_cast<bf16_t*>(ob) + at) = pack_bf16x4(v);
                                else
                                    *reinterpret_cast<f32x4_t*>(static_cast<float*>(ob) + at) = v;
                            }
                        } else if (MODE == kModeGateUpRaw) {   // h kept in fp32 (not an MFMA operand)
                            float* o = reinterpret_cast<float*>(cur.is_shared ? a.out_shared : a.out_routed) +
                                       (size_t)(cur.is_shared ? cur.t0 + m : cur.grow0 + m) * cur.N + n;
                            float w[4] = {v[0], v[1], v[2], v[3]};
                            store4<float>(o, w);
                        } else if (MODE == kModeWgrad) {
                            float w[4] = {v[0], v[1], v[2], v[3]};
                            store4<float>(static_cast<float*>(cur.out) + (size_t)(cur.t0 + m) * cur.N + n, w);
                        } else if (MODE == kModeGateUp) {
                            // optional fp32 copy of the projection itself (kept for the backward)
                            float* hs = cur.is_shared ? a.h_save_shared : a.h_save_routed;
                            if (cur.is_shared) {
                                const int t = cur.t0 + m;
                                const float g = (n / (2 * a.I) == ep_s0) ? ep_g0[j] : ep_g1[j];
                                TA* o = reinterpret_cast<TA*>(a.out_shared) + (size_t)t * a.S * a.I + (n >> 1);
                                store2<TA>(o, silu(v[0]) * v[1] * g, silu(v[2]) * v[3] * g);
                                if (hs != nullptr) hs += (size_t)t * cur.N + n;
                            } else {
                                const int row = cur.grow0 + m;
                                const float g = ep_g0[j];
                                TA* o = reinterpret_cast<TA*>(a.out_routed) + (size_t)row * a.I + (n >> 1);
                                store2<TA>(o, silu(v[0]) * v[1] * g, silu(v[2]) * v[3] * g);
                                if (hs != nullptr) hs += (size_t)row * cur.N + n;
                            }
                            if (hs != nullptr) {
                                float w[4] = {v[0], v[1], v[2], v[3]};
                                store4<float>(hs, w);
                            }
                        } else if (MODE == kModeDownOut) {
                            combine_store(cur.t0 + m, n, v, ep_row[j]);
                        } else if ((MODE == kModeDown || MODE == kModeDx) && !cur.is_shared) {
                            // routed rows (TA: fp16 for bf16 layers)
                            float w[4] = {v[0], v[1], v[2], v[3]};
                            store4<TA>(reinterpret_cast<TA*>(a.out_routed) + (size_t)ep_row[j] * a.H + n, w);
                        } else {
                            // fp32 rows (the shared sums of a down launch and of dx)
                            float w[4] = {v[0], v[1], v[2], v[3]};
                            float* o = reinterpret_cast<float*>(cur.is_shared ? a.out_shared : a.out_routed);
                            store4<float>(o + (size_t)ep_row[j] * a.H + n, w);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (!has_next) break;
        cur = nxt;
        prefetch_epilogue(cur);
        group_wait(cur);
    }
}

}  // namespace

}  // namespace inkling
