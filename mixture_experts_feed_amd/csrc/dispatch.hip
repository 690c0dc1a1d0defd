// Tokens sorted by expert, and back.
//
// Order (expert_order): the slots t*k + i of a token's chosen experts, sorted by
// expert and by slot within one: a stable counting sort.  A workgroup of 16 waves
// takes a chunk of slots, each wave a run of it.  Counts of every wave and expert,
// summed over the waves, the chunks and the experts before, give each (wave,
// expert) its first row; then a wave walks its run 64 slots at a time, and a slot's
// row is that plus its rank among the equal experts of the 64 lanes, from one
// ballot for each bit of the expert's number.  Integers throughout, so the order
// depends on nothing but the input.  Up to kOrderOne slots one workgroup does it
// all in one launch; more take a launch of counts before (65536 slots of 128 experts in
// 64 chunks: 4.8 + 6.7 us; 256 slots, one launch: 3.6).  Latency bounds it.
//
// Rows and tokens: positions [T][k] hold the row of each slot (-1: none), so both
// directions go by token, and nothing is summed by atomics:
//   spread (dispatch forward, combine backward)  rows[p(t,i)] = w(t,i) x[t]
//   gather (combine forward, dispatch backward)  out[t] = add[t] + sum_i w(t,i) rows[p(t,i)]
//   and where wanted the weights' gradient       dw(t,i) = <x[t], rows[p(t,i)]>.
// HBM bounds all of them: a token's row is read (or written) once, beside its k
// rows.  Arithmetic in fp32 in the order of the slots, rounded once.  A wave takes 64
// vectors of one token's row, so that up to eight rows' loads are on their way together.
// 8192 tokens of 6144 bf16, top-8: spread of 7168 tokens 135 us (6.0 TB/s), gather of
// 65536 rows 159 (5.7), weights' gradient with the rows written 325 (5.3), with the tokens'
// 165 (6.1).
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec.h"

namespace inkling {

namespace {

constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / kWave;
constexpr int kOrderExperts = 512;
constexpr int kOrderOne = 8192;          // slots of one workgroup that does it all
constexpr int kOrderChunks = 256;        // at most

// Expert of a slot: E where the slot has no row (padded token, expert out of range,
// slot past the end).
__device__ __forceinline__ int slot_expert(const int32_t* __restrict__ topk, const uint8_t* __restrict__ pad,
                                           long long slot, long long end, int E, int k) {
    if (slot >= end) return E;
    const int e = topk[slot];
    if (e < 0 || e >= E) return E;
    return pad != nullptr && pad[(uint32_t)slot / (uint32_t)k] != 0 ? E : e;
}

// hist[c][e] = slots of chunk c that go to expert e
__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(const int32_t* __restrict__ topk,
                                                                    const uint8_t* __restrict__ pad, long long n,
                                                                    int chunk, int E, int k,
                                                                    int32_t* __restrict__ hist) {
    __shared__ int32_t cnt[kOrderExperts];
    for (int e = threadIdx.x; e < E; e += kOrderThreads) cnt[e] = 0;
    __syncthreads();
    const long long beg = (long long)blockIdx.x * chunk, end = min(n, beg + chunk);
    for (long long s = beg + threadIdx.x; s < end; s += kOrderThreads) {
        const int e = slot_expert(topk, pad, s, end, E, k);
        if (e < E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kOrderThreads) hist[(size_t)blockIdx.x * E + e] = cnt[e];
}

// One workgroup a chunk (hist NULL: one chunk).  slots may be NULL.
__global__ __launch_bounds__(kOrderThreads) void order_place_kernel(
    const int32_t* __restrict__ topk, const uint8_t* __restrict__ pad, long long n, int chunk, int E, int bits, int k,
    const int32_t* __restrict__ hist, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ slots, int32_t* __restrict__ positions) {
    __shared__ int32_t first[kOrderWaves][kOrderExperts];   // counts, then the next row of (wave, expert)
    __shared__ int32_t total[kOrderExperts], before[kOrderExperts], off[kOrderExperts + 1];
    const int t = threadIdx.x, lane = lane_id(), wv = t >> 6;
    for (int e = t; e < E; e += kOrderThreads) {
        total[e] = 0;
        before[e] = 0;
    }
    for (int i = t; i < kOrderWaves * kOrderExperts; i += kOrderThreads) (&first[0][0])[i] = 0;
    __syncthreads();
    const int run = chunk / kOrderWaves;   // a multiple of 64
    const long long beg = (long long)blockIdx.x * chunk, end = min(n, beg + chunk);
    const long long wbeg = beg + (long long)wv * run, wend = min(end, wbeg + run);
    for (long long s = wbeg + lane; s < wend; s += kWave) {
        const int e = slot_expert(topk, pad, s, wend, E, k);
        if (e < E) atomicAdd(&first[wv][e], 1);
    }
    if (hist != nullptr) {
        // threads e + stride * part sum every parts-th chunk
        const int stride = 1 << bits;   // E rounded up to a power of two, at least 64
        const int e = t & (stride - 1), part = t >> bits, parts = kOrderThreads >> bits;
        int sum = 0, prior = 0;
        if (e < E) {
            for (int c = part; c < (int)gridDim.x; c += parts) {
                const int h = hist[(size_t)c * E + e];
                sum += h;
                prior += c < (int)blockIdx.x ? h : 0;
            }
            atomicAdd(&total[e], sum);
            atomicAdd(&before[e], prior);
        }
    }
    __syncthreads();
    if (hist == nullptr) {
        for (int e = t; e < E; e += kOrderThreads) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kOrderWaves; ++w) sum += first[w][e];
            total[e] = sum;
        }
        __syncthreads();
    }
    if (wv == 0) {
        int carry = 0;
        for (int base = 0; base < E; base += kWave) {
            const int e = base + lane;
            const int c = e < E ? total[e] : 0;
            int incl = c;
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            if (e < E) off[e] = carry + incl - c;
            carry += __shfl(incl, kWave - 1);
        }
        if (lane == 0) off[E] = carry;
    }
    __syncthreads();
    for (int e = t; e < E; e += kOrderThreads) {
        int row = off[e] + before[e];
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) {
            const int c = first[w][e];
            first[w][e] = row;
            row += c;
        }
    }
    if (blockIdx.x == 0)
        for (int e = t; e <= E; e += kOrderThreads) {
            offsets[e] = off[e];
            if (counts != nullptr && e < E) counts[e] = total[e];
        }
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1ull;
    for (long long s0 = wbeg; s0 < wend; s0 += kWave) {
        const long long s = s0 + lane;
        const int e = slot_expert(topk, pad, s, wend, E, k);
        uint64_t same = __ballot(e < E);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? m : ~m;
        }
        // the lowest lane of each expert takes the rows of all of its lanes
        int row = 0;
        const bool mine = e < E;
        const int leader = mine ? __ffsll((unsigned long long)same) - 1 : lane;
        if (mine && leader == lane) row = atomicAdd(&first[wv][e], __popcll(same));
        row = __shfl(row, leader) + __popcll(same & below);
        if (s < wend) {
            positions[s] = mine ? row : -1;
            if (mine && slots != nullptr) slots[row] = (int32_t)s;
        }
    }
    // entries behind the last row
    if (slots != nullptr) {
        const int used = off[E];
        for (long long s = max(beg, (long long)used) + t; s < end; s += kOrderThreads) slots[s] = -1;
    }
}

// ---- rows and tokens -----------------------------------------------------------------

// V values at the alignment of one (rows of any width; the hardware takes such
// accesses whole), past the caches where PAST
template <typename TE, int V>
struct LooseVec {
    typedef Raw<TE, V> type __attribute__((aligned(sizeof(TE))));
};
template <typename TE, int V, bool PAST>
__device__ __forceinline__ Raw<TE, V> load_row(const TE* p) {
    typedef typename LooseVec<TE, V>::type L;
    if constexpr (PAST) return __builtin_nontemporal_load(reinterpret_cast<const L*>(p));
    else return *reinterpret_cast<const L*>(p);
}
template <typename TE, int V, bool PAST>
__device__ __forceinline__ void store_row(TE* p, const float* v) {
    typedef typename LooseVec<TE, V>::type L;
    const Raw<TE, V> r = narrow<TE, V>(v);
    if constexpr (PAST) __builtin_nontemporal_store((L)r, reinterpret_cast<L*>(p));
    else *reinterpret_cast<L*>(p) = (L)r;
}

constexpr int kSlots = 8;   // rows of a token in flight at once

struct MoveArgs {
    const int32_t* positions;   // [T][k]
    const float* weights;       // [T][k] or NULL for 1
    const void* token_in;       // [T][H]: spread: x; gather: what is added first (or NULL); dw: x
    const void* rows_in;        // [rows][H]
    void* token_out;            // gather: [T][H]
    void* rows_out;             // spread: [rows][H] or NULL
    float* dweights;            // [T][k] or NULL
    long long T, rows;
    int k, H, nv;               // nv: vectors of a row
};

// UNI: an address that is the same for the whole wave, written by an earlier kernel
// only: a scalar load
template <bool UNI, typename V>
__device__ __forceinline__ V load_slot(const V* p) {
    if constexpr (UNI) return *(const __attribute__((address_space(4))) V*)p;
    else return *p;
}

// The rows of slots c0 .. c0 + 7 of token t (-1: none)
template <bool UNI>
__device__ __forceinline__ void slot_rows(const MoveArgs& a, long long t, int c0, int (&p)[kSlots], float (&w)[kSlots]) {
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        p[j] = -1;
        w[j] = 1.0f;
        if (c0 + j < a.k) {
            const long long s = t * a.k + c0 + j;
            p[j] = load_slot<UNI>(a.positions + s);
            if (p[j] >= a.rows) p[j] = -1;
            if (a.weights != nullptr) w[j] = load_slot<UNI>(a.weights + s);
        }
    }
}

// G lanes take G vectors of one token's row: a wave's worth of a wide row, or a
// whole narrow one.  Column of vector v: v V, the last one moved back to end with
// the row (two lanes then write the same values to the columns they share).
template <int G>
struct Unit {
    long long t;
    int v;
    bool live;
    __device__ __forceinline__ Unit(const MoveArgs& a) {
        const uint32_t segs = (uint32_t)(a.nv + G - 1) / G;
        uint32_t in_block = threadIdx.x / G;
        if constexpr (G == kWave) in_block = __builtin_amdgcn_readfirstlane(in_block);   // the same for the wave
        const uint32_t unit = blockIdx.x * (256 / G) + in_block;   // < 2^26 (move_fits)
        t = unit / segs;
        v = (int)(unit % segs) * G + threadIdx.x % G;
        live = t < a.T && v < a.nv;
    }
};

template <typename TT, typename TR, int V, int G>
__global__ __launch_bounds__(256) void spread_kernel(const MoveArgs a) {
    const Unit<G> u(a);
    if (!u.live) return;
    const int col = min(u.v * V, a.H - V);
    float x[V];
    widen<TT, V>(load_row<TT, V, false>(static_cast<const TT*>(a.token_in) + (size_t)u.t * a.H + col), x);
    TR* out = static_cast<TR*>(a.rows_out) + col;
    for (int c0 = 0; c0 < a.k; c0 += kSlots) {
        int p[kSlots];
        float w[kSlots];
        slot_rows<G >= kWave>(a, u.t, c0, p, w);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            if (p[j] < 0) continue;
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = w[j] * x[i];
            store_row<TR, V, true>(out + (size_t)p[j] * a.H, y);
        }
    }
}

template <typename TT, typename TR, int V, int G>
__global__ __launch_bounds__(256) void gather_kernel(const MoveArgs a) {
    const Unit<G> u(a);
    if (!u.live) return;
    const int col = min(u.v * V, a.H - V);
    const size_t at = (size_t)u.t * a.H + col;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (a.token_in != nullptr) widen<TT, V>(load_row<TT, V, false>(static_cast<const TT*>(a.token_in) + at), acc);
    const TR* rows = static_cast<const TR*>(a.rows_in) + col;
    for (int c0 = 0; c0 < a.k; c0 += kSlots) {
        int p[kSlots];
        float w[kSlots];
        slot_rows<G >= kWave>(a, u.t, c0, p, w);
        Raw<TR, V> r[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (p[j] >= 0) r[j] = load_row<TR, V, true>(rows + (size_t)p[j] * a.H);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            if (p[j] < 0) continue;
            float y[V];
            widen<TR, V>(r[j], y);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[j], y[i], acc[i]);
        }
    }
    store_row<TT, V, false>(static_cast<TT*>(a.token_out) + at, acc);
}

// With the weights' gradient: a whole token by G lanes, or (G == 256) by a
// workgroup.  SPREAD: also rows_out[p] = w x (where rows_out is given); otherwise
// also token_out = sum w rows.  Sums over the lanes in a fixed order.
// kMaxSlots: 8 or 32 (with 32 running sums a lane the fp32 gradients of 1001 x 1237,
// top-2, took 27 us for both operators' kernels instead of 10).  With 32 and fp32 rows a
// lane takes 236 to 243 registers and 96 to 128 of the matrix units', so a SIMD holds one wave:
// 8192 tokens of 6144 fp32, top-16, take 3420 us with the rows written (1.9 TB/s) and 2450
// with the tokens'; in bf16 645 (5.2) and 320 (5.7).
template <typename TT, typename TR, int V, int G, int kMaxSlots, bool SPREAD>
__global__ __launch_bounds__(256) void dweights_kernel(const MoveArgs a) {
    __shared__ float part[4][kMaxSlots];
    const int sub = threadIdx.x % G;
    long long t = (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
    if constexpr (G == kWave) t = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if constexpr (G == 256) t = blockIdx.x;
    if (t >= a.T) return;   // whole groups (G == 256: the workgroup)
    const TT* x = static_cast<const TT*>(a.token_in) + (size_t)t * a.H;
    const TR* rows = static_cast<const TR*>(a.rows_in);
    float dw[kMaxSlots];
#pragma unroll
    for (int j = 0; j < kMaxSlots; ++j) dw[j] = 0.0f;
    for (int v = sub; v < a.nv; v += G) {
        const int col = min(v * V, a.H - V), skip = v * V - col;   // columns that the lane before has
        float xv[V], acc[V];
        widen<TT, V>(load_row<TT, V, false>(x + col), xv);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kMaxSlots / kSlots; ++c) {
            if (c * kSlots >= a.k) break;
            int p[kSlots];
            float w[kSlots];
            slot_rows<G >= kWave>(a, t, c * kSlots, p, w);
            Raw<TR, V> r[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (p[j] >= 0) r[j] = load_row<TR, V, true>(rows + (size_t)p[j] * a.H + col);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (p[j] < 0) continue;
                float y[V];
                widen<TR, V>(r[j], y);
                float d = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (i >= skip) d = __builtin_fmaf(xv[i], y[i], d);
                    acc[i] = __builtin_fmaf(w[j], y[i], acc[i]);
                }
                dw[c * kSlots + j] += d;
                if constexpr (SPREAD) {
                    if (a.rows_out != nullptr) {
#pragma unroll
                        for (int i = 0; i < V; ++i) y[i] = w[j] * xv[i];
                        store_row<TR, V, true>(static_cast<TR*>(a.rows_out) + (size_t)p[j] * a.H + col, y);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // the next slots' rows in these ones' registers
        }
        if constexpr (!SPREAD) store_row<TT, V, false>(static_cast<TT*>(a.token_out) + (size_t)t * a.H + col, acc);
    }
    constexpr int L = G == 256 ? kWave : G;
#pragma unroll
    for (int j = 0; j < kMaxSlots; ++j) {
        if (j >= a.k) break;
        dw[j] = lanes_sum<L>(dw[j]);
        if constexpr (G == 256) {
            if (lane_id() == 0) part[threadIdx.x >> 6][j] = dw[j];
        } else if (sub == 0) {
            a.dweights[t * a.k + j] = dw[j];
        }
    }
    if constexpr (G == 256) {
        __syncthreads();
        const int j = threadIdx.x;
        if (j < a.k) a.dweights[t * a.k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
    }
}

template <typename TT, typename TR>
constexpr int move_cols() { return sizeof(TT) == 2 && sizeof(TR) == 2 ? 8 : 4; }

template <typename TT, typename TR, int V, int G, int SLOTS>
void launch_dweights(const MoveArgs& a, bool spread, hipStream_t stream) {
    const long long per = 256 / G;
    const dim3 grid((unsigned)((a.T + per - 1) / per)), block(256);
    if (spread) hipLaunchKernelGGL((dweights_kernel<TT, TR, V, G, SLOTS, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dweights_kernel<TT, TR, V, G, SLOTS, false>), grid, block, 0, stream, a);
}

template <typename TT, typename TR, int V, int G>
hipError_t launch_move_as(MoveArgs a, bool spread, hipStream_t stream) {
    a.nv = (a.H + V - 1) / V;
    if (a.dweights != nullptr) {
        // more than a vector a lane of a wave: a workgroup a token
        constexpr int WIDE = G == kWave ? 256 : G;
        const bool wide = a.nv > G;
        if (a.k <= 8) {
            if (wide) launch_dweights<TT, TR, V, WIDE, 8>(a, spread, stream);
            else launch_dweights<TT, TR, V, G, 8>(a, spread, stream);
        } else {
            if (wide) launch_dweights<TT, TR, V, WIDE, 32>(a, spread, stream);
            else launch_dweights<TT, TR, V, G, 32>(a, spread, stream);
        }
        return hipGetLastError();
    }
    const long long units = a.T * ((a.nv + G - 1) / G), per = 256 / G;
    const dim3 grid((unsigned)((units + per - 1) / per)), block(256);
    if (spread) hipLaunchKernelGGL((spread_kernel<TT, TR, V, G>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((gather_kernel<TT, TR, V, G>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <typename TT, typename TR>
hipError_t launch_move(const MoveArgs& a, bool spread, hipStream_t stream) {
    constexpr int V = move_cols<TT, TR>();
    if (a.H < V) return launch_move_as<TT, TR, 1, 16>(a, spread, stream);
    if (a.H <= 16 * V) return launch_move_as<TT, TR, V, 16>(a, spread, stream);
    return launch_move_as<TT, TR, V, 64>(a, spread, stream);
}

int order_chunk(long long n) {
    if (n <= kOrderOne) return (int)((n + 1023) / 1024 * 1024);
    const long long c = (n + kOrderChunks - 1) / kOrderChunks;
    return (int)((c + 1023) / 1024 * 1024);
}

}  // namespace

long long order_hist_ints(long long slots, int E) {
    if (slots <= kOrderOne) return 0;
    const long long chunk = order_chunk(slots);
    return (slots + chunk - 1) / chunk * E;
}

hipError_t launch_expert_order(const int32_t* topk, const uint8_t* pad, long long slots, int E, int k, int32_t* hist,
                               int32_t* counts, int32_t* offsets, int32_t* sorted, int32_t* positions,
                               hipStream_t stream) {
    const int chunk = order_chunk(slots);
    const int chunks = slots <= kOrderOne ? 1 : (int)((slots + chunk - 1) / chunk);
    int bits = 6;
    while ((1 << bits) < E) ++bits;
    if (chunks > 1) {
        hipLaunchKernelGGL(order_count_kernel, dim3(chunks), dim3(kOrderThreads), 0, stream, topk, pad, slots, chunk, E,
                           k, hist);
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    hipLaunchKernelGGL(order_place_kernel, dim3(chunks), dim3(kOrderThreads), 0, stream, topk, pad, slots, chunk, E, bits,
                       k, chunks > 1 ? hist : nullptr, counts, offsets, sorted, positions);
    return hipGetLastError();
}

// A launch has fewer than 2^32 threads: at most 2^24 - 1 workgroups, of four waves
// of at least 256 columns each, or (weights' gradients of wider rows) one a token.
bool move_fits(long long T, int H) { return T * (H / 256 + 1) < (1LL << 25); }

hipError_t launch_rows(const RowMoveParams& p, bool spread, hipStream_t stream) {
    MoveArgs a = {};
    a.positions = p.positions;
    a.weights = p.weights;
    a.token_in = p.token_in;
    a.rows_in = p.rows_in;
    a.token_out = p.token_out;
    a.rows_out = p.rows_out;
    a.dweights = p.dweights;
    a.T = p.T;
    a.rows = p.rows;
    a.k = p.k;
    a.H = p.H;
    if (p.token_dtype == 1) {
        if (p.rows_dtype == 1) return launch_move<bf16_t, bf16_t>(a, spread, stream);
        return launch_move<bf16_t, float>(a, spread, stream);
    }
    if (p.rows_dtype == 1) return launch_move<float, bf16_t>(a, spread, stream);
    return launch_move<float, float>(a, spread, stream);
}

}  // namespace inkling
