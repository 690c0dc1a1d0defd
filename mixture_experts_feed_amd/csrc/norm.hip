// Layer norm and RMS norm over the rows of x [R][H], forward and backward.
//
//   y = (x - m) r w + b,  r = 1 / sqrt(mean((x - m)^2) + eps),  m = mean(x)
//   (RMS norm: m = 0 and no b).  With xh = (x - m) r and c = dy w:
//   dx = r (c - mean(c) - xh mean(c xh))   (RMS norm: without mean(c))
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// HBM bounds both passes: x is read once and kept in registers for the second
// moment about the mean, the result is written once.  A large mean costs no
// digits: fp32 rows also take the sum of x - m in that second pass over the
// registers, which gives back what the first sum was rounded by (the sum of bf16
// rows is exact wherever that would matter).
//
// A row is held in 16-byte vectors, one a lane where the width allows: rows of
// up to 64 vectors by 8 to 64 neighbouring lanes of a wave (no LDS), wider ones
// by a workgroup with as many waves as they need (up to 1024 lanes, then up to
// 512 with 4 or 8 vectors each).  One vector a lane keeps the registers few, so that several
// workgroups a CU hide each other's sums.  Rows that are not whole vectors are
// read with the same accesses at their own alignment, the last partial vector
// value by value.  Lanes walk rows with their columns of w and b in registers
// and load the next row before the sums of the current one.
// The backward pass keeps its columns' sums of dw and db in registers over all
// its rows and writes one partial row for each workgroup (narrow rows: each
// wave); a second kernel adds the partial rows in order, so results repeat bit
// for bit.
// Measured, 8192 x 6144 bf16: forward 32 us (201 MB: the last cache holds part of
// it), backward 59 us and 5 for the partial rows (302 MB, 5.1 TB/s); 32 rows
// forward 4.1 us; fp32 1001 x 1237 backward 8 us and 4.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec.h"

namespace inkling {

namespace {

constexpr int kMaxWaves = 16;
// one vector a lane up to 1024 lanes; several a lane need the registers of 512
template <int NV, int G>
constexpr int max_threads() { return G != 0 ? 256 : NV == 1 ? 1024 : 512; }
// Waves a SIMD that the registers have to leave room for (second launch bound): 6
// with one vector a lane (80 registers), so that two workgroups of 12 waves share a
// CU (the backward, 8192 x 6144 bf16: 75 us with 76 registers, 90 with 86); 4 for
// the backward of narrow rows, which 80 registers make spill (98304 x 512 bf16: 77
// us against 84); 2 with several vectors a lane.

// Sums over the lanes that hold a row: G lanes of a wave (G < 64 or one wave),
// or G == 0: the workgroup.  `buf` alternates from call to call, so that one
// barrier a sum is enough; the waves' sums are added in order.
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*buf)[N]) {
    constexpr int L = G == 0 ? kWave : G;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<L>(v[i]);
    if constexpr (G == 0) {
        if (lane_id() == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[threadIdx.x >> 6][i] = v[i];
        __syncthreads();
        const int waves = blockDim.x >> 6;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = buf[0][i];
        for (int w = 1; w < waves; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += buf[w][i];
    }
}

template <typename TE>
struct LooseOf;
template <>
struct LooseOf<bf16_t> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <>
struct LooseOf<float> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };

// A lane's vectors of a row: vector j is columns (j * lanes + t) V ..
// TAIL: H is not a multiple of V (nor are rows 16-byte aligned); `last` values
// of the last vector exist.
template <typename TE, int NV, bool TAIL, bool NT>
struct Row {
    static constexpr int V = 16 / sizeof(TE);
    typedef Raw<TE, V> Vec;
    typedef typename LooseOf<TE>::type Loose;   // the same 16 bytes at the alignment of a value
    static __device__ __forceinline__ void load(Vec* r, const TE* p, int t, int lanes, int full, int last) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = j * lanes + t;
            if constexpr (TAIL) {
                if (k < full) {
                    r[j] = (Vec) * reinterpret_cast<const Loose*>(p + (size_t)k * V);
                } else {
                    TE e[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        e[i] = TE(0);
                        if (k == full && i < last) e[i] = p[(size_t)k * V + i];
                    }
                    __builtin_memcpy(&r[j], e, sizeof(Vec));
                }
            } else {
                // lanes past the row hold zeros
                r[j] = Vec{};
                if (k < full) r[j] = *reinterpret_cast<const Vec*>(p + (size_t)k * V);
            }
        }
    }
    static __device__ __forceinline__ void store(TE* p, int j, int t, int lanes, int full, int last, const float* v) {
        const int k = j * lanes + t;
        if (k < full) {
            if constexpr (TAIL) {
                *reinterpret_cast<Loose*>(p + (size_t)k * V) = (Loose)narrow<TE, V>(v);
            } else {
                put<NT>(p + (size_t)k * V, narrow<TE, V>(v));
            }
        } else if (TAIL && k == full) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < last) put<false>(p + (size_t)k * V + i, narrow<TE, 1>(v + i));
        }
    }
    // fp32 columns of w, b or of a partial row
    static __device__ __forceinline__ void column(float* c, const float* p, int j, int t, int lanes, int H) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (j * lanes + t) * V + i;
            c[i] = p != nullptr && (TAIL ? col < H : (j * lanes + t) * V < H) ? p[col] : 0.0f;
        }
    }
    static __device__ __forceinline__ void columns(float (*c)[V], const float* p, int t, int lanes, int H) {
#pragma unroll
        for (int j = 0; j < NV; ++j) column(c[j], p, j, t, lanes, H);
    }
};

// The row a lane starts with, how far the next one is, and its place in it.
template <int G>
struct Place {
    int t, lanes, row, step;
    __device__ __forceinline__ Place() {
        if constexpr (G == 0) {
            t = threadIdx.x;
            lanes = blockDim.x;
            row = blockIdx.x;
            step = gridDim.x;
        } else {
            t = threadIdx.x % G;
            lanes = G;
            row = blockIdx.x * (256 / G) + threadIdx.x / G;
            step = gridDim.x * (256 / G);
        }
    }
};

template <typename TE, int NV, int G, bool TAIL, bool RMS, bool NT>
__global__ __launch_bounds__((max_threads<NV, G>()), (NV == 1 ? 6 : 2)) void norm_forward_kernel(
    const TE* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, int rows, int H, float eps,
    TE* __restrict__ out, float* __restrict__ stats) {
    using R = Row<TE, NV, TAIL, NT>;
    constexpr int V = R::V;
    // fp32 rows: the sum of x - m too.  (bf16 rows whose mean is large against their
    // spread have values of one or two exponents, so at most 2^14 multiples of one
    // step below 2^9 of them: their sum is exact.  8192 x 6144 would take 46 us
    // instead of 40; fp32, 2048 x 12288, takes 47 instead of 46.)
    constexpr bool kShift = !RMS && sizeof(TE) == 4;
    constexpr int kSums = kShift ? 2 : 1;
    __shared__ float first[2][kMaxWaves][1], second[2][kMaxWaves][kSums];
    const Place<G> at;
    const int full = H / V, last = H - full * V, t = at.t, lanes = at.lanes;
    const float n = (float)H;
    typename R::Vec cur[NV], nxt[NV];
    int row = at.row;
    if (row < rows) R::load(cur, x + (size_t)row * H, t, lanes, full, last);
    float wr[NV][V], br[NV][V];
    R::columns(wr, w, t, lanes, H);
    if constexpr (!RMS) R::columns(br, b, t, lanes, H);
    // (G != 0: the lanes of a row leave together, and no barrier follows)
    for (int turn = 0; row < rows; row += at.step, turn ^= 1) {
        if (rows - row > at.step) R::load(nxt, x + ((size_t)row + at.step) * H, t, lanes, full, last);
        float v[NV][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            widen<TE, V>(cur[j], v[j]);
            if constexpr (!RMS)
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] += v[j][i];
        }
        float m = 0.0f;
        if constexpr (!RMS) {
            row_sums<G, 1>(s, first[turn]);
            m = s[0] / n;   // a quotient, not contracted into x - m
        }
        // d = x - m.  The mean of d is what the rounding of a long sum left in m: with
        // it, mean and variance are as exact as those of values around 0
        float q[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) q[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int left = H - (j * lanes + t) * V;   // columns of this vector that exist
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool real = RMS || (TAIL ? i < left : left > 0);   // RMS: absent columns are 0
                if constexpr (kShift) {
                    v[j][i] = real ? v[j][i] - m : 0.0f;   // d from here on
                    q[1] += v[j][i];
                    q[0] += v[j][i] * v[j][i];
                } else {
                    const float d = v[j][i] - m;
                    q[0] += real ? d * d : 0.0f;
                }
            }
        }
        row_sums<G, kSums>(q, second[turn]);
        float shift = 0.0f, var = q[0] / n;
        if constexpr (kShift) {
            shift = q[1] / n;
            var -= shift * shift;
            if (var < 0.0f) var = 0.0f;   // (a NaN stays)
        }
        const float r = 1.0f / sqrtf(var + eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = (v[j][i] - (kShift ? shift : m)) * r * wr[j][i];
                if constexpr (!RMS) y[i] += br[j][i];
            }
            R::store(out + (size_t)row * H, j, t, lanes, full, last, y);
        }
        if (stats != nullptr && t == 0)
            *reinterpret_cast<float2*>(stats + 2 * (size_t)row) = make_float2(kShift ? m + shift : m, r);
#pragma unroll
        for (int j = 0; j < NV; ++j) cur[j] = nxt[j];
    }
}

// part [partial rows][parts][H]: dw, and db where parts is 2
template <typename TE, int NV, int G, bool TAIL, bool RMS, bool NT>
__global__ __launch_bounds__((max_threads<NV, G>()), (NV != 1 ? 2 : G != 0 ? 4 : 6)) void norm_backward_kernel(
    const TE* __restrict__ dout, const TE* __restrict__ x, const float* __restrict__ stats,
    const float* __restrict__ w, int rows, int H, int parts, TE* __restrict__ dx, float* __restrict__ part) {
    using R = Row<TE, NV, TAIL, NT>;
    constexpr int V = R::V;
    __shared__ float sums[2][kMaxWaves][2];
    const Place<G> at;
    const int full = H / V, last = H - full * V, t = at.t, lanes = at.lanes;
    const float n = (float)H;
    typename R::Vec cx[NV], cd[NV], nx[NV], nd[NV];
    float2 st = make_float2(0.0f, 0.0f), nst = st;
    int row = at.row;
    if (row < rows) {
        st = *reinterpret_cast<const float2*>(stats + 2 * (size_t)row);
        R::load(cx, x + (size_t)row * H, t, lanes, full, last);
        R::load(cd, dout + (size_t)row * H, t, lanes, full, last);
    }
    float wr[NV][V], dw[NV][V], db[NV][V];
    constexpr bool kHoldW = NV < 8 || RMS;
    if constexpr (kHoldW) R::columns(wr, w, t, lanes, H);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.0f;
    for (int turn = 0; row < rows; row += at.step, turn ^= 1) {
        if (rows - row > at.step) {
            const size_t next = (size_t)row + at.step;
            nst = *reinterpret_cast<const float2*>(stats + 2 * next);
            R::load(nx, x + next * H, t, lanes, full, last);
            R::load(nd, dout + next * H, t, lanes, full, last);
        }
        const float m = RMS ? 0.0f : st.x, r = st.y;
        // columns that do not exist have dout 0 and w 0, and xh 0: they add nothing
        // ((0 - m) r may overflow where no xh of the row does, and 0 inf is NaN)
        float xh[NV][V], c[NV][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float d[V];
            widen<TE, V>(cx[j], xh[j]);
            widen<TE, V>(cd[j], d);
            if constexpr (!kHoldW) {
                // read for each row (from the L2): held over the rows, more registers
                // spill (2048 x 12288 fp32: 97 us against 130; the RMS norm, which
                // holds them, 63 against 71)
                const float* wp = w;
                __asm__ volatile("" : "+s"(wp), "+v"(s[0]));
                R::column(wr[j], wp, j, t, lanes, H);
            }
            const int left = H - (j * lanes + t) * V;   // columns of this vector that exist
            const float rj = RMS || left > 0 ? r : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[j][i] = (xh[j][i] - m) * rj;
                if constexpr (TAIL && !RMS) xh[j][i] = i < left ? xh[j][i] : 0.0f;
                c[j][i] = d[i] * wr[j][i];
                dw[j][i] += d[i] * xh[j][i];
                if constexpr (!RMS) {
                    db[j][i] += d[i];
                    s[1] += c[j][i];
                }
                s[0] += c[j][i] * xh[j][i];
            }
        }
        row_sums<G, 2>(s, sums[turn]);
        const float cx_mean = s[0] / n, c_mean = RMS ? 0.0f : s[1] / n;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = r * (c[j][i] - c_mean - xh[j][i] * cx_mean);
            R::store(dx + (size_t)row * H, j, t, lanes, full, last, o);
            cx[j] = nx[j];
            cd[j] = nd[j];
        }
        st = nst;
    }
    size_t at_part = blockIdx.x;
    if constexpr (G != 0) {
        // the rows of a wave's groups: one partial row a wave
#pragma unroll
        for (int d = G; d < kWave; d <<= 1)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dw[j][i] += __shfl_xor(dw[j][i], d);
                    db[j][i] += __shfl_xor(db[j][i], d);
                }
        at_part = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
        if (lane_id() >= G) return;
    }
    float* pw = part + at_part * parts * H;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (j * lanes + t) * V + i;
            if (col < H) {
                pw[col] = dw[j][i];
                if (!RMS && parts == 2) pw[H + col] = db[j][i];
            }
        }
}

// out[c] = sum over p < n of part[p][c] for the W = parts x H columns: a
// workgroup takes 64 columns, its 16 waves each every 16th partial row, and
// adds the 16 sums in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void norm_sum_kernel(const float* __restrict__ part, int n, int H, int W,
                                                                  float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float s[kSumWaves][64];
    const int lane = lane_id(), wv = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (c < W) {
        int p = wv;
        for (; p + 7 * kSumWaves < n; p += 8 * kSumWaves) {   // eight loads in flight
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = part[(size_t)(p + i * kSumWaves) * W + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) v += u[i];
        }
        for (; p < n; p += kSumWaves) v += part[(size_t)p * W + c];
    }
    s[wv][lane] = v;
    __syncthreads();
    if (wv == 0 && c < W) {
        for (int i = 1; i < kSumWaves; ++i) v += s[i][lane];
        if (c < H) dw[c] = v;
        else db[c - H] = v;
    }
}

// How H columns are held: lanes of a wave (g), or a workgroup of `threads` with
// nv vectors a lane.
struct Shape {
    int g, nv, threads;
};
Shape shape_of(int H, int V) {
    const int n = (H + V - 1) / V;
    if (n <= 64) return {n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64, 1, 256};
    const int nv = n <= 1024 ? 1 : n <= 2048 ? 4 : 8;
    return {0, nv, ((n + nv - 1) / nv + 63) / 64 * 64};
}
int values_of(int dtype) { return dtype == 1 ? 8 : 4; }

// Results larger than the 256 MB of the last cache with their operands are
// written past it (backward, 8192 x 6144 bf16, 302 MB: 66 against 75 us; the
// forward, 201 MB: 32 against 33); smaller ones are left for the next reader.
bool past_caches(const NormParams& p, int tensors) {
    return (double)p.rows * p.H * (p.dtype == 1 ? 2 : 4) * tensors > 256e6;
}

// f(nv, g) for the shape's template arguments
template <int V, typename F>
void with_shape(const Shape& s, F&& f) {
    using std::integral_constant;
    const integral_constant<int, 1> one = {};
    if (s.g == 8) f(one, integral_constant<int, 8>{});
    else if (s.g == 16) f(one, integral_constant<int, 16>{});
    else if (s.g == 32) f(one, integral_constant<int, 32>{});
    else if (s.g == 64) f(one, integral_constant<int, 64>{});
    else if (s.nv == 1) f(one, integral_constant<int, 0>{});
    else if (s.nv == 4) f(integral_constant<int, 4>{}, integral_constant<int, 0>{});
    else if constexpr (V == 4) f(integral_constant<int, 8>{}, integral_constant<int, 0>{});   // fp32 past 8192 columns
}

// workgroups that hold `rows` rows, at most `most`
int workgroups(const Shape& s, int rows, int most) {
    const int per = s.g == 0 ? 1 : 256 / s.g;
    return std::max(1, std::min((rows + per - 1) / per, most));
}

template <typename TE, bool TAIL, bool RMS>
hipError_t forward_typed(const NormParams& p, hipStream_t stream) {
    const Shape s = shape_of(p.H, values_of(p.dtype));
    const int grid = workgroups(s, p.rows, device_cu_count() * (2048 / s.threads));
    auto go = [&](auto nt) {
        with_shape<16 / sizeof(TE)>(s, [&](auto nv, auto g) {
            hipLaunchKernelGGL((norm_forward_kernel<TE, decltype(nv)::value, decltype(g)::value, TAIL, RMS,
                                                    decltype(nt)::value>),
                               dim3(grid), dim3(s.threads), 0, stream, static_cast<const TE*>(p.x), p.weight, p.bias,
                               p.rows, p.H, p.eps, static_cast<TE*>(p.out), p.stats_out);
        });
    };
    if (!TAIL && past_caches(p, 2)) go(std::integral_constant<bool, !TAIL>{});
    else go(std::false_type{});
    return hipGetLastError();
}

// Workgroups of the backward pass.  Each ends with one partial row (narrow rows:
// four) that is written and read back, so each takes 4 rows a lane or more, and
// 16 or more where 512 workgroups are enough; at most what the card holds.
// Several vectors a lane: one workgroup a CU is what the registers allow (256
// against 512 workgroups, 4096 x 12288 bf16: 76 us against 92; 8192 x 16384: 174
// against 198; 16384 x 8192 fp32: 296 against 312).
int backward_grid(const Shape& s, int rows) {
    const int per = s.g == 0 ? 1 : 256 / s.g;
    const int steps = (rows + per - 1) / per;
    const int most = s.nv > 1 ? 256 : std::min(std::max(512, steps / 16), 256 * std::max(1, 2048 / s.threads));
    return std::max(1, std::min((steps + 3) / 4, most));
}

template <typename TE, bool TAIL, bool RMS>
hipError_t backward_typed(const NormParams& p, hipStream_t stream) {
    const Shape s = shape_of(p.H, values_of(p.dtype));
    const int grid = backward_grid(s, p.rows);
    const int parts = p.dbias != nullptr ? 2 : 1;
    auto go = [&](auto nt) {
        with_shape<16 / sizeof(TE)>(s, [&](auto nv, auto g) {
            hipLaunchKernelGGL((norm_backward_kernel<TE, decltype(nv)::value, decltype(g)::value, TAIL, RMS,
                                                     decltype(nt)::value>),
                               dim3(grid), dim3(s.threads), 0, stream, static_cast<const TE*>(p.dout),
                               static_cast<const TE*>(p.x), p.stats, p.weight, p.rows, p.H, parts,
                               static_cast<TE*>(p.dx), p.part);
        });
    };
    if (!TAIL && past_caches(p, 3)) go(std::integral_constant<bool, !TAIL>{});
    else go(std::false_type{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int W = parts * p.H;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((W + 63) / 64), dim3(64 * kSumWaves), 0, stream, p.part,
                       norm_parts(p.dtype, p.rows, p.H), p.H, W, p.dweight, p.dbias);
    return hipGetLastError();
}

template <typename F>
hipError_t by_type(const NormParams& p, F&& f) {
    const bool tail = p.H % values_of(p.dtype) != 0;
    auto kind = [&](auto te, auto tl) { return p.rms ? f(te, tl, std::true_type{}) : f(te, tl, std::false_type{}); };
    auto ends = [&](auto te) { return tail ? kind(te, std::true_type{}) : kind(te, std::false_type{}); };
    return p.dtype == 1 ? ends(bf16_t{}) : ends(float{});
}

}  // namespace

int norm_parts(int dtype, int rows, int H) {
    const Shape s = shape_of(H, values_of(dtype));
    return backward_grid(s, rows) * (s.g == 0 ? 1 : 4);
}

hipError_t launch_norm_forward(const NormParams& p, hipStream_t stream) {
    return by_type(p, [&](auto te, auto tail, auto rms) {
        return forward_typed<decltype(te), decltype(tail)::value, decltype(rms)::value>(p, stream);
    });
}

hipError_t launch_norm_backward(const NormParams& p, hipStream_t stream) {
    return by_type(p, [&](auto te, auto tail, auto rms) {
        return backward_typed<decltype(te), decltype(tail)::value, decltype(rms)::value>(p, stream);
    });
}

}  // namespace inkling
