// Layer norm and RMS norm over the rows of x [R][H], forward and backward.
//
//   y = (x - m) r w + b,  r = 1 / sqrt(mean((x - m)^2) + eps),  m = mean(x)
//   (RMS norm: m = 0 and no b).  With xh = (x - m) r and c = dy w:
//   dx = r (c - mean(c) - xh mean(c xh))   (RMS norm: without mean(c))
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// HBM bounds both passes: x is read once and kept in registers for the second
// moment about the mean (two passes over registers, so a large mean costs no
// digits), the result is written once.  A workgroup walks rows with its columns
// of w and b in registers, and loads the next row before the sums of the
// current one.  The backward pass keeps its columns' sums of dw and db in
// registers over all its rows and writes one partial row for each workgroup;
// a second kernel adds the partial rows in order, so results repeat bit for bit.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec.h"

namespace inkling {

namespace {

// Sums over a workgroup of TPR threads (one wave: no LDS).  `buf` alternates
// from call to call, so one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*buf)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TPR > kWave) {
        const int wv = threadIdx.x >> 6;
        if (lane_id() == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[wv][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = buf[0][i];
#pragma unroll
            for (int w = 1; w < TPR / kWave; ++w) v[i] += buf[w][i];
        }
    }
}

// V values a vector, NV vectors a thread: vector j of a thread is columns
// (j TPR + thread) V.
template <typename TE, int V, int NV, int TPR, bool RMS>
__global__ __launch_bounds__(TPR) void norm_forward_kernel(const TE* __restrict__ x, const float* __restrict__ w,
                                                           const float* __restrict__ b, int rows, int H, float eps,
                                                           TE* __restrict__ out, float* __restrict__ stats) {
    __shared__ float sums[2][2][TPR / kWave][1];
    const int nv = H / V, t = threadIdx.x;
    const float inv_h = 1.0f / (float)H;
    float wr[NV][V], br[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = j * TPR + t < nv;
            const int col = (j * TPR + t) * V + i;
            wr[j][i] = in ? w[col] : 0.0f;
            br[j][i] = in && b != nullptr ? b[col] : 0.0f;
        }
    Raw<TE, V> cur[NV], nxt[NV];
    auto load = [&](Raw<TE, V>* r, size_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) r[j] = load_raw<TE, V>(x + row * H + (size_t)(j * TPR + t) * V);
    };
    int row = blockIdx.x, turn = 0;
    load(cur, row);
    for (; row < rows; row += gridDim.x, turn ^= 1) {
        if (row + (int)gridDim.x < rows) load(nxt, (size_t)row + gridDim.x);
        float v[NV][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) {
                widen(cur[j], v[j]);
                if constexpr (!RMS)
#pragma unroll
                    for (int i = 0; i < V; ++i) s[0] += v[j][i];
            }
        float m = 0.0f;
        if constexpr (!RMS) {
            block_sums<TPR, 1>(s, sums[turn][0]);
            m = s[0] * inv_h;
        }
        s[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv)
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] += (v[j][i] - m) * (v[j][i] - m);
        block_sums<TPR, 1>(s, sums[turn][1]);
        const float r = 1.0f / sqrtf(s[0] * inv_h + eps);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) {
                float y[V];
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = (v[j][i] - m) * r * wr[j][i] + br[j][i];
                store_vec<TE, V>(out + (size_t)row * H + (size_t)(j * TPR + t) * V, y);
            }
        if (stats != nullptr && t == 0) *reinterpret_cast<float2*>(stats + 2 * (size_t)row) = make_float2(m, r);
#pragma unroll
        for (int j = 0; j < NV; ++j) cur[j] = nxt[j];
    }
}

// part [gridDim.x][2][H] (RMS norm or no bias wanted: [gridDim.x][1][H])
template <typename TE, int V, int NV, int TPR, bool RMS>
__global__ __launch_bounds__(TPR) void norm_backward_kernel(const TE* __restrict__ dout, const TE* __restrict__ x,
                                                            const float* __restrict__ stats,
                                                            const float* __restrict__ w, int rows, int H, int parts,
                                                            TE* __restrict__ dx, float* __restrict__ part) {
    __shared__ float sums[2][TPR / kWave][2];
    const int nv = H / V, t = threadIdx.x;
    const float inv_h = 1.0f / (float)H;
    float wr[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wr[j][i] = j * TPR + t < nv ? w[(j * TPR + t) * V + i] : 0.0f;
            dw[j][i] = 0.0f;
            db[j][i] = 0.0f;
        }
    Raw<TE, V> cx[NV], cd[NV], nx[NV], nd[NV];
    auto load = [&](Raw<TE, V>* r, const TE* p, size_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) r[j] = load_raw<TE, V>(p + row * H + (size_t)(j * TPR + t) * V);
    };
    int row = blockIdx.x, turn = 0;
    if (row < rows) {
        load(cx, x, row);
        load(cd, dout, row);
    }
    for (; row < rows; row += gridDim.x, turn ^= 1) {
        const float2 st = *reinterpret_cast<const float2*>(stats + 2 * (size_t)row);
        const float m = RMS ? 0.0f : st.x, r = st.y;
        if (row + (int)gridDim.x < rows) {
            load(nx, x, (size_t)row + gridDim.x);
            load(nd, dout, (size_t)row + gridDim.x);
        }
        float xh[NV][V], c[NV][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) {
                float d[V];
                widen(cx[j], xh[j]);
                widen(cd[j], d);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[j][i] = (xh[j][i] - m) * r;
                    c[j][i] = d[i] * wr[j][i];
                    dw[j][i] += d[i] * xh[j][i];
                    if constexpr (!RMS) {
                        db[j][i] += d[i];
                        s[1] += c[j][i];
                    }
                    s[0] += c[j][i] * xh[j][i];
                }
            }
        block_sums<TPR, 2>(s, sums[turn]);
        const float cx_mean = s[0] * inv_h, c_mean = RMS ? 0.0f : s[1] * inv_h;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TPR + t < nv) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = r * (c[j][i] - c_mean - xh[j][i] * cx_mean);
                store_vec<TE, V>(dx + (size_t)row * H + (size_t)(j * TPR + t) * V, o);
            }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            cx[j] = nx[j];
            cd[j] = nd[j];
        }
    }
    float* pw = part + (size_t)blockIdx.x * parts * H;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (j * TPR + t < nv)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                pw[(j * TPR + t) * V + i] = dw[j][i];
                if (!RMS && parts == 2) pw[H + (j * TPR + t) * V + i] = db[j][i];
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
    if (c < W)
        for (int p = wv; p < n; p += kSumWaves) v += part[(size_t)p * W + c];
    s[wv][lane] = v;
    __syncthreads();
    if (wv == 0 && c < W) {
        for (int i = 1; i < kSumWaves; ++i) v += s[i][lane];
        if (c < H) dw[c] = v;
        else db[c - H] = v;
    }
}

// Threads a row and vectors a thread for H columns in vectors of V: one wave up
// to 2 vectors a lane, then 256 threads up to 4, 512 and 1024 (unaligned rows:
// 256 or 1024 threads, up to 16 single values).
struct Shape {
    int tpr, nv;
};
Shape shape_of(int H, int V) {
    const int n = H / V;
    if (V == 1) {
        if (n <= 256 * 4) return {256, 4};
        if (n <= 256 * 16) return {256, 16};
        return {1024, 16};
    }
    if (n <= 128) return {64, 2};
    if (n <= 1024) return {256, (n + 255) / 256};
    if (n <= 2048) return {512, 4};
    return {1024, 4};
}

template <typename TE, int V, bool RMS, typename F>
void with_shape(int H, F&& f) {
    const Shape s = shape_of(H, V);
    auto go = [&](auto nv, auto tpr) { f(nv, tpr); };
#define NORM_SHAPE(NV_, TPR_) \
    if (s.nv == NV_ && s.tpr == TPR_) return go(std::integral_constant<int, NV_>{}, std::integral_constant<int, TPR_>{})
    if constexpr (V == 1) {
        NORM_SHAPE(4, 256);
        NORM_SHAPE(16, 256);
        NORM_SHAPE(16, 1024);
    } else {
        NORM_SHAPE(2, 64);
        NORM_SHAPE(1, 256);
        NORM_SHAPE(2, 256);
        NORM_SHAPE(3, 256);
        NORM_SHAPE(4, 256);
        NORM_SHAPE(4, 512);
        if constexpr (V == 4) NORM_SHAPE(4, 1024);   // past 8192 columns
    }
#undef NORM_SHAPE
}

template <typename TE, int V, bool RMS>
hipError_t forward_typed(const NormParams& p, hipStream_t stream) {
    with_shape<TE, V, RMS>(p.H, [&](auto nv, auto tpr) {
        constexpr int NV = decltype(nv)::value, TPR = decltype(tpr)::value;
        const int grid = std::min(p.rows, device_cu_count() * (2048 / TPR));
        hipLaunchKernelGGL((norm_forward_kernel<TE, V, NV, TPR, RMS>), dim3(grid), dim3(TPR), 0, stream,
                           static_cast<const TE*>(p.x), p.weight, p.bias, p.rows, p.H, p.eps, static_cast<TE*>(p.out),
                           p.stats_out);
    });
    return hipGetLastError();
}

template <typename TE, int V, bool RMS>
hipError_t backward_typed(const NormParams& p, hipStream_t stream) {
    const int grid = norm_parts(p.rows, p.H);
    const int parts = p.dbias != nullptr ? 2 : 1;
    with_shape<TE, V, RMS>(p.H, [&](auto nv, auto tpr) {
        constexpr int NV = decltype(nv)::value, TPR = decltype(tpr)::value;
        hipLaunchKernelGGL((norm_backward_kernel<TE, V, NV, TPR, RMS>), dim3(grid), dim3(TPR), 0, stream,
                           static_cast<const TE*>(p.dout), static_cast<const TE*>(p.x), p.stats, p.weight, p.rows, p.H,
                           parts, static_cast<TE*>(p.dx), p.part);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int W = parts * p.H;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((W + 63) / 64), dim3(64 * kSumWaves), 0, stream, p.part, grid, p.H, W,
                       p.dweight, p.dbias);
    return hipGetLastError();
}

// 16-byte vectors where rows are whole vectors (the entry points ask for
// 16-byte aligned tensors), else single values
template <typename F>
hipError_t by_type(const NormParams& p, F&& f) {
    auto kind = [&](auto te, auto v) { return p.rms ? f(te, v, std::true_type{}) : f(te, v, std::false_type{}); };
    using One = std::integral_constant<int, 1>;
    if (p.dtype == 1)
        return p.H % 8 == 0 ? kind(bf16_t{}, std::integral_constant<int, 8>{}) : kind(bf16_t{}, One{});
    return p.H % 4 == 0 ? kind(float{}, std::integral_constant<int, 4>{}) : kind(float{}, One{});
}

}  // namespace

// Workgroups of the backward pass, one partial row each: 16 rows or more for
// each, so that the partial rows stay a small part of the traffic, two a CU.
int norm_parts(int rows, int H) { return std::max(1, std::min((rows + 15) / 16, 512)); }

hipError_t launch_norm_forward(const NormParams& p, hipStream_t stream) {
    return by_type(p, [&](auto te, auto v, auto rms) {
        return forward_typed<decltype(te), decltype(v)::value, decltype(rms)::value>(p, stream);
    });
}

hipError_t launch_norm_backward(const NormParams& p, hipStream_t stream) {
    return by_type(p, [&](auto te, auto v, auto rms) {
        return backward_typed<decltype(te), decltype(v)::value, decltype(rms)::value>(p, stream);
    });
}

}  // namespace inkling
