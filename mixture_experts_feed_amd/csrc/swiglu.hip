// SwiGLU between an expert's two projections with its input kept in 8 bits.
//
// h [R][2I] holds [g0, u0, g1, u1, ...]; act = gamma g sigmoid(g) u.  For the
// backward pass h is kept as one byte a value: 32 consecutive columns share a
// power of two 2^e, the smallest (e >= -126) with max|h| <= 127 2^e, and each
// value is the int8 nearest to h / 2^e (ties to even), off by at most 2^(e-1).
// That is at most max|h| / 127 of its block while e > -126, that is from
// max|h| > 127 2^-127 on; below, at most 2^-127.  A power of two makes h / 2^e and q 2^e
// exact, so that the kept values do not depend on how a quotient is rounded.
// The exponent is a byte, e + 127; 255 marks a block with an infinity or a NaN,
// whose values come back as NaN.
// The backward pass takes g and u from the bytes:
//   s = sigmoid(g), p = g s u:  a = gamma p,  dgamma = sum over I of dact p,
//   dg = gamma dact u s (1 + g (1 - s)),  du = gamma dact g s.
//
// Both passes are one read of their inputs and one write of their outputs, so
// HBM bounds them: per row of I columns bf16 moves 8 I bytes forward (4 I in,
// 2 I + 2 I out) and 10 I backward (2 I + 2 I in, 4 I + 2 I out).  A lane holds
// 16 bytes of h (8 bf16 or 4 fp32 columns), so that every access of a wave is
// one contiguous run; with 16 columns a lane, two accesses 32 bytes apart, the
// backward took 268 us for 65536 rows of 2048 where this takes 234 (5.7 TB/s; the
// forward 201 us, 5.4 TB/s).
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec.h"

namespace inkling {

namespace {

// columns of h a lane holds, and lanes that share an exponent
template <typename TE>
constexpr int cols() { return 16 / (int)sizeof(TE); }
template <typename TE>
constexpr int block_lanes() { return 32 / cols<TE>(); }

// bf16 rows take the hardware exponential and reciprocal: exp(-v) as 2^(-v log2 e)
// is off by (1.5 |v| + 2) 2^-24 of itself (the rounding of v log2 e grows with |v|),
// the sum and the reciprocal by 3 steps more: 2^-18 at |v| = 40, against bf16's
// half step of 2^-8.  fp32 rows take the library exponential and a division.  Below
// v = -87.3, where the sigmoid is less than 2^-126, it may come out as 0 (exp(-v)
// passes fp32 at -88.7).
template <typename TE>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (sizeof(TE) == 2) return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    else return 1.0f / (1.0f + expf(-v));
}

// Kept byte of the exponent for a block whose largest |h| has these bits.
// Adding 0x1FFFF carries into the exponent exactly when the significand passes
// 127/64 = 1.1111110b, the largest that 127 steps of 2^(exponent - 6) hold.
__device__ __forceinline__ int exponent_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255;
    return max((int)((top + 0x1FFFFu) >> 23) - 6, 1);
}

template <typename TE, bool NT>
__global__ __launch_bounds__(256) void swiglu_forward_kernel(const TE* __restrict__ h, const float* __restrict__ gamma,
                                                             const int32_t* __restrict__ row_count, int row0, int rows,
                                                             int I, TE* __restrict__ act, int8_t* __restrict__ kept,
                                                             uint8_t* __restrict__ exps) {
    constexpr int C = cols<TE>(), P = C / 2, BL = block_lanes<TE>();
    const int end = row_count != nullptr ? min(rows, max(*row_count, row0) - row0) : rows;
    const uint32_t per_row = 2u * (uint32_t)I / C;            // lanes a row takes
    const uint32_t total = (uint32_t)end * per_row;           // < 2^31 (launcher)
    for (uint32_t c = blockIdx.x * 256 + threadIdx.x; c < total; c += gridDim.x * 256) {
        const size_t row = row0 + c / per_row;
        const uint32_t lane = c % per_row;
        const size_t at = row * 2 * I + (size_t)lane * C;
        float v[C];
        widen<TE, C>(get<Raw<TE, C>, NT>(h + at), v);
        const float gm = gamma != nullptr ? gamma[row] : 1.0f;
        float a[P];
#pragma unroll
        for (int i = 0; i < P; ++i) a[i] = gm * (v[2 * i] * sigmoid_of<TE>(v[2 * i]) * v[2 * i + 1]);
        put<NT>(act + at / 2, narrow<TE, P>(a));
        if (kept != nullptr) {
            uint32_t top = 0;   // integer order of |h|: NaN above infinity
#pragma unroll
            for (int i = 0; i < C; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
            for (int d = 1; d < BL; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
            const int e = exponent_byte(top);
            const float inv = e == 255 ? 0.0f : __uint_as_float((uint32_t)(254 - e) << 23);
            // h / 2^e + 1.5 2^23 rounds to an integer, nearest even, whose low
            // byte is the int8
            Raw<int8_t, C> w;
            uint32_t word[C / 4];
#pragma unroll
            for (int j = 0; j < C / 4; ++j) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__builtin_fmaf(v[4 * j + i], inv, 12582912.0f));
                word[j] = (b[0] & 0xFFu) | (b[1] & 0xFFu) << 8 | (b[2] & 0xFFu) << 16 | b[3] << 24;
            }
            __builtin_memcpy(&w, word, sizeof(w));
            put<NT>(kept + at, w);
            if (lane % BL == 0) exps[row * (size_t)(I / 16) + lane / BL] = (uint8_t)e;
        }
    }
}

// G lanes a row (a row's lanes are neighbours in a wave): dgamma is the sum of
// a fixed order over a lane's columns, then over the lanes.
template <typename TE, int G, bool NT>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(
    const TE* __restrict__ dact, const int8_t* __restrict__ kept, const uint8_t* __restrict__ exps,
    const float* __restrict__ gamma, const int32_t* __restrict__ row_count, int rows, int I, TE* __restrict__ dh,
    TE* __restrict__ act, float* __restrict__ dgamma) {
    constexpr int C = cols<TE>(), P = C / 2, BL = block_lanes<TE>(), kRows = 256 / G;
    const int end = row_count != nullptr ? max(0, min(rows, *row_count)) : rows;
    const int sub = threadIdx.x % G, per_row = 2 * I / C;
    for (long long r = (long long)blockIdx.x * kRows + threadIdx.x / G; r < end; r += (long long)gridDim.x * kRows) {
        const size_t row = (size_t)r;
        const float gm = gamma != nullptr ? gamma[row] : 1.0f;
        float part = 0.0f;
#pragma unroll 4
        for (int lane = sub; lane < per_row; lane += G) {
            const size_t at = row * 2 * I + (size_t)lane * C;
            const Raw<int8_t, C> q = get<Raw<int8_t, C>, NT>(kept + at);
            const int e = exps[row * (size_t)(I / 16) + lane / BL];
            const float scale = __uint_as_float(e == 255 ? 0x7FC00000u : (uint32_t)e << 23);
            float da[P];
            widen<TE, P>(get<Raw<TE, P>, NT>(dact + at / 2), da);
            uint32_t word[C / 4];
            __builtin_memcpy(word, &q, sizeof(q));
            float dv[C], av[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint32_t pair = word[i >> 1] >> (16 * (i & 1));
                const float g = (float)(int8_t)(pair & 0xFFu) * scale;
                const float u = (float)(int8_t)((pair >> 8) & 0xFFu) * scale;
                const float s = sigmoid_of<TE>(g);
                const float si = g * s, p = si * u;
                const float dp = gm * da[i];
                part += da[i] * p;
                av[i] = gm * p;
                dv[2 * i] = dp * u * s * (1.0f + g * (1.0f - s));
                dv[2 * i + 1] = dp * si;
            }
            put<NT>(dh + at, narrow<TE, C>(dv));
            if (act != nullptr) put<NT>(act + at / 2, narrow<TE, P>(av));
        }
        if (dgamma != nullptr) {
            part = lanes_sum<G>(part);
            if (sub == 0) dgamma[row] = part;
        }
    }
}

// Lanes a row: the widest of which three quarters or more have columns (few
// steps a row: 104 vectors take 64 lanes twice, 4.4 us for 1003 rows, against 9.1
// with 8 lanes 13 times), else the one with the fewest idle.
int lanes_per_row(int per_row) {
    int best = 8;
    double most = 0.0;
    for (int g = 64; g >= 8; g /= 2) {
        const double used = (double)per_row / ((per_row + g - 1) / g * g);
        if (used >= 0.75) return g;
        if (used > most) {
            most = used;
            best = g;
        }
    }
    return best;
}

// Data that the 256 MB of the last cache cannot hold goes past it (65536 rows of
// 2048 bf16: forward 201 against 215 us, backward 234 against 240; the stores
// make the difference); smaller data is left for the next reader.
bool past_caches(const SwigluParams& p, double bytes_per_value) {
    return (double)p.rows * p.I * bytes_per_value > 256e6;
}

template <typename TE>
hipError_t backward_typed(const SwigluParams& p, hipStream_t stream) {
    const int G = lanes_per_row(2 * p.I / cols<TE>());
    const long long blocks = ((long long)p.rows * G + 255) / 256;
    const dim3 grid((unsigned)std::min<long long>(blocks, (long long)device_cu_count() * 32));
    auto go = [&](auto g, auto nt) {
        hipLaunchKernelGGL((swiglu_backward_kernel<TE, decltype(g)::value, decltype(nt)::value>), grid, dim3(256), 0,
                           stream, static_cast<const TE*>(p.dact), p.kept, p.exps, p.gamma, p.row_count, p.rows, p.I,
                           static_cast<TE*>(p.dh), static_cast<TE*>(p.act), p.dgamma);
    };
    auto width = [&](auto nt) {
        if (G == 64) go(std::integral_constant<int, 64>{}, nt);
        else if (G == 32) go(std::integral_constant<int, 32>{}, nt);
        else if (G == 16) go(std::integral_constant<int, 16>{}, nt);
        else go(std::integral_constant<int, 8>{}, nt);
    };
    if (past_caches(p, 2.0 + 4 * sizeof(TE))) width(std::true_type{});
    else width(std::false_type{});
    return hipGetLastError();
}

template <typename TE>
hipError_t forward_typed(const SwigluParams& p, hipStream_t stream) {
    const unsigned per_row = 2u * (unsigned)p.I / cols<TE>();
    const bool nt = past_caches(p, (p.kept != nullptr ? 2.0 : 0.0) + 3 * sizeof(TE));
    // bands of rows whose lanes a 32-bit index counts (with room for the stride)
    const int band = std::max(1, (int)((1u << 30) / per_row));
    for (int row0 = 0; row0 < p.rows; row0 += std::min(band, p.rows - row0)) {
        const int n = std::min(band, p.rows - row0);
        const long long blocks = ((long long)n * per_row + 255) / 256;
        const dim3 grid((unsigned)std::min<long long>(blocks, (long long)device_cu_count() * 32));
        auto go = [&](auto past) {
            hipLaunchKernelGGL((swiglu_forward_kernel<TE, decltype(past)::value>), grid, dim3(256), 0, stream,
                               static_cast<const TE*>(p.h), p.gamma, p.row_count, row0, n, p.I,
                               static_cast<TE*>(p.act), p.kept, p.exps);
        };
        if (nt) go(std::true_type{});
        else go(std::false_type{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_swiglu_forward(const SwigluParams& p, hipStream_t stream) {
    return p.dtype == 1 ? forward_typed<bf16_t>(p, stream) : forward_typed<float>(p, stream);
}

hipError_t launch_swiglu_backward(const SwigluParams& p, hipStream_t stream) {
    return p.dtype == 1 ? backward_typed<bf16_t>(p, stream) : backward_typed<float>(p, stream);
}

}  // namespace inkling
