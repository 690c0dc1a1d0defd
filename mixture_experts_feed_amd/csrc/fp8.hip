// 8-bit floating point (e4m3) with a scale for each block of 128: rows and weights
// turned into it, and products grouped by expert.
//
// Quantising: the scale of a block (128 columns of a row; 128 x 128 of a weight) is the
// smallest power of two 2^e, e >= -126, with max|block| <= 448 2^e, so v / 2^e is exact
// and each value is rounded once, to nearest even (v_cvt_pk_fp8_f32; tested on every e4m3
// value, every midpoint of two and the numbers next to each of them, of both signs).  Half a
// step is 2^-4 of a value from 2^-6 2^e on, and 2^-10 2^e below.  A block with an infinity or a NaN gets a NaN scale and zeros, so that
// every product with it is NaN.  One read and one write: HBM bounds both kernels (8192
// rows of 6144: bf16 25 to 29 us, 5.2 to 6.0 TB/s, fp32 35; weights 32 x 4096 x 6144: bf16 449
// us, 5.4 TB/s, fp32 720, 5.6).
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "common.h"
#include "fp8_common.h"
#include "fp8_stream.h"
#include "fp8_tiles.h"
#include "kernels.h"
#include "vec.h"

namespace inkling {

namespace {

// Eight values of TE as they lie in memory, and widened
template <typename TE>
struct Eight {
    Raw<TE, 16 / (int)sizeof(TE)> r[8 * sizeof(TE) / 16];
    __device__ __forceinline__ void load(const TE* p) {
        constexpr int V = 16 / (int)sizeof(TE);
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) r[i] = *reinterpret_cast<const Raw<TE, V>*>(p + i * V);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (size_t i = 0; i < sizeof(r) / sizeof(r[0]); ++i) r[i] = {};
    }
    __device__ __forceinline__ void get(float* v) const {
        constexpr int V = 16 / (int)sizeof(TE);
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) widen<TE, V>(r[i], v + i * V);
    }
    // largest |v|, in integer order (NaN above infinity)
    __device__ __forceinline__ uint32_t top() const {
        float v[8];
        get(v);
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        return t;
    }
};

// Scale of a block whose largest |v| has these bits, and its inverse (0: every value
// becomes 0).  448 = 1.75 2^8: adding 0x1FFFFF carries into the exponent exactly when the
// significand passes 1.75.
__device__ __forceinline__ float block_scale(uint32_t top, float& inv) {
    if (top >= 0x7F800000u) {
        inv = 0.0f;
        return __uint_as_float(0x7FC00000u);
    }
    const int e = max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
    return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ uint2 to_fp8(const float* v, float inv) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = inv == 0.0f ? 0.0f : v[i] * inv;
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// largest over 16 neighbouring lanes
__device__ __forceinline__ uint32_t lanes16_max(uint32_t v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    return dpp_max<0x140>(v);
}

// 16 lanes a block of a row, eight values each
template <typename TE>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const TE* __restrict__ x, const int32_t* __restrict__ row_count,
                                                            int rows, int cols, uint8_t* __restrict__ out,
                                                            float* __restrict__ scales) {
    const uint32_t nb = (uint32_t)(cols + kQBlock - 1) / kQBlock;
    const int end = row_count != nullptr ? max(0, min(rows, *row_count)) : rows;
    const uint32_t total = (uint32_t)end * nb;   // < 2^31 (host)
    const int sub = threadIdx.x & 15;
    for (uint32_t u = blockIdx.x * 16u + (threadIdx.x >> 4); u < total; u += gridDim.x * 16u) {
        const uint32_t row = u / nb, col = (u - row * nb) * kQBlock + sub * 8;
        const size_t at = (size_t)row * cols + col;
        Eight<TE> v;
        v.zero();
        const bool in = (int)col < cols;   // cols is a multiple of 16
        if (in) v.load(x + at);
        float inv, w[8];
        const float s = block_scale(lanes16_max(v.top()), inv);
        v.get(w);
        if (in) *reinterpret_cast<uint2*>(out + at) = to_fp8(w, inv);
        if (sub == 0) scales[u] = s;
    }
}

// A workgroup a block of 128 x 128: 16 lanes a row, 16 rows at a time
template <typename TE>
__global__ __launch_bounds__(256) void quantize_weight_kernel(const TE* __restrict__ w, int E, int N, int K,
                                                              uint8_t* __restrict__ out, float* __restrict__ scales) {
    __shared__ uint32_t tops[2][4];
    const int nb = (N + kQBlock - 1) / kQBlock, kb = (K + kQBlock - 1) / kQBlock;
    const long long total = (long long)E * nb * kb;
    const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    int turn = 0;
    for (long long u = blockIdx.x; u < total; u += gridDim.x, turn ^= 1) {
        const long long rest = u / kb;
        const int b = (int)(u - rest * kb), n = (int)(rest % nb), e = (int)(rest / nb);
        const int col = b * kQBlock + sub * 8;
        Eight<TE> v[8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = n * kQBlock + i * 16 + r0;
            v[i].zero();
            if (row < N && col < K) v[i].load(w + ((size_t)e * N + row) * K + col);
            top = max(top, v[i].top());
        }
        top = lanes16_max(top);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (lane_id() == 0) tops[turn][threadIdx.x >> 6] = top;   // two in turn: one barrier a block
        __syncthreads();
        top = max(max(tops[turn][0], tops[turn][1]), max(tops[turn][2], tops[turn][3]));
        float inv;
        const float s = block_scale(top, inv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = n * kQBlock + i * 16 + r0;
            float f[8];
            v[i].get(f);
            if (row < N && col < K) *reinterpret_cast<uint2*>(out + ((size_t)e * N + row) * K + col) = to_fp8(f, inv);
        }
        if (threadIdx.x == 0) scales[u] = s;
    }
}

Fp8Args fp8_args(const Fp8Params& p) {
    Fp8Args a = {};
    a.weight = static_cast<const uint8_t*>(p.weight);
    a.weight_scale = p.weight_scale;
    a.x = static_cast<const uint8_t*>(p.x);
    a.x_scale = p.x_scale;
    a.row_index = p.row_index;
    a.offsets = p.offsets;
    a.out = p.out;
    a.rows = p.rows;
    a.x_rows = p.x_rows;
    a.E = p.E;
    a.N = p.N;
    a.K = p.K;
    a.out_bf16 = p.out_bf16;
    return a;
}

// 64 x 64 tasks of the forward, at most, and as rows spread over a few experts make them
long long tasks64(const Fp8Params& p) { return (((long long)p.rows + 63) / 64 + p.E - 1) * ((p.N + 63) / 64); }
double expected64(const Fp8Params& p) {
    const double tiles = p.E == 1 ? (p.rows + 63LL) / 64 : std::max<double>(p.E, p.rows / 64.0 + p.E / 4.0);
    return tiles * ((p.N + 63) / 64);
}

// The forward streams the weights (fp8_stream.h) where experts have few rows; 256-row
// tiles otherwise, whose stages without rows cost little: 5.5 TB/s of weights at 2 to 48
// rows an expert.  us, streamed against tiles (E experts of r rows, K x N):
// - up to 8 rows and K from 2048 on: 387 / 465 at 128 x 2 (6144 x 4096), 78 / 98 at 128 x
//   2 and 101 / 106 at 128 x 8 (2048 x 2048), 77 / 114 at 64 x 2 (4096 x 2048), 36 / 38 at
//   64 x 2 (2048 x 1536); 22 / 14 at 64 x 2 (1024 x 1024);
// - up to 16 rows and K from 4096 on: 532 / 563 at 128 x 16 (6144 x 4096), 104 / 136 at 16
//   x 16 (6144 x 6144); 121 / 109 at 128 x 16 (2048 x 2048), 655 / 566 at 128 x 24 (6144 x
//   4096);
// - up to 48 rows where fewer than 64 tiles would run, K from 2048 on: 9.8 / 44 at one
//   expert of 1 row and 17 / 44 of 40 (6144 x 4096), 7.3 / 18 of 1 (2048 x 2048), 28 / 32 at 30
//   x 48 (4096 x 512), 18.6 / 19.4 at 60 x 40 (2048 x 256); from 1024 on with 16 tiles at most:
//   11.1 / 12.0 at 1 x 48 (1024 x 4096), 11.2 / 12.1 at 4 x 40 (1024 x 1024), otherwise up to 20
//   rows: 13.2 / 15.3 at 15 x 20 (1536 x 1024), 10.9 / 11.8 at 15 x 8 and 15.8 / 12.3 at 15 x 40
//   (1024 x 1024); 8.8 / 8.7 at 1 x 48 (512 x 4096);
// - any number where few experts' 64 x 64 tasks give a CU one at most (of several experts: a
//   tenth more by their average), since a tile's stages wait for their loads, and few CUs
//   have one, K from 2048 on: 29.5 / 48 at one expert of 256 rows and 51 / 48 of 320 (6144 x
//   4096), 16.6 / 18.8 of 512 and 24 / 19 of 768 (2048 x 2048), 24 / 33 at 2 x 100 and 39 / 33
//   at 4 x 64 (4096 x 4096), 22 / 32 at 2 x 256 (4096 x 2048), 27 / 32 at 16 x 48 and 39 / 33 at
//   16 x 60 (4096 x 1024), 17.9 / 18.9 at 8 x 100 (2048 x 1024), 26 / 19 at 4 x 150 (2048 x 2048).
bool fp8_streams(const Fp8Params& p) {
    if (p.input_grad) return false;
    const long long rows = p.rows, E = p.E, tiles = E * ((p.N + 255) / 256);
    if (p.K >= 2048 && E <= (p.K >= 4096 ? 16 : 8) && expected64(p) <= (E == 1 ? 1.0 : 1.1) * device_cu_count())
        return true;
    if (tiles < 64) return p.K >= 1024 && rows <= (p.K >= 2048 || tiles <= 16 ? 48 : 20) * E;
    return rows <= (p.K >= 4096 ? 16 : p.K >= 2048 ? 8 : 0) * E;
}

// Rows of a tile.  fp32 results take 128: the conversions need the registers.  Otherwise
// 256, or less where that leaves the last of few rounds of the grid nearly empty: of 256,
// 192, 128 and 64 what takes least by rounds times a stage's time (8192 x 8192 x 8192:
// 2.07, 1.64, 1.30, 0.91 us).  The experts' last tiles are half full on average.  us,
// against 256 rows: 150 / 167 for 16 experts of 8192 uneven rows (input gradient, 2048
// columns from 6144), 38 / 58 for one of 512 (6144 from 4096), 99 / 113 for 4 of 1000 (4096 x
// 4096); 73 / 64 for 32 of 300 (2048 x 2048), whose rounds come out differently.
int tile_rows(const Fp8Params& p) {
    if (!p.out_bf16) return 128;
    const double cus = device_cu_count(), ntn = ((p.input_grad ? p.K : p.N) + 255) / 256;
    int best = 256;
    double least = 0.0;
    for (const auto& c : {std::pair<int, double>{256, 2.07}, {192, 1.64}, {128, 1.30}, {64, 0.91}}) {
        const double tiles = p.E == 1 ? (p.rows + c.first - 1) / c.first : (double)p.rows / c.first + 0.5 * p.E;
        const double rounds = std::ceil(tiles * ntn / cus);
        if (c.first == 256) {
            least = rounds * c.second;
            if (rounds > 2.0) break;   // more rounds even out
        } else if (rounds * c.second < least) {
            least = rounds * c.second;
            best = c.first;
        }
    }
    return best;
}

template <int FM, bool KN, bool EXACT>
void launch_tiles(const Fp8Args& a, int grid, hipStream_t stream) {
    // offsets into the rows: 32 bits, or not
    if ((uint64_t)a.x_rows * (KN ? a.N : a.K) < (1ull << 32))
        hipLaunchKernelGGL((fp8_tile_kernel<FM, KN, EXACT, false>), dim3(grid), dim3(kTileThreads), 0, stream, a);
    else hipLaunchKernelGGL((fp8_tile_kernel<FM, KN, EXACT, true>), dim3(grid), dim3(kTileThreads), 0, stream, a);
}

template <int BN, int NW, int DEPTH, int FM>
void launch_stream_as(const Fp8Args& a, hipStream_t stream) {
    const long long tasks = ((long long)(a.rows + 16 * FM - 1) / (16 * FM) + a.E) * ((a.N + BN - 1) / BN);
    const long long most = (long long)device_cu_count() * stream_per_cu<BN, NW, DEPTH, FM>();
    const dim3 grid((unsigned)std::min<long long>(tasks, most)), block(NW * 64);
    if (a.out_bf16) hipLaunchKernelGGL((fp8_stream_kernel<BN, NW, DEPTH, FM, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((fp8_stream_kernel<BN, NW, DEPTH, FM, true>), grid, block, 0, stream, a);
}

// Rows of a task: 16, 32 or 64, so that few experts have more (their weights are read
// again).  Columns: 64 where that gives every CU two tasks (with 32 rows: three of four
// CUs one, with 64 rows: every second one), else 16, of which a CU holds three workgroups
// (two with 64 rows).  us, 64 columns against 16 (E experts of r rows, K x N):
// - 16 rows: 16.1 / 13.2 at 64 x 6 (2048 x 320, 320 tasks of 64 columns), 18.1 / 17.7 at 120 x
//   6 (2048 x 256, 480), 18.4 / 18.7 at 128 x 6 (512), 22.7 / 23.8 at 64 x 6
//   (2048 x 768, 768);
// - 32 rows: 15.8 / 13.1 at 2 x 12 (4096 x 4096, 128), 17.3 / 24.0 at 40 x 12 (4096 x 320, 200),
//   19.2 / 21.9 at 4 x 12 (4096 x 4096, 256), 27.6 / 33.7 at 7 x 12 (448);
// - 64 rows: 16.5 / 12.6 at 1 x 64 (2048 x 4096, 64), 28.1 / 35.5 at 1 x 128 (6144 x 4096, 128),
//   16.8 / 26.9 at 1 x 512 (2048 x 2048, 256).
// 16 columns and rows: eight waves share out a reduction from 16384 on where few CUs have
// more than a task (eight against four: 12.2 / 10.0 at 1 x 1 (8192 x 4096), 17.8 / 18.2
// (16384 x 4096), 16.9 / 21.4 (32768 x 512), 27 / 36 (65536 x 256)).
void launch_stream(const Fp8Params& p, const Fp8Args& a, hipStream_t stream) {
    const double mean = (double)a.rows / a.E;
    const long long cus = device_cu_count(), E = a.E, tasks = E * ((a.N + 63) / 64);
    if (mean <= (E == 1 ? 16.0 : 8.0)) {
        if (tasks >= 2 * cus) launch_stream_as<64, 4, 4, 1>(a, stream);
        else if (a.K >= 128 * kQBlock && E * ((a.N + 15) / 16) < 2 * cus) launch_stream_as<16, 8, 6, 1>(a, stream);
        else launch_stream_as<16, 4, 4, 1>(a, stream);
    } else if (mean <= (E == 1 ? 32.0 : 20.0)) {
        if (4 * tasks >= 3 * cus) launch_stream_as<64, 4, 4, 2>(a, stream);
        else launch_stream_as<16, 4, 4, 2>(a, stream);
    } else {
        if (2 * tasks64(p) >= cus) launch_stream_as<64, 4, 4, 4>(a, stream);
        else launch_stream_as<16, 4, 4, 4>(a, stream);
    }
}

// tiles of a launch, at most
long long max_tiles(const Fp8Params& p) {
    const int rows = tile_rows(p);
    return (((long long)p.rows + rows - 1) / rows + p.E) * (((p.input_grad ? p.K : p.N) + 255) / 256);
}

}  // namespace

// Tiles count in 31 bits.  The bound on the groups' columns is the documented one, of 512
// groups of 2^20 columns only; no launch is near a limit there (the grids are persistent, and
// the streamed form's tasks fewer than 2^28).
bool fp8_product_fits(const Fp8Params& p) {
    return (long long)p.E * ((p.N + 63) / 64) < (1LL << 23) && max_tiles(p) <= INT32_MAX - 4096;
}

hipError_t launch_quantize_rows(int dtype, const void* x, const int32_t* row_count, int rows, int cols, void* values,
                                float* scales, hipStream_t stream) {
    const long long units = (long long)rows * ((cols + kQBlock - 1) / kQBlock);
    const dim3 grid((unsigned)std::min<long long>((units + 15) / 16, 1 << 18)), block(256);
    if (dtype == 1)
        hipLaunchKernelGGL(quantize_rows_kernel<bf16_t>, grid, block, 0, stream, static_cast<const bf16_t*>(x), row_count,
                           rows, cols, static_cast<uint8_t*>(values), scales);
    else
        hipLaunchKernelGGL(quantize_rows_kernel<float>, grid, block, 0, stream, static_cast<const float*>(x), row_count,
                           rows, cols, static_cast<uint8_t*>(values), scales);
    return hipGetLastError();
}

hipError_t launch_quantize_weight(int dtype, const void* w, int E, int N, int K, void* values, float* scales,
                                  hipStream_t stream) {
    const long long blocks = (long long)E * ((N + kQBlock - 1) / kQBlock) * ((K + kQBlock - 1) / kQBlock);
    const dim3 grid((unsigned)std::min<long long>(blocks, 1 << 20)), block(256);
    if (dtype == 1)
        hipLaunchKernelGGL(quantize_weight_kernel<bf16_t>, grid, block, 0, stream, static_cast<const bf16_t*>(w), E, N, K,
                           static_cast<uint8_t*>(values), scales);
    else
        hipLaunchKernelGGL(quantize_weight_kernel<float>, grid, block, 0, stream, static_cast<const float*>(w), E, N, K,
                           static_cast<uint8_t*>(values), scales);
    return hipGetLastError();
}

hipError_t launch_fp8_product(const Fp8Params& p, hipStream_t stream) {
    Fp8Args a = fp8_args(p);
    if (fp8_streams(p)) {
        launch_stream(p, a, stream);
        return hipGetLastError();
    }
    a.tile_rows = tile_rows(p);
    const long long tiles = max_tiles(p);
    const int grid = ((int)std::min<long long>(tiles, device_cu_count()) + 7) / 8 * 8;
    if (p.input_grad) {
        if (p.out_bf16) launch_tiles<8, true, false>(a, grid, stream);
        else launch_tiles<4, true, true>(a, grid, stream);
    } else {
        if (p.out_bf16) launch_tiles<8, false, false>(a, grid, stream);
        else launch_tiles<4, false, true>(a, grid, stream);
    }
    return hipGetLastError();
}

}  // namespace inkling
