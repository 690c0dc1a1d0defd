// Products grouped by expert with ragged row counts, reached on their own:
//   out[r] = W_e x[row_index[r]]   dx[r] = W_e^T dout[r]   dW_e = sum_r dout[r] (x) x[row_index[r]]
// for the rows offsets[e] <= r < offsets[e + 1] of expert e.  The matrix work is
// moe_gemm_kernel (gemm_kernel.h) in its three grouped modes; here are the plan
// that turns the caller's offsets into row tiles, and the launches.
#include <algorithm>

#include "common.h"
#include "gemm_kernel.h"
#include "kernels.h"

namespace inkling {

namespace {

constexpr int kMaxGroups = 512;

// One workgroup.  offs[0..E] = the caller's offsets made safe to index rows
// with: clamped to [0, rows] and non-decreasing (each at least every one before
// it); tiles of bm rows in expert order (bm 0: none); the tile counters zeroed.
__global__ __launch_bounds__(kMaxGroups) void group_plan_kernel(const int32_t* __restrict__ offsets, int E, int rows,
                                                                int bm, int32_t* __restrict__ offs,
                                                                RoutedTile* __restrict__ tiles,
                                                                int32_t* __restrict__ num_tiles,
                                                                int32_t* __restrict__ counters) {
    __shared__ int32_t wave_max[kMaxGroups / kWave], wave_sum[kMaxGroups / kWave];
    __shared__ int32_t first[kMaxGroups + 1];   // first tile of each expert
    const int t = threadIdx.x, lane = lane_id(), wv = t >> 6;
    if (t < kRoundCounters) counters[t] = 0;
    // end of expert t: the running maximum of offsets[0 .. t + 1]
    const int start = max(0, min(offsets[0], rows));
    int end = t < E ? max(0, min(offsets[t + 1], rows)) : 0;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(end, d);
        if (lane >= d) end = max(end, o);
    }
    if (lane == kWave - 1) wave_max[wv] = end;
    __syncthreads();
    end = max(end, start);
    for (int w = 0; w < wv; ++w) end = max(end, wave_max[w]);
    // begin of expert t: the end of the one before
    int begin = __shfl_up(end, 1);
    if (lane == 0) {
        begin = start;
        for (int w = 0; w < wv; ++w) begin = max(begin, wave_max[w]);
    }
    if (t < E) offs[t + 1] = end;
    if (t == 0) offs[0] = start;
    if (bm == 0) return;   // uniform over the workgroup
    const int n = t < E ? (end - begin + bm - 1) / bm : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) wave_sum[wv] = incl;
    __syncthreads();
    for (int w = 0; w < wv; ++w) incl += wave_sum[w];
    if (t < E) first[t + 1] = incl;
    if (t == 0) first[0] = 0;
    __syncthreads();
    const int total = first[E];
    if (t == 0) *num_tiles = total;
    // one thread per tile: the last expert whose first tile is not after it
    for (int j = t; j < total; j += kMaxGroups) {
        int lo = 0, hi = E - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= j) lo = mid;
            else hi = mid - 1;
        }
        tiles[j] = RoutedTile{lo, (j - first[lo]) * bm};
    }
}

// out[r] = src[row_index[r]] for offs[0] <= r < offs[E] (an index out of range
// takes the nearest row in it): rows of D elements, D a multiple of 8.
template <typename TE>
__global__ __launch_bounds__(256) void group_gather_kernel(const TE* __restrict__ src, int src_rows,
                                                           const int32_t* __restrict__ row_index,
                                                           const int32_t* __restrict__ offs, int E, int D,
                                                           TE* __restrict__ out) {
    constexpr int V = 16 / sizeof(TE);
    const int nv = D / V;
    for (int r = offs[0] + blockIdx.x; r < offs[E]; r += gridDim.x) {
        const size_t row = (size_t)max(0, min(row_index[r], src_rows - 1));
        const uint4* s = reinterpret_cast<const uint4*>(src + row * D);
        uint4* o = reinterpret_cast<uint4*>(out + (size_t)r * D);
        for (int v = threadIdx.x; v < nv; v += 256) o[v] = s[v];
    }
}

// Tile configurations (see gemm.hip for what they measured in the layer):
// 0: 256 output columns x 256 rows; 1: 128 x 16, weights streamed.
int tile_rows(int cfg) { return cfg == 0 ? 256 : 16; }
int tile_cols(int cfg) { return cfg == 0 ? 256 : 128; }

int grid_of(long long tiles, int per_cu) {
    const int grid = (int)std::min<long long>(tiles, (long long)device_cu_count() * per_cu);
    return (grid + 7) / 8 * 8;
}

template <typename TE, int MODE>
hipError_t launch_rows(int cfg, const GemmKArgs& a, long long max_tiles, hipStream_t stream) {
    if (cfg == 0)
        hipLaunchKernelGGL((moe_gemm_kernel<TE, 256, 256, 4, 2, 2, 2, 128, 8, kSchedGroup, MODE>),
                           dim3(grid_of(max_tiles, 1)), dim3(512), 0, stream, a);
    else if constexpr (MODE == kModeGroup)
        hipLaunchKernelGGL((moe_gemm_kernel<TE, 128, 16, 8, 1, 4, 4, 128, 1, kSchedStride, MODE>),
                           dim3(grid_of(max_tiles, 1)), dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int group_cfg(int rows, int E, bool input_grad) {
    return !input_grad && (double)rows / E <= 48.0 ? 1 : 0;
}

long long group_max_row_tiles(int rows, int E, int cfg) {
    const int bm = tile_rows(cfg);
    return ((long long)rows + bm - 1) / bm + E;
}

long long group_max_tiles(const GroupParams& p) {
    return group_max_row_tiles(p.rows, p.E, p.cfg) * ((p.n_cols + tile_cols(p.cfg) - 1) / tile_cols(p.cfg));
}

hipError_t launch_group_plan(const GroupParams& p, const int32_t* offsets, bool tiles, hipStream_t stream) {
    hipLaunchKernelGGL(group_plan_kernel, dim3(1), dim3(kMaxGroups), 0, stream, offsets, p.E, p.rows,
                       tiles ? tile_rows(p.cfg) : 0, p.offs, p.tiles, p.num_tiles, p.counters);
    return hipGetLastError();
}

hipError_t launch_group_rows(const GroupParams& p, hipStream_t stream) {
    GemmKArgs a = {};
    a.round_counter = p.counters;
    a.tiles = p.tiles;
    a.num_tiles = p.num_tiles;
    a.offsets = p.offs;
    a.row_token = p.row_index;
    a.T = p.src_rows;
    a.A_routed = p.weight;
    a.B_routed = p.src;
    a.out_routed = p.out;
    a.out_final_bf16 = p.out_bf16;
    a.K_r = p.k_len;
    a.N_r = p.n_cols;
    a.lda_r = p.n_cols;   // input gradient: the weights as K rows of n_cols
    a.ntn_r = (p.n_cols + tile_cols(p.cfg) - 1) / tile_cols(p.cfg);
    a.has_routed = 1;
    const long long tiles = group_max_tiles(p);
    if (p.input_grad)
        return p.dtype == 1 ? launch_rows<bf16_t, kModeGroupDx>(p.cfg, a, tiles, stream)
                            : launch_rows<float, kModeGroupDx>(p.cfg, a, tiles, stream);
    return p.dtype == 1 ? launch_rows<bf16_t, kModeGroup>(p.cfg, a, tiles, stream)
                        : launch_rows<float, kModeGroup>(p.cfg, a, tiles, stream);
}

hipError_t launch_group_gather(int dtype, const void* src, int src_rows, const int32_t* row_index,
                               const int32_t* offs, int E, int rows, int D, void* out, hipStream_t stream) {
    const int blocks = std::min(rows, 4096);
    if (dtype == 1)
        hipLaunchKernelGGL(group_gather_kernel<bf16_t>, dim3(blocks), dim3(256), 0, stream,
                           static_cast<const bf16_t*>(src), src_rows, row_index, offs, E, D, static_cast<bf16_t*>(out));
    else
        hipLaunchKernelGGL(group_gather_kernel<float>, dim3(blocks), dim3(256), 0, stream,
                           static_cast<const float*>(src), src_rows, row_index, offs, E, D, static_cast<float*>(out));
    return hipGetLastError();
}

hipError_t launch_group_wgrad(const GroupParams& p, const void* x, const void* dout, int n_in, int n_out, void* dw,
                              int dw_bf16, hipStream_t stream) {
    GemmKArgs a = {};
    a.round_counter = p.counters;
    a.offsets = p.offs;
    a.poff = p.offs;      // tile costs by row count
    a.A_routed = x;
    a.B_routed = dout;
    a.lda_r = n_in;
    a.ldb_r = n_out;
    a.K_r = 1;
    a.wg_E = p.E;
    a.wg_M = n_out;
    a.wg_N = n_in;
    a.wg_mtiles = (n_out + 255) / 256;
    a.wg_ntiles = (n_in + 127) / 128;
    a.w_out_routed = dw;
    a.w_out_bf16 = dw_bf16;
    const int grid = grid_of((long long)p.E * a.wg_mtiles * a.wg_ntiles, 2);
    if (p.dtype == 1)
        hipLaunchKernelGGL((moe_gemm_kernel<bf16_t, 128, 256, 2, 2, 2, 2, 64, 4, kSchedQueue, kModeGroupWgrad>),
                           dim3(grid), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((moe_gemm_kernel<float, 128, 256, 2, 2, 2, 2, 64, 4, kSchedQueue, kModeGroupWgrad>),
                           dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace inkling
