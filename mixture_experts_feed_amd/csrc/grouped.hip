// Products grouped by expert with ragged row counts, reached on their own:
//   out[r] = W_e x[row_index[r]]   dx[r] = W_e^T dout[r]   dW_e = sum_r dout[r] (x) x[row_index[r]]
// for the rows offsets[e] <= r < offsets[e + 1] of expert e.  Two kernels:
//   small_product_kernel (grouped_small.h)  64 x 64 tiles, one launch without a
//     plan: fp32, and bf16 products with too few large tiles for the card or few
//     rows an expert against small weights (group_small, group_small_wgrad);
//   moe_gemm_kernel (gemm_kernel.h)  the layer's tiles, in its grouped modes:
//     everything else, after a plan (the caller's offsets made safe, row tiles).
#include <algorithm>

#include "common.h"
#include "gemm_kernel.h"
#include "grouped_small.h"
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

// Tile configurations (see gemm.hip for what they measured in the layer):
// 0: 256 output columns x 256 rows; 1: 128 x 16, weights streamed.
int tile_rows(int cfg) { return cfg == 0 ? 256 : 16; }
int tile_cols(int cfg) { return cfg == 0 ? 256 : 128; }

int grid_of(long long tiles, int per_cu) {
    const int grid = (int)std::min<long long>(tiles, (long long)device_cu_count() * per_cu);
    return (grid + 7) / 8 * 8;
}

// Forward and input gradient on 256 x 256 tiles, one workgroup a CU: bound by the
// matrix units once an expert has some hundred rows (each stage of 64 K moves 64 KB
// through LDS for 8.4 MFLOP), less what the last row tile of an expert lacks.
// Forward, 128 experts of 512 rows each, 6144 x 4096: 2934 us, 1.12 PFLOP/s; of 316
// to 754 rows, whose tiles hold 1.23 times the rows: 3392 us, 0.97 PFLOP/s.  Input
// gradient, 64 experts of 27 to 1200 rows (384 on average), 2048 columns from 1536:
// 205 us, 0.75 PFLOP/s (128 row tiles, a quarter of their rows empty, by 8 column
// tiles: four rounds).  128 x 256 and 256 x 128 tiles, two workgroups a CU, were 5 to
// 30% slower at 1.2 to 24 rounds, and one wave a SIMD with 128 x 128 tiles of its own
// 0 to 10% faster on even experts only.
// kSchedGroup (gemm_kernel.h) starts the tiles that share rows or weights on one
// XCD together: 1 to 25% faster than the other walks.
template <int SCHED, int MODE>
void launch_256(const GemmKArgs& a, long long max_tiles, hipStream_t stream) {
    hipLaunchKernelGGL((moe_gemm_kernel<bf16_t, 256, 256, 4, 2, 2, 2, 128, 8, SCHED, MODE>),
                       dim3(grid_of(max_tiles, 1)), dim3(512), 0, stream, a);
}

}  // namespace

// Up to 48 rows an expert on average, the forward streams the weights past tiles
// of 16 rows (the layer's decode tiles): 805 us at 2 rows an expert, 6144 x 4096,
// 6.9 TB/s.  The host knows the average only: where one expert of 128 holds all of
// 6000 rows, its weights stream past 375 tiles, 1588 us, and the same rows given as
// one expert take 305 (46 rows in each: 2421).  Input gradients always take 256 x 256
// tiles (whose few-row form skips the row blocks without rows): 407 us at 64 rows,
// 4096 x 2048, 5.4 TB/s.
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

// The row products (forward, input gradient) on 64 x 64 tiles:
// - below one 256 x 256 tile a CU.  Forward, us, 64 x 64 against the large tiles: 7 /
//   11 at 12 experts of 30 rows (512 x 512), 25 / 36 at 16 of 256 rows (1024 x 1024, 128
//   large tiles), 43 / 40 at 16 of 512 (192); forward and input gradient 41, 40 / 39, 56
//   at 8 of 512 (2048 x 1024, 192);
// - with at most 64 rows an expert while the weights are at most 2^27 values (beyond,
//   streaming them past 16-row tiles wins).  Forward and input gradient: 32, 32 / 50, 38
//   at 64 experts of 40 rows (1024 x 1024), 16, 17 / 17, 28 at 128 of 2 (512 x 512), 48,
//   47 / 46, 57 at 128 of 2 (1024 x 1024), 65, 71 / 64, 66 at 128 of 64 (1024 x 1024);
//   209, 209 / 156, 206 at 128 of 2 (2048 x 2048, 2^29 values);
// - fp32 at every size: 11 / 34 us at 8 experts of 83 rows (136 x 200), 50 / 84 at 32
//   of 64 (1024 x 1024).  At 16 of 512 (2048 x 2048), even or not: 594 to 654 (105 to
//   116 TFLOP/s; input gradient 585 to 615, weight gradient 622 to 639), where the large
//   tiles, whose fp32 form is gone, took 594.
bool group_small(int dtype, int rows, int E, int n_cols, int k_len) {
    if (dtype == 0) return true;
    if (rows <= 64LL * E && (double)E * n_cols * k_len <= (double)(1 << 27)) return true;
    return group_max_row_tiles(rows, E, 0) * ((n_cols + 255) / 256) < 256;
}

// The weight gradients on 64 x 64 tiles: up to 256 rows an expert and 24 M
// values.  bf16, us, against 128 x 256 tiles: 22 / 28 at 64 experts of 100 rows (512 x
// 512), 18 / 26 at 16 of 64 and 32 / 31 at 16 of 256 (1024 x 1024), 22 / 28 at 40 of 3
// (1024 x 512); 46 / 36 at 16 of 512 (1024 x 1024), 38 / 35 at 32 of 128 (1024 x 1024,
// 34 M values), 52 / 39 at 12 of 30 (2048 x 2048, 50 M).  fp32 at every size, as above.
bool group_small_wgrad(int dtype, int rows, int E, int n_in, int n_out) {
    if (dtype == 0) return true;
    return rows <= 256LL * E && (double)E * n_in * n_out <= 24e6;
}

long long group_small_tiles(int rows, int E, int n_cols) {
    return (((long long)rows + 63) / 64 + E) * ((n_cols + 63) / 64);
}

hipError_t launch_group_small(const GroupParams& p, const int32_t* offsets, hipStream_t stream) {
    SmallArgs a = {};
    a.A = p.weight;
    a.B = p.src;
    a.offsets = offsets;
    a.row_index = p.row_index;
    a.src_rows = p.src_rows;
    a.rows = p.rows;
    a.E = p.E;
    a.K = p.k_len;
    a.N = p.n_cols;
    a.ntn = (p.n_cols + 63) / 64;
    a.out = p.out;
    a.out_bf16 = p.out_bf16;
    const dim3 grid((unsigned)group_small_tiles(p.rows, p.E, p.n_cols)), block(256);
    if (p.dtype == 1) {
        if (p.input_grad) hipLaunchKernelGGL((small_product_kernel<bf16_t, kProdDx>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((small_product_kernel<bf16_t, kProdRows>), grid, block, 0, stream, a);
    } else {
        if (p.input_grad) hipLaunchKernelGGL((small_product_kernel<float, kProdDx>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((small_product_kernel<float, kProdRows>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_group_small_wgrad(const GroupParams& p, const int32_t* offsets, const void* x, const void* dout,
                                    int n_in, int n_out, void* dw, hipStream_t stream) {
    SmallArgs a = {};
    a.A = x;
    a.B = dout;
    a.offsets = offsets;
    a.row_index = p.row_index;
    a.src_rows = p.src_rows;
    a.rows = p.rows;
    a.E = p.E;
    a.N = n_in;
    a.M = n_out;
    a.ntn = (n_in + 63) / 64;
    a.ntm = (n_out + 63) / 64;
    a.out = dw;
    a.out_bf16 = p.out_bf16;
    const dim3 grid((unsigned)((long long)p.E * a.ntm * a.ntn)), block(256);
    if (p.dtype == 1) hipLaunchKernelGGL((small_product_kernel<bf16_t, kProdWgrad>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((small_product_kernel<float, kProdWgrad>), grid, block, 0, stream, a);
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
    a.ntn_r = (p.n_cols + tile_cols(p.cfg) - 1) / tile_cols(p.cfg);
    a.has_routed = 1;
    a.lda_r = p.n_cols;   // input gradient: the weights as K rows of n_cols
    const long long tiles = group_max_tiles(p);
    if (p.cfg != 0)
        hipLaunchKernelGGL((moe_gemm_kernel<bf16_t, 128, 16, 8, 1, 4, 4, 128, 1, kSchedStride, kModeGroup>),
                           dim3(grid_of(tiles, 1)), dim3(512), 0, stream, a);
    else if (p.input_grad) launch_256<kSchedGroup, kModeGroupDx>(a, tiles, stream);
    else launch_256<kSchedGroup, kModeGroup>(a, tiles, stream);
    return hipGetLastError();
}

// Weight gradients on 128 x 256 tiles, two workgroups a CU: tiles with a K of a
// few hundred rows are mostly stores (dW is written once, 1536 x 2048 x 4 bytes an
// expert against 384 rows read), and one workgroup stores while the other multiplies.
// 64 experts of 384 rows (2048 x 1536): 261 us in fp32 (1.0 GB, 3.8 TB/s), with
// gathered rows of x or without; 16 of 512 (2048 x 6144), bf16: 240 us, 0.86 PFLOP/s.
hipError_t launch_group_wgrad(const GroupParams& p, const void* x, const void* dout, int n_in, int n_out, void* dw,
                              int dw_bf16, hipStream_t stream) {
    GemmKArgs a = {};
    a.round_counter = p.counters;
    a.offsets = p.offs;
    a.poff = p.offs;      // tile costs by row count
    a.row_token = p.row_index;
    a.T = p.src_rows;
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
    hipLaunchKernelGGL((moe_gemm_kernel<bf16_t, 128, 256, 2, 2, 2, 2, 64, 4, kSchedQueue, kModeGroupWgrad>),
                       dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace inkling
