// y = act(x W^T + bias) + residual, for AMD Instinct MI355X (gfx950). C ABI declared in
// block/moe_block.h.
//
// Two shapes of the same product. Up to 64 rows of x it is a stream of W: a workgroup takes
// 16 rows of W, its waves split k, and their sums meet in LDS. More rows are tiled for the
// matrix cores with both operands staged through LDS. Bias, activation and residual are
// applied to the fp32 sums in registers, and each output is rounded once.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_host.h"
#include "weight_stream.h"

namespace {

using namespace block;

struct Args {
    const uint16_t *x, *w, *bias, *residual;
    uint16_t *y;
    int m, n, k, act;
};

template <int DT>
__device__ __forceinline__ void finish(const Args &a, int row, int col, float z)
{
    if (a.bias)
        z += load1<DT>(a.bias, col);
    z = activate(a.act, z);
    const int64_t at = (int64_t)row * a.n + col;
    if (a.residual)
        z += load1<DT>(a.residual, at);
    store1<DT>(a.y, at, z);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
template <int DT, int G, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void linear_few_kernel(Args a)
{
    __shared__ u32x4 shared[WAVES * kStage<1, G>];
    const int lane = lane_id(), wave = wave_in_block();
    const int c0 = blockIdx.x * 16;
    constexpr int DEPTH = G == 4 ? 2 : 3;
    const int there = a.n - c0 < 16 ? a.n - c0 : 16;
    const uint32_t row_bytes = (uint32_t)a.k * 2u;
    const rsrc_t w[1] = {make_rsrc(a.w + (int64_t)c0 * a.k, (uint32_t)there * row_bytes)};
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.m * row_bytes);
    uint32_t col[G][2];
    f32x4 acc[1][G];
    clear(acc);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int r = g * 16 + p * 8 + lane / 8;
            col[g][p] = r < a.m ? (uint32_t)r * row_bytes + lane % 8 * 16 : kNowhere;
        }
    stream_products<DT, 1, G, DEPTH, 1>(acc, w, row_bytes, x, col, a.k, wave * kLineK, WAVES * kLineK,
                                        shared + wave * kStage<1, G>);
    __syncthreads();  // the sums take the place of the stages
    f32x4 *joined = reinterpret_cast<f32x4 *>(shared);
#pragma unroll
    for (int g = 0; g < G; ++g)
        joined[(wave * G + g) * 64 + lane] = acc[0][g];
    __syncthreads();
    for (int i = threadIdx.x; i < G * 256; i += WAVES * 64) {
        const int c = i % 16, row = i / 16, g = row / 16;  // c: row of W, within the tile
        const int from = c / 4 * 16 + row % 16;            // the lane that holds it, in element c % 4
        float z = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q)
            z += joined[(q * G + g) * 64 + from][c % 4];
        if (row < a.m && c0 + c < a.n)
            finish<DT>(a, row, c0 + c, z);
    }
}

// ---------------------------------------------------------------------------
// Many rows: 128 x 128 tiles, 64 k a step; four waves of 64 x 64
// ---------------------------------------------------------------------------
constexpr int kTile = 128, kTileK = 64;

template <int DT>
__global__ __launch_bounds__(256) void linear_tile_kernel(Args a)
{
    // rows of eight 16-byte chunks; chunk c of row r lies at c ^ (r % 8), so that the 16 rows
    // a matrix operand reads at one k fall into different banks
    __shared__ u32x4 sx[kTile * 8], sw[kTile * 8];
    const int lane = lane_id(), wave = wave_in_block(), tid = threadIdx.x;
    const int wide = (a.n + kTile - 1) / kTile;
    const int r0 = (int)blockIdx.x / wide * kTile, c0 = (int)blockIdx.x % wide * kTile;
    u32x4 px[4], pw[4];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 32 + tid / 8, k = k0 + tid % 8 * 8;
            const bool in = k < a.k;
            const int xr = r0 + row < a.m ? r0 + row : a.m - 1, wr = c0 + row < a.n ? c0 + row : a.n - 1;
            const u32x4 vx = *reinterpret_cast<const u32x4 *>(a.x + (int64_t)xr * a.k + (in ? k : 0));
            const u32x4 vw = *reinterpret_cast<const u32x4 *>(a.w + (int64_t)wr * a.k + (in ? k : 0));
            px[i] = in ? vx : u32x4{0, 0, 0, 0};
            pw[i] = in ? vw : u32x4{0, 0, 0, 0};
        }
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
    const int wx = wave / 2 * 64, ww = wave % 2 * 64;
    fetch(0);
    for (int k0 = 0; k0 < a.k; k0 += kTileK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 32 + tid / 8, slot = row * 8 + (tid % 8 ^ row % 8);
            sx[slot] = px[i];
            sw[slot] = pw[i];
        }
        __syncthreads();
        if (k0 + kTileK < a.k)
            fetch(k0 + kTileK);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c = u * 4 + lane / 16;
            u32x4 ax[4], aw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rx = wx + i * 16 + lane % 16, rw = ww + i * 16 + lane % 16;
                ax[i] = sx[rx * 8 + (c ^ rx % 8)];
                aw[i] = sw[rw * 8 + (c ^ rw % 8)];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = mfma16<DT>(aw[j], ax[i], acc[i][j]);
        }
    }
    // acc[i][j][q]: row wx + 16 i + lane % 16, column ww + 16 j + 4 (lane / 16) + q
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = r0 + wx + i * 16 + lane % 16;
        if (row >= a.m)
            continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = c0 + ww + j * 16 + lane / 16 * 4 + q;
                if (col < a.n)
                    finish<DT>(a, row, col, acc[i][j][q]);
            }
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool good_sizes(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m <= (1 << 24) && n >= 8 && k >= 8 && n <= (1 << 20) && k <= (1 << 20) &&
           n * k <= ((int64_t)1 << 36) && m * n <= ((int64_t)1 << 36) && m * k <= ((int64_t)1 << 36);
}

template <int DT>
block_status_t run(const Args &a, hipStream_t st)
{
    if (a.m <= 64) {
        const dim3 grid((unsigned)ceil_div(a.n, 16));
        if (a.m <= 16)
            return launch(linear_few_kernel<DT, 1, 16>, grid, dim3(1024), 0, st, a);
        if (a.m <= 32)
            return launch(linear_few_kernel<DT, 2, 8>, grid, dim3(512), 0, st, a);
        return launch(linear_few_kernel<DT, 4, 8>, grid, dim3(512), 0, st, a);
    }
    const dim3 grid((unsigned)(ceil_div(a.n, kTile) * ceil_div(a.m, kTile)));
    return launch(linear_tile_kernel<DT>, grid, dim3(256), 0, st, a);
}

}  // namespace

extern "C" {

int64_t block_linear_act_workspace(int64_t, int64_t, int64_t) { return 0; }

block_status_t block_linear_act(const void *x, const void *weight, const void *bias, const void *residual, void *y,
                                int64_t m, int64_t n, int64_t k, block_act_t act, block_dtype_t dtype, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream)
{
    if (!good_sizes(m, n, k) || act < BLOCK_ACT_NONE || act > BLOCK_ACT_SQUARED_RELU ||
        (dtype != BLOCK_BF16 && dtype != BLOCK_FP16))
        return BLOCK_ERR_INVALID_ARG;
    if (n % 8 || k % 8)
        return BLOCK_ERR_ALIGNMENT;
    if (m == 0)
        return BLOCK_OK;
    const int64_t need = block_linear_act_workspace(m, n, k);
    if (!x || !weight || !y || (need > 0 && (!workspace || workspace_bytes < need)))
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(weight, 16) || misaligned(bias, 16) || misaligned(residual, 16) ||
        misaligned(y, 16) || (need > 0 && misaligned(workspace, 16)))
        return BLOCK_ERR_ALIGNMENT;
    if (any_overlap<2, 4>({{y, m * n * 2}, {workspace, need}},
                          {{x, m * k * 2}, {weight, n * k * 2}, {bias, n * 2}, {residual, m * n * 2}}))
        return BLOCK_ERR_INVALID_ARG;
    Args a = {};
    a.x = static_cast<const uint16_t *>(x), a.w = static_cast<const uint16_t *>(weight);
    a.bias = static_cast<const uint16_t *>(bias), a.residual = static_cast<const uint16_t *>(residual);
    a.y = static_cast<uint16_t *>(y), a.m = (int)m, a.n = (int)n, a.k = (int)k, a.act = act;
    return dtype == BLOCK_BF16 ? run<DT_BF16>(a, stream) : run<DT_F16>(a, stream);
}

}  // extern "C"
