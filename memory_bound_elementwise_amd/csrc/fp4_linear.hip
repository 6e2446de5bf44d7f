// y = act(x W^T + bias) + residual with W in 4 bits (layout in fp4.h), for AMD Instinct MI355X
// (gfx950). C ABI declared in block/moe_block.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp4_host.h"
#include "fp4_stream.h"

namespace {

using namespace block;

struct Args {
    const uint16_t *x;
    const uint8_t *codes, *scales;
    const uint16_t *bias, *residual;
    uint16_t *y;
    int m, n, k, act;
};

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// Up to 16 rows of x: the cost is reading W once. A workgroup takes 16 rows of W, its waves split k,
// and their sums meet in shared memory. 16 waves, so that 7168 x 4096, a workgroup a CU, has all
// its loads in flight at once.
constexpr int kWaves = 16;

template <int NX, int D>
__global__ __launch_bounds__(kWaves * 64) void fp4_linear_few_kernel(Args a)
{
    __shared__ u32x4 shared[kWaves * NX * 64];  // the waves' stages, then their sums
    const int lane = lane_id(), wave = wave_in_block(), k_tiles = (a.k + kFp4K - 1) / kFp4K;
    const Tiles w[1] = {tiles_of(a.codes, a.scales, blockIdx.x, k_tiles)};
    Stream<1, NX, D> stream;
    stream.start(w, wave, kWaves);
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.m * (uint32_t)a.k * 2u);
    uint32_t col[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int row = 4 * i + lane / 16;
        col[i] = row < a.m ? (uint32_t)row * (uint32_t)a.k * 2u + lane % 16 * 16 : kNowhere;
    }
    f32x4 acc[1] = {};
    stream.run(acc, w, x, col, a.k, wave, kWaves, shared + wave * NX * 64);
    __syncthreads();
    f32x4 *joined = reinterpret_cast<f32x4 *>(shared);
    joined[wave * 64 + lane] = acc[0];
    __syncthreads();
    if (threadIdx.x >= 256)
        return;
    const int c = threadIdx.x % 16, row = threadIdx.x / 16, col_n = blockIdx.x * 16 + c;
    if (row >= a.m || col_n >= a.n)
        return;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)  // row c of W's tile is element c % 4 of lane 16 (c / 4) + its column
        z += joined[i * 64 + c / 4 * 16 + row][c % 4];
    if (a.bias)
        z += load1<DT_BF16>(a.bias, col_n);
    z = activate(a.act, z);
    const int64_t at = (int64_t)row * a.n + col_n;
    if (a.residual)
        z += load1<DT_BF16>(a.residual, at);
    store1<DT_BF16>(a.y, at, z);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;

bool good_sizes(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m <= (1 << 24) && n >= 8 && k >= 32 && n <= (1 << 20) && k <= (1 << 20) &&
           n * k <= ((int64_t)1 << 36) && m * n <= ((int64_t)1 << 36) && m * k <= ((int64_t)1 << 36);
}

}  // namespace

extern "C" {

int64_t block_linear_act_fp4_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!good_sizes(m, n, k) || k % 32 || n % 8 || m <= kFewRows)
        return 0;
    return round_up(n * k * 2, 16) + block_linear_act_workspace(m, n, k);
}

block_status_t block_linear_act_fp4(const uint16_t *x, const uint8_t *codes, const uint8_t *scales, const uint16_t *bias,
                                    const uint16_t *residual, uint16_t *y, int64_t m, int64_t n, int64_t k,
                                    block_act_t act, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (!good_sizes(m, n, k) || act < BLOCK_ACT_NONE || act > BLOCK_ACT_SQUARED_RELU)
        return BLOCK_ERR_INVALID_ARG;
    if (n % 8 || k % 32)
        return BLOCK_ERR_ALIGNMENT;
    if (m == 0)
        return BLOCK_OK;
    const int64_t need = block_linear_act_fp4_workspace(m, n, k);
    if (!x || !codes || !scales || !y || (need > 0 && (!workspace || workspace_bytes < need)))
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(codes, 16) || misaligned(scales, 16) || misaligned(bias, 16) ||
        misaligned(residual, 16) || misaligned(y, 16) || (need > 0 && misaligned(workspace, 16)))
        return BLOCK_ERR_ALIGNMENT;
    const Fp4Shape s = {1, n, k};
    if (any_overlap<2, 5>({{y, m * n * 2}, {workspace, need}},
                          {{x, m * k * 2}, {codes, s.codes()}, {scales, s.scales()}, {bias, n * 2}, {residual, m * n * 2}}))
        return BLOCK_ERR_INVALID_ARG;
    if (m > kFewRows) {  // the weights' bf16 values, then the product with those
        const int64_t wide = round_up(n * k * 2, 16);
        uint16_t *weight = static_cast<uint16_t *>(workspace);
        if (const block_status_t r = block_fp4_dequantize(codes, scales, weight, 1, n, k, stream))
            return r;
        return block_linear_act(x, weight, bias, residual, y, m, n, k, act, BLOCK_BF16,
                                static_cast<char *>(workspace) + wide, need - wide, stream);
    }
    const Args a = {x, codes, scales, bias, residual, y, (int)m, (int)n, (int)k, act};
    const dim3 grid((unsigned)s.row_tiles()), threads(kWaves * 64);
    return m <= 4 ? launch(fp4_linear_few_kernel<1, 4>, grid, threads, 0, stream, a)
                  : launch(fp4_linear_few_kernel<4, 2>, grid, threads, 0, stream, a);
}

}  // extern "C"
