// y = act(x W^T + bias) + residual, for AMD Instinct MI355X (gfx950). C ABI declared in
// block/moe_block.h.
//
// Two shapes of the same product. Up to 32 rows of x it is a stream of W: a workgroup takes
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

// Eight neighbouring columns at once (col and n multiples of 8), with the bias and the residual
// there.
template <int DT>
__device__ __forceinline__ void finish8(const Args &a, int row, int col, float (&z)[8], const Raw8<DT> &bias,
                                        const Raw8<DT> &residual)
{
    float f[8];
    if (a.bias) {
        widen8<DT>(bias, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += f[i];
    }
    activate8(a.act, z);
    if (a.residual) {
        widen8<DT>(residual, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += f[i];
    }
    // past the caches, which the operands need (6720 x 7168 x 4096: 357 us against 377)
    __builtin_nontemporal_store(narrow8<DT>(z).v[0], reinterpret_cast<u32x4 *>(a.y + (int64_t)row * a.n + col));
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
template <int DT, int G, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void linear_few_kernel(Args a)
{
    __shared__ u32x4 shared[WAVES * kStage<1, G, false>];
    const int lane = lane_id(), wave = wave_in_block();
    const int c0 = blockIdx.x * 16;
    const int there = a.n - c0 < 16 ? a.n - c0 : 16;
    const uint32_t row_bytes = (uint32_t)a.k * 2u;
    const rsrc_t w[1] = {make_rsrc(a.w + (int64_t)c0 * a.k, (uint32_t)there * row_bytes)};
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.m * row_bytes);
    uint32_t col[2 * G];
    f32x4 acc[1][G];
    clear(acc);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int r = g * 16 + p * 8 + lane / 8;
            col[2 * g + p] = r < a.m ? (uint32_t)r * row_bytes + lane % 8 * 16 : kNowhere;
        }
    stream_products<DT, 1, G, false>(acc, w, row_bytes, x, col, a.k, wave * kLineK, WAVES * kLineK,
                                     shared + wave * kStage<1, G, false>);
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
// Many rows
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void shared_void;

// The largest divisor of n up to most.
constexpr int most_dividing(int n, int most)
{
    int d = most < n ? most : n;
    while (n % d)
        --d;
    return d;
}

// Waits for the wave's loads into shared memory and its reads of it, then for the workgroup.
// (Loads into shared memory count as loads from memory: a fence need not wait for them.)
// Nothing is moved across.
__device__ __forceinline__ void wait_and_sync()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
}

// Tiles of TM rows of x by TN rows of W, WM x WN waves, 64 k a step. Both operands go straight
// from memory to shared memory (no registers) into two buffers in turn. A row of a buffer is
// its eight 16-byte chunks of 64 k, a whole line; chunk c of row r lies at c ^ (r % 8), so that
// the 16 lanes whose reads of an operand go together fall into different banks. A load's
// lanes fill shared memory in order, so the exchange is made in the addresses they read.
// (Four buffers of 32 k reach further ahead but ask the cache for half lines: 9 TB/s of
// requests were the limit, 413 us for 6720 x 7168 x 4096 in tiles of 256 x 256 where this
// takes 385; with tiles of 224 x 256 and the epilogue's loads together 325 to 357: 1.2 PFLOP/s,
// 81% of the library's product alone. What bounds it now is shared memory, which the eight
// waves read three quarters of the time, and power: the clock falls to 1.8 GHz. Four waves of
// 112 x 128 read a third less, but one wave a SIMD hides less: no faster, even with loads of W
// two steps ahead.)
// Operands are read from shared memory half a step before their products, which leaves one
// barrier a step and no product waiting for a read.
//   parts > 1: the sums over one of `parts` ranges of k, to partial [parts][m][n] in fp32.
template <int DT, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void linear_tile_kernel(Args a, int tiles_m, int tiles_n, int parts,
                                                                   float *partial)
{
    constexpr int W = WM * WN, FM = TM / WM / 16, FN = TN / WN / 16;
    // half of the waves load x, half W: loads of a wave a step, of 8 rows each
    constexpr int kLoadsX = TM / 8 / (W / 2), kLoadsW = TN / 8 / (W / 2);
    static_assert(TM % (4 * W) == 0 && TN % (4 * W) == 0 && kLoadsX <= kLoadsW, "");
    constexpr int kBuffer = (TM + TN) * 8;  // 16-byte chunks
    // one object each: the compiler then knows that a load into one does not touch the other
    __shared__ u32x4 s0[kBuffer], s1[kBuffer];
    const int lane = lane_id(), wave = wave_in_block();

    // Workgroups go to the eight XCDs in turn; each XCD takes a run of tiles, in bands of
    // rows of x, so that its cache serves one band's x and W moving past it.
    const int tiles = tiles_m * tiles_n, all = tiles * parts;
    const int run = (all + 7) / 8, id = (int)blockIdx.x % 8 * run + (int)blockIdx.x / 8;
    if ((int)blockIdx.x / 8 >= run || id >= all)
        return;
    const int part = id / tiles, tile = id % tiles;
    constexpr int kBand = 4;
    const int band = tile / (kBand * tiles_n) * kBand, in_band = tile % (kBand * tiles_n);
    const int high = tiles_m - band < kBand ? tiles_m - band : kBand;
    const int r0 = (band + in_band % high) * TM, c0 = in_band / high * TN;

    const uint32_t row_bytes = (uint32_t)a.k * 2u;
    const int rows = a.m - r0 < TM ? a.m - r0 : TM, cols = a.n - c0 < TN ? a.n - c0 : TN;
    // a wave loads rows of x or rows of W (rows past the end read zeros)
    const bool loads_x = wave < W / 2;
    const int chunk = lane % 8 ^ lane / 8;
    const int group0 = loads_x ? wave * kLoadsX : TM / 8 + (wave - W / 2) * kLoadsW;
    const rsrc_t from = make_rsrc(loads_x ? a.x + (int64_t)r0 * a.k : a.w + (int64_t)c0 * a.k,
                                  (uint32_t)(loads_x ? rows : cols) * row_bytes);
    const uint32_t base = (uint32_t)((group0 - (loads_x ? 0 : TM / 8)) * 8 + lane / 8) * row_bytes + chunk * 16;

    const int steps = (a.k + kLineK - 1) / kLineK;
    const int first = (int)((int64_t)steps * part / parts), last = (int)((int64_t)steps * (part + 1) / parts);
    auto load = [&](u32x4 *to, int step) {
        const int k = step * kLineK;
        const uint32_t at = step < last && k + chunk * 8 < a.k ? base : kNowhere;  // past the last step: zeros
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) {
            const int g = i < kLoadsX || !loads_x ? i : kLoadsX - 1;  // rather twice than a branch
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (shared_void *)(to + (group0 + g) * 64), 16,
                                                     at + (uint32_t)g * 8u * row_bytes, k * 2, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
    const int wm = wave / WN * (TM / WM), wn = wave % WN * (TN / WN);
    const int i16 = lane % 16, q = lane / 16;
    struct Operands {
        u32x4 x[FM], w[FN];
    };
    auto read = [&](Operands &o, const u32x4 *from, int half) {
        const int c = (4 * half + q) ^ i16 % 8;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            o.w[j] = from[(TM + wn + j * 16 + i16) * 8 + c];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            o.x[i] = from[(wm + i * 16 + i16) * 8 + c];
    };
    auto multiply = [&](const Operands &o) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = mfma16<DT>(o.w[j], o.x[i], acc[i][j]);
        // order of issue: the reads of the next operands spread over the products
#pragma unroll
        for (int i = 0; i < FM + FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                    // a read of shared memory
            __builtin_amdgcn_sched_group_barrier(0x8, FM * FN / (FM + FN), 0);   // products
        }
    };
    Operands lo, hi;
    // One step, its first half's operands in lo. At the barrier everyone has read all of `now`,
    // which the loads of two steps ahead may then fill, and `after` has come.
    auto step = [&](u32x4 *now, const u32x4 *after, int t) {
        read(hi, now, 1);
        multiply(lo);
        wait_and_sync();
        load(now, t + 2);
        read(lo, after, 0);
        multiply(hi);
    };
    load(s0, first);
    load(s1, first + 1);
    wait_and_sync();
    read(lo, s0, 0);
    for (int t = first; t < last; t += 2) {  // a step past the last adds zeros
        step(s0, s1, t);
        step(s1, s0, t + 1);
    }
    // What a lane adds at the end, its rows of the residual all together: one after another in
    // the loop over rows, each a round trip to memory, they cost 20 us (348 against 328 for
    // 6720 x 7168 x 4096, two tiles a CU one after the other).
    constexpr int kLanes = FN * 2, kTogether = 64 / kLanes, kOuts = FM * 16 / kTogether;  // lanes a row of eights
    int late = lane;
    asm volatile("" : "+v"(late));  // computed here, not kept over the loop
    const int my_row = late / kLanes, my_col = late % kLanes * 8, col = c0 + wn + my_col;
    Raw8<DT> bias, residual[kOuts];
    if (a.bias && col < a.n)
        bias = load8<DT>(reinterpret_cast<const char *>(a.bias), col, a.n);
    if (a.residual && parts == 1) {
        const rsrc_t from_r = make_rsrc(a.residual + (int64_t)r0 * a.n, (uint32_t)rows * (uint32_t)a.n * 2u);
#pragma unroll
        for (int i = 0; i < kOuts; ++i) {
            const uint32_t row = wm + i * kTogether + my_row;  // rows past the end read zeros
            residual[i].v[0] = __builtin_amdgcn_raw_buffer_load_b128(
                from_r, col < a.n ? (row * (uint32_t)a.n + col) * 2u : kNowhere, 0, 0);
        }
    }
    wait_and_sync();  // the last loads, of nothing, also write shared memory
    // acc[i][j][e] is row wm + 16 i + lane % 16, column wn + 16 j + 4 (lane / 16) + e. Through
    // shared memory, kRows rows at a time, into rows of eight columns a lane.
    constexpr int kCols = FN * 16, kChunks = kCols / 4, kOwn = kBuffer * 2 / W;  // 16-byte chunks of a wave
    constexpr int kRows = 16 * most_dividing(FM, kOwn / kChunks / 16);
    u32x4 *const own = wave < W / 2 ? s0 + wave * kOwn : s1 + (wave - W / 2) * kOwn;
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += kRows / 16) {
#pragma unroll
        for (int i = 0; i < kRows / 16; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int row = i * 16 + i16;
                own[row * kChunks + (j * 4 + q ^ row % kChunks)] = __builtin_bit_cast(u32x4, acc[i0 + i][j]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int t = 0; t < kRows / kTogether; ++t) {
            const int r = t * kTogether + my_row, row = r0 + wm + i0 * 16 + r;
            float z[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 v = own[r * kChunks + (my_col / 4 + h ^ r % kChunks)];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[4 * h + e] = __uint_as_float(v[e]);
            }
            if (row >= a.m || col >= a.n)
                continue;
            if (parts > 1)
                store8<DT_F32>(reinterpret_cast<char *>(partial + ((int64_t)part * a.m + row) * a.n), col, a.n, z);
            else
                finish8<DT>(a, row, col, z, bias, residual[i0 * 16 / kTogether + t]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The parts' sums in order, then the epilogue. A lane takes eight neighbouring columns.
template <int DT>
__global__ __launch_bounds__(256) void linear_join_kernel(Args a, int parts, const float *partial)
{
    const int64_t all = (int64_t)a.m * a.n;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < all; i += (int64_t)gridDim.x * 2048) {
        float z[8] = {};
        for (int p = 0; p < parts; p += 2) {  // a power of two, at least 2; two loads at a time
            float f0[8], f1[8];
            widen8<DT_F32>(load8<DT_F32>(reinterpret_cast<const char *>(partial + p * all + i), 0, 8), f0);
            widen8<DT_F32>(load8<DT_F32>(reinterpret_cast<const char *>(partial + (p + 1) * all + i), 0, 8), f1);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = z[e] + f0[e] + f1[e];
        }
        const int row = (int)(i / a.n), col = (int)(i % a.n);
        Raw8<DT> bias, residual;
        if (a.bias)
            bias = load8<DT>(reinterpret_cast<const char *>(a.bias), col, a.n);
        if (a.residual)
            residual = load8<DT>(reinterpret_cast<const char *>(a.residual + i), 0, 8);
        finish8<DT>(a, row, col, z, bias, residual);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int kFewRows = 32;

bool good_sizes(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m <= (1 << 24) && n >= 8 && k >= 8 && n <= (1 << 20) && k <= (1 << 20) &&
           n * k <= ((int64_t)1 << 36) && m * n <= ((int64_t)1 << 36) && m * k <= ((int64_t)1 << 36);
}

// How a product of many rows is cut: tiles of rows x cols, and the parts of k.
struct Plan {
    int rows, cols;
    int parts;
};

int64_t tile_count(int64_t m, int64_t n, const Plan &p) { return ceil_div(m, p.rows) * ceil_div(n, p.cols); }

// The largest square tile that leaves work for most of the 256 CUs; of the largest ones, the
// height whose rounds over the CUs cost least (6720 x 4096: 432 tiles of 256 x 256 take two
// rounds and fill 84% of them, 480 of 224 x 256 94%). Tiles of 64 that are still too few for
// two workgroups a CU share their k.
Plan plan(int64_t m, int64_t n, int64_t k)
{
    Plan p = {256, 256, 1};
    while (p.rows > 64 && tile_count(m, n, p) < 192)
        p.rows = p.cols = p.rows / 2;
    if (p.rows == 256) {
        auto cost = [&](int rows) { return ceil_div(tile_count(m, n, {rows, 256, 1}), 256) * rows; };
        if (cost(224) < cost(p.rows))
            p.rows = 224;
        if (cost(192) < cost(p.rows))
            p.rows = 192;
    }
    const int64_t steps = ceil_div(k, kLineK), tiles = tile_count(m, n, p);
    while (p.rows == 64 && p.parts < 16 && tiles * p.parts * 2 <= 512 && p.parts * 16 < steps)
        p.parts *= 2;
    return p;
}

template <int DT, int TM, int TN, int WM, int WN>
block_status_t run_tiles(const Args &a, int parts, float *partial, hipStream_t st)
{
    const int tm = (int)ceil_div(a.m, TM), tn = (int)ceil_div(a.n, TN);
    const int64_t blocks = ceil_div((int64_t)tm * tn * parts, 8) * 8;
    return launch(linear_tile_kernel<DT, TM, TN, WM, WN>, dim3((unsigned)blocks), dim3(WM * WN * 64), 0, st, a, tm, tn,
                  parts, partial);
}

template <int DT>
block_status_t run(const Args &a, float *partial, hipStream_t st)
{
    if (a.m <= kFewRows) {
        const dim3 grid((unsigned)ceil_div(a.n, 16));
        if (a.m <= 16)
            return launch(linear_few_kernel<DT, 1, 16>, grid, dim3(1024), 0, st, a);
        return launch(linear_few_kernel<DT, 2, 8>, grid, dim3(512), 0, st, a);
    }
    const Plan p = plan(a.m, a.n, a.k);
    block_status_t s;
    if (p.rows == 256)
        s = run_tiles<DT, 256, 256, 2, 4>(a, p.parts, partial, st);
    else if (p.rows == 224)
        s = run_tiles<DT, 224, 256, 2, 4>(a, p.parts, partial, st);
    else if (p.rows == 192)
        s = run_tiles<DT, 192, 256, 2, 4>(a, p.parts, partial, st);
    else if (p.rows == 128)
        s = run_tiles<DT, 128, 128, 2, 2>(a, p.parts, partial, st);
    else
        s = run_tiles<DT, 64, 64, 2, 2>(a, p.parts, partial, st);
    if (s || p.parts == 1)
        return s;
    const int64_t blocks = ceil_div((int64_t)a.m * a.n, 2048);
    return launch(linear_join_kernel<DT>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a, p.parts,
                  partial);
}

}  // namespace

extern "C" {

int64_t block_linear_act_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!good_sizes(m, n, k) || m <= kFewRows)
        return 0;
    const Plan p = plan(m, n, k);
    return p.parts > 1 ? p.parts * m * n * 4 : 0;
}

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
    float *partial = static_cast<float *>(workspace);
    return dtype == BLOCK_BF16 ? run<DT_BF16>(a, partial, stream) : run<DT_F16>(a, partial, stream);
}

}  // extern "C"
