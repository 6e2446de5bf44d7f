// y = act(x W^T + bias) + residual with W in 4 bits (layout in fp4.h), for AMD Instinct MI355X
// (gfx950). C ABI declared in block/moe_block.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp4_host.h"
#include "fp4_stream.h"
#include "linear_tiles.h"

namespace {

using namespace block;

struct Args : LinearArgs {
    const uint8_t *codes, *scales;
};

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// Up to 16 rows of x and W not too wide (few_rows below): the cost is reading W once. A workgroup
// takes 16 rows of W, its waves split k, and their sums meet in shared memory. 16 waves, so that 7168 x
// 4096, a workgroup a CU, has all its loads in flight at once: one row 5.5 us for 15.6 MB, which is
// mostly the start and the end of that one round. Up to four rows are one load a step and leave room
// for four steps in flight, more are four (4 rows 6.9 and 8.2 us, 2 rows 6.2 and 10.2).
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
    finish<DT_BF16>(a, row, col_n, z);
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
// Tiles of 16 FM rows of x by 64 FN rows of W, four waves, 128 k a step. x goes straight from memory
// to shared memory into two buffers in turn, as chunks of 16 bytes, chunk c of row r at c ^ (r % 8)
// (a load's lanes fill shared memory in order, so the exchange is made in the addresses they
// read). W needs no shared memory: each wave has 16 FN rows of it for itself, loads their tiles a
// step ahead and widens a word of each when its turn comes. What is read from shared memory is so
// 1 / FN of an operand a matrix instruction. (Three buffers and loads two steps ahead leave room
// for fewer workgroups: 1009 x 1408 x 7168 26.6 -> 29.5 us, 6720 x 4096 x 7168 323 -> 371. Tiles of 128
// x 256, a wave a SIMD: 33.8 and 340. Two waves a workgroup: 27.4 and 470.) Weights come from cache for
// all tiles but the first. 6720 x 4096 x 7168 takes 298 to 327 us in different sessions, 1.32 to 1.21
// PFLOP/s; the 896 tiles of 1009 x 1408 x 7168 24.8, 0.82, of 11 steps each and no whole number a CU.
//   parts > 1: the sums over one of `parts` ranges of k, to partial [parts][m][n] in fp32.
constexpr int kTileWaves = 4;

template <int FM, int FN>
__global__ __launch_bounds__(kTileWaves * 64, FN == 4 ? 3 : 4) void fp4_linear_tile_kernel(Args a, int tiles_m, int tiles_n,
                                                                                              int parts, float *partial)
{
    constexpr int W = kTileWaves, TM = FM * 16, TN = W * FN * 16, kLoads = TM / 4 / W;
    static_assert(kLoads % 2 == 0, "");
    // one object each: the compiler then knows that a load into one does not touch the other
    __shared__ u32x4 s0[TM * 16], s1[TM * 16];
    const int lane = lane_id(), wave = wave_in_block(), i16 = lane % 16, q = lane / 16;

    // Workgroups go to the eight XCDs in turn; each XCD takes a run of tiles, in bands of rows of x,
    // so that its cache serves one band's x and W moving past it.
    const int tiles = tiles_m * tiles_n, all = tiles * parts;
    const int run = (all + 7) / 8, id = (int)blockIdx.x % 8 * run + (int)blockIdx.x / 8;
    if ((int)blockIdx.x / 8 >= run || id >= all)
        return;
    const int part = id / tiles, tile = id % tiles;
    constexpr int kBand = 8;
    const int band = tile / (kBand * tiles_n) * kBand, in_band = tile % (kBand * tiles_n);
    const int high = tiles_m - band < kBand ? tiles_m - band : kBand;
    const int r0 = (band + in_band % high) * TM, c0 = in_band / high * TN + wave * FN * 16;

    const int k_tiles = (a.k + kFp4K - 1) / kFp4K, blocks = (a.n + 15) / 16;
    Tiles w[FN];
#pragma unroll
    for (int g = 0; g < FN; ++g) {
        const bool there = c0 / 16 + g < blocks;
        w[g] = tiles_of(a.codes, a.scales, there ? c0 / 16 + g : 0, k_tiles, there);
    }
    const uint32_t row_bytes = (uint32_t)a.k * 2u;
    const int rows = a.m - r0 < TM ? a.m - r0 : TM;
    const rsrc_t x = make_rsrc(a.x + (int64_t)r0 * a.k, (uint32_t)rows * row_bytes);  // further rows read zeros
    const int first = (int)((int64_t)k_tiles * part / parts), last = (int)((int64_t)k_tiles * (part + 1) / parts);
    // load i of the wave: rows 4 (wave kLoads + i) ..+4, chunk i16 ^ row % 8 of each
    const int chunk[2] = {i16 ^ q, i16 ^ (4 + q)};
    const uint32_t base = (uint32_t)(4 * wave * kLoads + q) * row_bytes;
    auto load = [&](u32x4 *to, int t) {
        const int k = t * kFp4K;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool in = t < last && k + chunk[i % 2] * 8 < a.k;  // past the last step: zeros
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x, (shared_void *)(to + (wave * kLoads + i) * 64), 16,
                                                     in ? base + (uint32_t)(4 * i) * row_bytes + chunk[i % 2] * 16 : kNowhere,
                                                     k * 2, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 acc[FM][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int g = 0; g < FN; ++g)
            acc[f][g] = f32x4{0, 0, 0, 0};
    // Units of up to four row tiles of x and one word of W; a unit's operands are read beside the
    // products of the one before it.
    constexpr int kUnit = FM < 4 ? FM : 4, kUnits = 4 * FM / kUnit;
    const int get = i16 * 16 + (q ^ i16 % 8), get_odd = get ^ 4;  // word j: 8 (j / 2) further
    auto step = [&](u32x4 *now, const Ahead<FN> &tiles_now, Ahead<FN> &tiles_next, int t) {
        tiles_next.template load<true>(w, t + 1 < last ? t + 1 : k_tiles);
        __builtin_amdgcn_sched_barrier(0);  // here, not where the step ends and waits for them
        u32x4 b[2][kUnit], wide[FN];
        auto read = [&](int u) __attribute__((always_inline)) {
            const int j = u / (FM / kUnit), f0 = u % (FM / kUnit) * kUnit;
#pragma unroll
            for (int f = 0; f < kUnit; ++f)
                b[u % 2][f] = now[(j % 2 ? get_odd : get) + j / 2 * 8 + (f0 + f) * 256];
        };
        read(0);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int j = u / (FM / kUnit), f0 = u % (FM / kUnit) * kUnit;
            if (u + 1 < kUnits)
                read(u + 1);
            if (f0 == 0) {
#pragma unroll
                for (int g = 0; g < FN; ++g)
                    wide[g] = fp4_widen(tiles_now.codes[g][j], fp4_scale(tiles_now.scales[g], j));
            }
#pragma unroll
            for (int f = 0; f < kUnit; ++f)
#pragma unroll
                for (int g = 0; g < FN; ++g)
                    acc[f0 + f][g] = mfma16<DT_BF16>(wide[g], b[u % 2][f], acc[f0 + f][g]);
            __builtin_amdgcn_sched_barrier(0);  // or later units' operands are read early, and spilt
        }
        wait_and_sync();  // everyone has read `now`, and the other buffer has come
        load(now, t + 2);
    };
    Ahead<FN> even, odd;
    load(s0, first);
    even.template load<true>(w, first);
    load(s1, first + 1);
    wait_and_sync();
    for (int t = first; t < last; ++t) {
        step(s0, even, odd, t);
        if (++t >= last)
            break;
        step(s1, odd, even, t);
    }
    // What a lane adds at the end, its rows of the residual all together.
    constexpr int kLanes = FN * 2, kTogether = 64 / kLanes, kOuts = TM / kTogether;  // lanes a row of eights
    int late = lane;
    asm volatile("" : "+v"(late));  // computed here, not kept over the loop
    const int my_row = late / kLanes, my_col = late % kLanes * 8, col = c0 + my_col;
    Raw8<DT_BF16> bias, residual[kOuts];
    if (a.bias && col < a.n)
        bias = load8<DT_BF16>(reinterpret_cast<const char *>(a.bias), col, a.n);
    if (a.residual && parts == 1) {
        const rsrc_t from = make_rsrc(a.residual + (int64_t)r0 * a.n, (uint32_t)rows * (uint32_t)a.n * 2u);
#pragma unroll
        for (int i = 0; i < kOuts; ++i) {
            const uint32_t row = i * kTogether + my_row;  // rows past the end read zeros
            residual[i].v[0] = __builtin_amdgcn_raw_buffer_load_b128(
                from, col < a.n ? (row * (uint32_t)a.n + col) * 2u : kNowhere, 0, 0);
        }
    }
    wait_and_sync();  // the last loads, of nothing, also write shared memory
    // acc[f][g][e] is row 16 f + lane % 16, column c0 + 16 g + 4 (lane / 16) + e. Through shared memory,
    // 16 rows at a time, into rows of eight columns a lane.
    constexpr int kChunks = FN * 4, kOwn = TM * 16 * 2 / W;
    static_assert(16 * kChunks <= kOwn, "");
    u32x4 *const own = wave < W / 2 ? s0 + wave * kOwn : s1 + (wave - W / 2) * kOwn;
#pragma unroll
    for (int f = 0; f < FM; ++f) {
#pragma unroll
        for (int g = 0; g < FN; ++g)
            own[i16 * kChunks + (g * 4 + q ^ i16 % kChunks)] = __builtin_bit_cast(u32x4, acc[f][g]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int t = 0; t < 16 / kTogether; ++t) {
            const int r = t * kTogether + my_row, row = r0 + f * 16 + r;
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
                finish8<DT_BF16>(a, row, col, z, bias, residual[f * 16 / kTogether + t]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Whether a workgroup takes 16 rows of W (the first kernel) or a tile: up to 16 rows of x, and W no wider
// than two such workgroups a CU, or four where a step is one load (its lines of 16 waves cost more to
// start than they read). (us, this and tiles: 16 rows, 2048 x 4096 5.6 and 9.8, 2048 x 16384 13.9 and
// 12.1, 7168 x 16384 24.4 and 14.5 + 3.8, 2048 x 65536 48 and 15.6; one row, 7168 x 16384 15.2 and 13.6 +
// 3.8, 4096 x 32768 24.2 and 14.9 + 3.8.)
bool few_rows(int64_t m, int64_t n) { return m <= 16 && n <= (m <= 4 ? 16384 : 8192); }

bool good_sizes(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m <= (1 << 24) && n >= 8 && k >= 32 && n <= (1 << 20) && k <= (1 << 20) &&
           n * k <= ((int64_t)1 << 36) && m * n <= ((int64_t)1 << 36) && m * k <= ((int64_t)1 << 36);
}

// How a product of many rows is cut: tiles of 16 fm rows of x by 64 fn of W, and the parts of k.
struct Plan {
    int fm, fn;
    int parts;
};

int64_t tile_count(int64_t m, int64_t n, const Plan &p) { return ceil_div(m, 16 * p.fm) * ceil_div(n, 64 * p.fn); }

// The largest tile that leaves work for all of the 256 CUs. (us, with the time of the joining kernel, of
// 64 x 256 and 64 x 128: 1009 x 4096 x 7168, 448 of the larger tiles, 55.9 and 56.1; 1536 rows, 672
// tiles, 77 and 85; 6720 rows 298 and 321. Of 64 x 128 and 32 x 128: 128 x 7168 x 4096, 64 of the
// larger tiles, 19.0 + 4.0 and 16.4 + 4.0; 256 x 1408 x 7168, 224 tiles, 16.0 + 4.1 and 11.0; 512 x 1408 x
// 7168, 448 tiles, 15.2 and 15.8; 1009 x 7168 x 4096, 512 tiles, 56.4 and 61.5; 17 rows fill half of
// a tile of 64: 10.3 and 9.0.) The smaller ones share their k where they are too few for two
// workgroups a CU and k is long, as the joining kernel is a launch more. (Wall time a call in one part
// and in two, 64 x 2048 x 4096 9.5 and 12.4, 64 x 1408 x 7168 8.0 and 12.8; 64 x 7168 x 2048 18.4 and 12.9,
// in eight 12.3. Kernels alone, 17 x 7168 x 4096: 12.3 + 4.0 in four, 9.0 + 4.0 in eight.)
Plan plan(int64_t m, int64_t n, int64_t k)
{
    Plan p = {4, 4, 1};
    if (tile_count(m, n, p) < 512) {
        p = {4, 2, 1};
        if (m <= 32 || tile_count(m, n, p) < 256)
            p.fm = 2;
    }
    const int64_t steps = ceil_div(k, kFp4K), tiles = tile_count(m, n, p);
    while (p.fn == 2 && steps >= 24 && p.parts < 16 && tiles * p.parts * 2 <= 512 && p.parts * 8 <= steps)
        p.parts *= 2;
    return p;
}

template <int FM, int FN>
block_status_t run_tiles(const Args &a, int parts, float *partial, hipStream_t st)
{
    const int tm = (int)ceil_div(a.m, FM * 16), tn = (int)ceil_div(a.n, kTileWaves * FN * 16);
    const int64_t blocks = ceil_div((int64_t)tm * tn * parts, 8) * 8;
    return launch(fp4_linear_tile_kernel<FM, FN>, dim3((unsigned)blocks), dim3(kTileWaves * 64), 0, st, a, tm, tn, parts, partial);
}

block_status_t run_many(const Args &a, float *partial, hipStream_t st)
{
    const Plan p = plan(a.m, a.n, a.k);
    const block_status_t r = p.fn == 4   ? run_tiles<4, 4>(a, p.parts, partial, st)
                             : p.fm == 4 ? run_tiles<4, 2>(a, p.parts, partial, st)
                                         : run_tiles<2, 2>(a, p.parts, partial, st);
    if (r || p.parts == 1)
        return r;
    const int64_t blocks = ceil_div((int64_t)a.m * a.n, 2048);
    return launch(linear_join_kernel<DT_BF16>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a, p.parts,
                  partial);
}

}  // namespace

extern "C" {

int64_t block_linear_act_fp4_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!good_sizes(m, n, k) || k % 32 || n % 8 || few_rows(m, n))
        return 0;
    const Plan p = plan(m, n, k);
    return p.parts > 1 ? p.parts * m * n * 4 : 0;
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
    const Args a = {{x, nullptr, bias, residual, y, (int)m, (int)n, (int)k, act}, codes, scales};
    if (!few_rows(m, n))
        return run_many(a, static_cast<float *>(workspace), stream);
    const dim3 grid((unsigned)s.row_tiles()), threads(kWaves * 64);
    return m <= 4 ? launch(fp4_linear_few_kernel<1, 4>, grid, threads, 0, stream, a)
                  : launch(fp4_linear_few_kernel<4, 2>, grid, threads, 0, stream, a);
}

}  // extern "C"
