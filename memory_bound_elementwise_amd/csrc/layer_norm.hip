// Layer norm, forward and backward, for AMD Instinct MI355X (gfx950). C ABI declared in
// block/moe_block.h.
//
// Both directions read each row once: its elements stay in registers, spread over WPR
// waves of CH groups of eight per lane, while the row's sums are formed (a lane's own
// elements in order, then the wave's fixed DPP tree, then the waves in order through
// LDS). Rows too wide for that are walked again from cache (the *_wide kernels).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "block_device.h"
#include "block_host.h"

namespace {

using namespace block;

// Sum over the WPR waves that share a row, the same value in every one of their lanes.
// `slot`: WPR floats of LDS of the row's own. The caller alternates between two sets of
// slots, so one barrier a sum is enough: nobody can write a set again before everyone
// has passed the barrier of the other.
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*slot)[16], int wave)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_sum(v[i]);
    if constexpr (WPR > 1) {
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                slot[i][wave] = v[i];
        }
        __syncthreads();
        const int first = wave / WPR * WPR;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = slot[i][first];
#pragma unroll
            for (int w = 1; w < WPR; ++w)
                t += slot[i][first + w];
            v[i] = t;
        }
    }
}

template <int WDT>
__device__ __forceinline__ void weights8(const char *w, int j, int n, float absent, float (&f)[8])
{
    if (w) {
        widen8<WDT>(load8<WDT>(w, j, n), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = absent;
    }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// A first mean is the row's sum divided once; it can be off by some steps of the row's largest
// value, however small the row's deviations are. The second pass therefore sums the deviations from
// it beside their squares, in one exchange: their mean (`rest`) is what the first one lacked.
__device__ __forceinline__ float reciprocal_deviation(float mean_square, float rest, float eps)
{
    const float var = __builtin_elementwise_maximum(mean_square - rest * rest, 0.0f);  // keeps NaN
    return 1.0f / sqrtf(var + eps);
}

// A fixed number of workgroups walks the rows: each keeps its columns' weights in registers,
// as they lie in memory, and loads its next row while it sums this one. (One workgroup a row
// read the weights from cache for each: with fp32 ones, twice the row's own bytes; 6720 x 7168
// bf16 took 45.6 us so, and takes 31: 6.2 TB/s.)
template <int DT, int WDT, int WPR, int CH, int BLOCK, bool EVEN>
__global__ __launch_bounds__(BLOCK) void layer_norm_fwd_kernel(const char *x, const char *weight, const char *bias,
                                                               char *y, float *mean, float *rstd, int64_t rows,
                                                               int cols, float eps)
{
    constexpr int kGroups = BLOCK / 64 / WPR;
    __shared__ float slots[2][2][16];
    const int wave = wave_in_block();
    const int at = (int)threadIdx.x % (WPR * 64) * 8;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float n_cols = (float)cols;
    Raw8<DT> next[CH];
    auto fetch = [&](int64_t r) {
        const Row<DT, EVEN> row(x, r, cols, r < rows);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            next[c] = row.load(at + c * WPR * 512);
    };
    int64_t r = (int64_t)blockIdx.x * kGroups + wave / WPR;
    fetch(r);
    Raw8<WDT> w[CH], b[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int j = at + c * WPR * 512;
        if (weight)
            w[c] = load8<WDT>(weight, j, cols);
        if (bias)
            b[c] = load8<WDT>(bias, j, cols);
    }
    // every group of the workgroup makes the same number of turns (the sums hold barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < rows; r0 += step, r += step) {
        const bool live = r < rows;
        const int n = live ? cols : 0;
        float v[CH][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            widen8<DT>(next[c], v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[0] += v[c][i];
        }
        fetch(r + step);
        row_sums<WPR>(sum, slots[0], wave);
        const float mu = sum[0] / n_cols;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            const float m = j < n ? mu : 0.0f;  // a group past the row's end stays 0
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[c][i] -= m;
                const float d = EVEN || j + i < n ? v[c][i] : 0.0f;
                s[0] += d;
                s[1] = __builtin_fmaf(d, d, s[1]);
            }
        }
        row_sums<WPR>(s, slots[1], wave);
        const float rest = s[0] / n_cols, rs = reciprocal_deviation(s[1] / n_cols, rest, eps);
        const float shift = -rest * rs;  // (v - rest) rs = v rs + shift
        const Row<DT, EVEN> out(y, r, cols, live);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float fw[8], fb[8];
            widen8<WDT>(w[c], fw);
            widen8<WDT>(b[c], fb);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c][i] = __builtin_fmaf(__builtin_fmaf(v[c][i], rs, shift), weight ? fw[i] : 1.0f, bias ? fb[i] : 0.0f);
            out.store(at + c * WPR * 512, v[c]);
        }
        if (live && mean && threadIdx.x % (WPR * 64) == 0) {
            mean[r] = mu + rest;
            rstd[r] = rs;
        }
    }
}

constexpr int kWideThreads = 1024;

// Rows of any width: one workgroup of 16 waves a row, which it reads three times (the
// second and third time from cache).
template <int DT, int WDT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_fwd_wide_kernel(const char *x, const char *weight,
                                                                   const char *bias, char *y, float *mean,
                                                                   float *rstd, int64_t rows, int cols, float eps)
{
    __shared__ float slots[2][2][16];
    const int wave = wave_in_block();
    const float n_cols = (float)cols;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t off = r * cols * kSize<DT>;
        float f[8];
        float sum[1] = {0.0f}, s[2] = {0.0f, 0.0f};
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            widen8<DT>(load8<DT>(x + off, j, cols), f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[0] += f[i];
        }
        row_sums<16>(sum, slots[0], wave);
        const float mu = sum[0] / n_cols;
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            widen8<DT>(load8<DT>(x + off, j, cols), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = j + i < cols ? f[i] - mu : 0.0f;
                s[0] += d;
                s[1] = __builtin_fmaf(d, d, s[1]);
            }
        }
        row_sums<16>(s, slots[1], wave);
        const float rest = s[0] / n_cols, rs = reciprocal_deviation(s[1] / n_cols, rest, eps);
        const float shift = -rest * rs;  // (v - rest) rs = v rs + shift
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            float w[8], b[8];
            widen8<DT>(load8<DT>(x + off, j, cols), f);
            weights8<WDT>(weight, j, cols, 1.0f, w);
            weights8<WDT>(bias, j, cols, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __builtin_fmaf(__builtin_fmaf(f[i] - mu, rs, shift), w[i], b[i]);
            store8<DT>(y + off, j, cols, f);
        }
        if (mean && threadIdx.x == 0) {
            mean[r] = mu + rest;
            rstd[r] = rs;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// A fixed number of workgroups walks the rows. Each lane owns its columns for the whole walk,
// so it adds their weight and bias gradients in registers, and a workgroup writes one partial
// row of each at its end; layer_norm_partials_kernel adds those. A row's successor is loaded
// while the row is summed, into registers of its own where there are enough (rows in two groups
// of eight a lane): a copy from one set to the other at the end of a row would wait for that
// row's stores too, and so would loads counted behind a branch around the stores. Without grad_x
// the stores are masked, not skipped. (6720 x 7168 bf16: 61 us with the copies, 53 so: 5.5 TB/s;
// 6720 x 2048: 18.2, 15.7; 6720 x 12000: 106, 96; 1009 x 1411 fp32: 10.5, 8.9.)
// part: fp32 [gridDim.x][2][cols] or null.
constexpr int kBwdWaves = 8;
constexpr int kBwdParts = 256;  // one workgroup a CU, so one partial row a CU

template <int DT, int WDT, int WPR, int CH, bool EVEN>
__global__ __launch_bounds__(kBwdWaves * 64) void layer_norm_bwd_kernel(const char *gy, const char *x,
                                                                        const char *weight, const float *mean,
                                                                        const float *rstd, char *gx, float *part,
                                                                        int64_t rows, int cols)
{
    constexpr int kGroups = kBwdWaves / WPR, kOwn = WPR * 64;
    __shared__ float slots[2][2][16];
    // the groups' gradients at the end, but the first's: two 16-byte halves of each lane's eight
    __shared__ f32x4 others[kGroups > 1 ? (kGroups - 1) * 2 * CH * 2 * kOwn : 1];
    const int wave = wave_in_block(), group = wave / WPR;
    const int lane = (int)threadIdx.x % kOwn, at = lane * 8;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float n_cols = (float)cols;
    struct Loaded {
        Raw8<DT> g[CH], x[CH];
        float mean, rstd;
    };
    auto fetch = [&](Loaded &to, int64_t r) __attribute__((always_inline)) {
        const bool live = r < rows;
        const Row<DT, EVEN> row_g(gy, r, cols, live), row_x(x, r, cols, live);
        const Row<DT_F32, true> m(mean, r, 1, live), q(rstd, r, 1, live);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            to.g[c] = row_g.load(at + c * WPR * 512);
            to.x[c] = row_x.load(at + c * WPR * 512);
        }
        to.mean = m.load1(0);
        to.rstd = q.load1(0);
    };
    constexpr bool kAhead = CH <= 2;
    Loaded even, odd;
    int64_t r = (int64_t)blockIdx.x * kGroups + group;
    fetch(even, r);
    Raw8<WDT> w[CH];
    float dw[CH][8], db[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (weight)
            w[c] = load8<WDT>(weight, at + c * WPR * 512, cols);  // zeros past the end
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[c][i] = db[c][i] = 0.0f;
    }
    // One row, and the loads of the next. The caller gives the two sets in turn, or one twice.
    auto one = [&](const Loaded &row, Loaded &next, int64_t r, float(*slot)[16]) __attribute__((always_inline)) {
        const bool live = r < rows;
        const int n = live ? cols : 0;
        const float mu = row.mean, rs = row.rstd;
        if constexpr (kAhead)
            fetch(next, r + step);
        float g[CH][8], h[CH][8];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            float fw[8];
            widen8<DT>(row.g[c], g[c]);
            widen8<DT>(row.x[c], h[c]);
            widen8<WDT>(w[c], fw);
            // past the row's end g and x are 0; h is kept 0 too, so an infinite statistic of the
            // row cannot put a NaN there
            const float m = j < n ? mu : 0.0f, q = j < n ? rs : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] = EVEN || j + i < n ? (h[c][i] - m) * q : 0.0f;
                dw[c][i] = __builtin_fmaf(g[c][i], h[c][i], dw[c][i]);
                db[c][i] += g[c][i];
                if (weight)
                    g[c][i] *= fw[i];
                s[0] += g[c][i];
                s[1] = __builtin_fmaf(g[c][i], h[c][i], s[1]);
            }
        }
        if constexpr (!kAhead) {
            __builtin_amdgcn_sched_barrier(0);
            fetch(next, r + step);
            __builtin_amdgcn_sched_barrier(0);
        }
        row_sums<WPR>(s, slot, wave);
        const float a = s[0] / n_cols, b = s[1] / n_cols;
        const Row<DT, EVEN> out(gx, r, cols, live && gx);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = (g[c][i] - a - h[c][i] * b) * rs;
            out.store(at + c * WPR * 512, o);
        }
    };
    // every group of the workgroup makes the same number of turns (the sums hold barriers)
    int64_t r0 = (int64_t)blockIdx.x * kGroups;
    if constexpr (kAhead) {
        for (; r0 + step < rows; r0 += 2 * step, r += 2 * step) {
            one(even, odd, r, slots[0]);
            one(odd, even, r + step, slots[1]);
        }
        if (r0 < rows)
            one(even, odd, r, slots[0]);
    } else {
        for (int turn = 0; r0 < rows; r0 += step, r += step, turn ^= 1)
            one(even, even, r, slots[turn]);
    }
    if (!part)
        return;
    if (group > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f32x4 *to = others + ((group - 1) * CH + c) * 4 * kOwn + k * kOwn + lane;
                to[0] = f32x4{dw[c][4 * k], dw[c][4 * k + 1], dw[c][4 * k + 2], dw[c][4 * k + 3]};
                to[2 * kOwn] = f32x4{db[c][4 * k], db[c][4 * k + 1], db[c][4 * k + 2], db[c][4 * k + 3]};
            }
    }
    __syncthreads();
    if (group > 0)
        return;
    char *pw = reinterpret_cast<char *>(part + (int64_t)blockIdx.x * 2 * cols);
    char *pb = pw + (int64_t)cols * 4;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        for (int o = 0; o < kGroups - 1; ++o)  // the groups' sums, in group order
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4 *from = others + (o * CH + c) * 4 * kOwn + k * kOwn + lane;
                const f32x4 vw = from[0], vb = from[2 * kOwn];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dw[c][4 * k + i] += vw[i];
                    db[c][4 * k + i] += vb[i];
                }
            }
        store8<DT_F32>(pw, at + c * WPR * 512, cols, dw[c]);
        store8<DT_F32>(pb, at + c * WPR * 512, cols, db[c]);
    }
}

// Rows of any width, grad_x only: one workgroup a row, which it reads twice.
template <int DT, int WDT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_bwd_x_wide_kernel(const char *gy, const char *x,
                                                                     const char *weight, const float *mean,
                                                                     const float *rstd, char *gx, int64_t rows,
                                                                     int cols)
{
    __shared__ float slots[2][2][16];
    const int wave = wave_in_block();
    const float n_cols = (float)cols;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
        const int64_t off = r * cols * kSize<DT>;
        const float mu = mean[r], rs = rstd[r];
        float s[2] = {0.0f, 0.0f};
        float g[8], h[8], w[8];
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            widen8<DT>(load8<DT>(gy + off, j, cols), g);
            widen8<DT>(load8<DT>(x + off, j, cols), h);
            weights8<WDT>(weight, j, cols, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (j + i < cols) {
                    s[0] += g[i] * w[i];
                    s[1] = __builtin_fmaf(g[i] * w[i], (h[i] - mu) * rs, s[1]);
                }
        }
        row_sums<16>(s, slots[turn], wave);
        const float a = s[0] / n_cols, b = s[1] / n_cols;
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            widen8<DT>(load8<DT>(gy + off, j, cols), g);
            widen8<DT>(load8<DT>(x + off, j, cols), h);
            weights8<WDT>(weight, j, cols, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = (g[i] * w[i] - a - (h[i] - mu) * rs * b) * rs;
            store8<DT>(gx + off, j, cols, g);
        }
    }
}

// Rows of any width, the weight's gradients: a workgroup takes 2048 columns and every
// gridDim.y-th row.
template <int DT>
__global__ __launch_bounds__(256) void layer_norm_bwd_w_wide_kernel(const char *gy, const char *x, const float *mean,
                                                                    const float *rstd, float *part, int64_t rows,
                                                                    int cols)
{
    const int j = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (j >= cols)
        return;
    float dw[8] = {}, db[8] = {};
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const int64_t off = r * cols * kSize<DT>;
        const float mu = mean[r], rs = rstd[r];
        float g[8], h[8];
        widen8<DT>(load8<DT>(gy + off, j, cols), g);
        widen8<DT>(load8<DT>(x + off, j, cols), h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = __builtin_fmaf(g[i], (h[i] - mu) * rs, dw[i]);
            db[i] += g[i];
        }
    }
    char *pw = reinterpret_cast<char *>(part + (int64_t)blockIdx.y * 2 * cols);
    store8<DT_F32>(pw, j, cols, dw);
    store8<DT_F32>(pw + (int64_t)cols * 4, j, cols, db);
}

// Adds the partial rows: part [parts][2][cols] -> grad_weight, grad_bias. A workgroup takes N
// neighbouring values of the 2 cols; each of its 1024 / N slices of N lanes adds every
// (1024 / N)-th partial row, and the slices' sums are added in order. parts == 0 writes zeros.
template <int WDT, int N>
__global__ __launch_bounds__(1024) void layer_norm_partials_kernel(const float *part, char *gw, char *gb, int parts,
                                                                   int cols)
{
    constexpr int kSlices = 1024 / N;
    __shared__ float sums[kSlices][N];
    const int slice = threadIdx.x / N, i = threadIdx.x % N;
    const int64_t j = (int64_t)blockIdx.x * N + i;
    const int64_t n = 2 * (int64_t)cols;
    // at most kBwdParts partial rows, so a fixed number of loads, all under way at once
    float v[kBwdParts / kSlices];
#pragma unroll
    for (int k = 0; k < kBwdParts / kSlices; ++k) {
        const int p = slice + k * kSlices;
        v[k] = j < n && p < parts ? part[p * n + j] : 0.0f;
    }
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kBwdParts / kSlices; ++k)
        t += v[k];
    sums[slice][i] = t;
    __syncthreads();
    if (slice == 0 && j < n) {
#pragma unroll
        for (int k = 1; k < kSlices; ++k)
            t += sums[k][i];
        char *out = j < cols ? gw : gb;
        if (out)
            store1<WDT>(out, j < cols ? j : j - cols, t);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kMaxCols = 1 << 20;
constexpr int64_t kMaxHeld = 16384;  // columns of a row that is held in registers
constexpr int64_t kMaxElems = (int64_t)1 << 48;
constexpr int kFwdWaves = 256 * 8;     // two a SIMD: 31.2 us for 6720 x 7168 bf16; three 32.1, four 36
constexpr int kFwdBlocks = 256;        // but a workgroup a CU: 2000 x 12000 bf16 21 us, with 128 36

int elem_size(block_dtype_t d) { return d == BLOCK_FP32 ? 4 : 2; }

bool known(block_dtype_t d) { return d == BLOCK_BF16 || d == BLOCK_FP16 || d == BLOCK_FP32; }

struct Args {
    const void *x, *gy, *weight, *bias;
    const float *mean, *rstd;
    void *y;
    float *mean_out, *rstd_out;
    void *gx, *gw, *gb;
    float *part;
    int64_t rows;
    int cols;
    float eps;
    hipStream_t st;
};

int bwd_groups(int64_t cols)
{
    // waves a row: the fewest that hold it in two groups of eight a lane
    int wpr = 1;
    while (wpr < kBwdWaves && cols > (int64_t)wpr * 1024)
        wpr *= 2;
    return kBwdWaves / wpr;
}

int bwd_parts(int64_t rows, int64_t cols)
{
    const int64_t groups = cols > kMaxHeld ? 1 : bwd_groups(cols);
    const int64_t need = ceil_div(rows, groups);
    return (int)(need < kBwdParts ? need : kBwdParts);
}

dim3 wide_grid(const Args &a)
{
    return dim3((unsigned)(a.rows < max_groups(kWideThreads) ? a.rows : max_groups(kWideThreads)));
}

template <int DT, int WDT, int WPR, int CH, int BLOCK, bool EVEN>
block_status_t fwd_as(const Args &a)
{
    constexpr int64_t most = kFwdWaves / (BLOCK / 64) > kFwdBlocks ? kFwdWaves / (BLOCK / 64) : kFwdBlocks;
    const int64_t blocks = ceil_div(a.rows, BLOCK / 64 / WPR);
    return launch(layer_norm_fwd_kernel<DT, WDT, WPR, CH, BLOCK, EVEN>, dim3((unsigned)(blocks < most ? blocks : most)),
                  dim3(BLOCK), 0, a.st, static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                  static_cast<const char *>(a.bias), static_cast<char *>(a.y), a.mean_out, a.rstd_out, a.rows, a.cols,
                  a.eps);
}

template <int DT, int WDT>
struct Fwd {
    template <bool EVEN>
    static block_status_t held(const Args &a)
    {
        if (a.cols <= 512)
            return fwd_as<DT, WDT, 1, 1, 256, EVEN>(a);
        if (a.cols <= 1024)
            return fwd_as<DT, WDT, 1, 2, 256, EVEN>(a);
        if (a.cols <= 2048)  // two waves a row wait less on each other than four: 6720 x 2048 bf16 12.1 us, 15.9
            return fwd_as<DT, WDT, 2, 2, 256, EVEN>(a);
        if (a.cols <= 4096)
            return fwd_as<DT, WDT, 4, 2, 256, EVEN>(a);
        if (a.cols <= 8192)
            return fwd_as<DT, WDT, 4, 4, 256, EVEN>(a);
        return fwd_as<DT, WDT, 16, 2, 1024, EVEN>(a);
    }
    static block_status_t run(const Args &a)
    {
        if (a.cols <= kMaxHeld)
            return a.cols % 8 == 0 ? held<true>(a) : held<false>(a);
        return launch(layer_norm_fwd_wide_kernel<DT, WDT>, wide_grid(a), dim3(kWideThreads), 0, a.st,
                      static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                      static_cast<const char *>(a.bias), static_cast<char *>(a.y), a.mean_out, a.rstd_out, a.rows,
                      a.cols, a.eps);
    }
};

template <int DT, int WDT, int WPR, int CH, bool EVEN>
block_status_t bwd_as(const Args &a)
{
    return launch(layer_norm_bwd_kernel<DT, WDT, WPR, CH, EVEN>, dim3(bwd_parts(a.rows, a.cols)), dim3(kBwdWaves * 64), 0, a.st,
                  static_cast<const char *>(a.gy), static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                  a.mean, a.rstd, static_cast<char *>(a.gx), a.part, a.rows, a.cols);
}

template <int DT, int WDT>
struct Bwd {
    template <bool EVEN>
    static block_status_t held(const Args &a)
    {
        if (a.cols <= 512)
            return bwd_as<DT, WDT, 1, 1, EVEN>(a);
        if (a.cols <= 1024)
            return bwd_as<DT, WDT, 1, 2, EVEN>(a);
        if (a.cols <= 2048)
            return bwd_as<DT, WDT, 2, 2, EVEN>(a);
        if (a.cols <= 4096)
            return bwd_as<DT, WDT, 4, 2, EVEN>(a);
        if (a.cols <= 8192)
            return bwd_as<DT, WDT, 8, 2, EVEN>(a);
        return bwd_as<DT, WDT, 8, 4, EVEN>(a);
    }
    static block_status_t run(const Args &a)
    {
        if (a.cols <= kMaxHeld)
            return a.cols % 8 == 0 ? held<true>(a) : held<false>(a);
        block_status_t s = BLOCK_OK;
        if (a.gx)
            s = launch(layer_norm_bwd_x_wide_kernel<DT, WDT>, wide_grid(a), dim3(kWideThreads), 0, a.st,
                       static_cast<const char *>(a.gy), static_cast<const char *>(a.x),
                       static_cast<const char *>(a.weight), a.mean, a.rstd, static_cast<char *>(a.gx), a.rows, a.cols);
        if (s == BLOCK_OK && a.part)
            s = launch(layer_norm_bwd_w_wide_kernel<DT>, dim3((unsigned)ceil_div(a.cols, 2048), bwd_parts(a.rows, a.cols)),
                       dim3(256), 0, a.st, static_cast<const char *>(a.gy), static_cast<const char *>(a.x), a.mean,
                       a.rstd, a.part, a.rows, a.cols);
        return s;
    }
};

// Wide rows of sums are added 64 values a workgroup (whole lines), narrow ones 16, so that
// there are workgroups enough (7168 columns: 5.2 against 6.6 us; 1411: 6.7 against 4.1).
template <int WDT>
block_status_t add_partials(const float *part, char *gw, char *gb, int parts, int cols, hipStream_t st)
{
    if (2 * cols >= 64 * 128)
        return launch(layer_norm_partials_kernel<WDT, 64>, dim3((unsigned)ceil_div(2 * cols, 64)), dim3(1024), 0, st,
                      part, gw, gb, parts, cols);
    return launch(layer_norm_partials_kernel<WDT, 16>, dim3((unsigned)ceil_div(2 * cols, 16)), dim3(1024), 0, st, part,
                  gw, gb, parts, cols);
}

template <template <int, int> class K>
block_status_t by_type(block_dtype_t d, block_dtype_t w, const Args &a)
{
    if (d == BLOCK_BF16)
        return w == BLOCK_FP32 ? K<DT_BF16, DT_F32>::run(a) : K<DT_BF16, DT_BF16>::run(a);
    if (d == BLOCK_FP16)
        return w == BLOCK_FP32 ? K<DT_F16, DT_F32>::run(a) : K<DT_F16, DT_F16>::run(a);
    return K<DT_F32, DT_F32>::run(a);
}

block_status_t check_sizes(int64_t rows, int64_t cols, block_dtype_t d, block_dtype_t w)
{
    if (!known(d) || !known(w) || (w != d && w != BLOCK_FP32))
        return BLOCK_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols > kMaxCols || rows > kMaxElems / cols)
        return BLOCK_ERR_INVALID_ARG;
    return BLOCK_OK;
}

}  // namespace

extern "C" {

block_status_t block_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean,
                                    float *rstd, int64_t rows, int64_t cols, float eps, block_dtype_t dtype,
                                    block_dtype_t weight_dtype, hipStream_t stream)
{
    if (const block_status_t s = check_sizes(rows, cols, dtype, weight_dtype))
        return s;
    if (!(eps >= 0.0f) || std::isinf(eps) || (mean == nullptr) != (rstd == nullptr))
        return BLOCK_ERR_INVALID_ARG;
    if (rows == 0)
        return BLOCK_OK;
    if (!x || !y)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(weight, 16) || misaligned(bias, 16) ||
        misaligned(mean, 4) || misaligned(rstd, 4))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t n = rows * cols * elem_size(dtype), v = cols * elem_size(weight_dtype);
    if (any_overlap<3, 3>({{y, n}, {mean, rows * 4}, {rstd, rows * 4}}, {{x, n}, {weight, v}, {bias, v}}))
        return BLOCK_ERR_INVALID_ARG;
    Args a = {};
    a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.mean_out = mean, a.rstd_out = rstd;
    a.rows = rows, a.cols = (int)cols, a.eps = eps, a.st = stream;
    return by_type<Fwd>(dtype, weight_dtype, a);
}

int64_t block_layer_norm_bwd_workspace(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || cols > kMaxCols || rows > kMaxElems / cols)
        return 0;
    return (int64_t)bwd_parts(rows, cols) * 2 * cols * 4;
}

block_status_t block_layer_norm_bwd(const void *grad_y, const void *x, const void *weight, const float *mean,
                                    const float *rstd, void *grad_x, void *grad_weight, void *grad_bias, int64_t rows,
                                    int64_t cols, block_dtype_t dtype, block_dtype_t weight_dtype, void *workspace,
                                    int64_t workspace_bytes, hipStream_t stream)
{
    if (const block_status_t s = check_sizes(rows, cols, dtype, weight_dtype))
        return s;
    const bool sums = grad_weight || grad_bias;
    const int64_t need = sums ? block_layer_norm_bwd_workspace(rows, cols) : 0;
    if (rows > 0 && (!grad_y || !x || !mean || !rstd || (need > 0 && (!workspace || workspace_bytes < need))))
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(grad_y, 16) || misaligned(weight, 16) || misaligned(grad_x, 16) ||
        misaligned(grad_weight, 16) || misaligned(grad_bias, 16) || misaligned(mean, 4) || misaligned(rstd, 4) ||
        (need > 0 && misaligned(workspace, 16)))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t n = rows * cols * elem_size(dtype), v = cols * elem_size(weight_dtype);
    if (any_overlap<4, 5>({{grad_x, n}, {grad_weight, v}, {grad_bias, v}, {workspace, need}},
                          {{grad_y, n}, {x, n}, {weight, v}, {mean, rows * 4}, {rstd, rows * 4}}))
        return BLOCK_ERR_INVALID_ARG;
    Args a = {};
    a.x = x, a.gy = grad_y, a.weight = weight, a.mean = mean, a.rstd = rstd;
    a.gx = grad_x, a.gw = grad_weight, a.gb = grad_bias, a.part = sums ? static_cast<float *>(workspace) : nullptr;
    a.rows = rows, a.cols = (int)cols, a.st = stream;
    if (rows > 0 && (sums || grad_x))
        if (const block_status_t s = by_type<Bwd>(dtype, weight_dtype, a))
            return s;
    if (!sums)
        return BLOCK_OK;
    const int parts = rows > 0 ? bwd_parts(rows, cols) : 0;
    const float *part = static_cast<const float *>(workspace);
    char *gw = static_cast<char *>(grad_weight), *gb = static_cast<char *>(grad_bias);
    if (weight_dtype == BLOCK_BF16)
        return add_partials<DT_BF16>(part, gw, gb, parts, (int)cols, stream);
    if (weight_dtype == BLOCK_FP16)
        return add_partials<DT_F16>(part, gw, gb, parts, (int)cols, stream);
    return add_partials<DT_F32>(part, gw, gb, parts, (int)cols, stream);
}

}  // extern "C"
