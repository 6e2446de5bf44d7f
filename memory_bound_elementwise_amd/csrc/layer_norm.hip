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
template <int DT, int WDT, int WPR, int CH, int BLOCK>
__global__ __launch_bounds__(BLOCK) void layer_norm_fwd_kernel(const char *x, const char *weight, const char *bias,
                                                               char *y, float *mean, float *rstd, int64_t rows,
                                                               int cols, float eps)
{
    constexpr int kGroups = BLOCK / 64 / WPR;
    __shared__ float slots[2][1][16];
    const int wave = wave_in_block();
    const int at = (int)threadIdx.x % (WPR * 64) * 8;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float n_cols = (float)cols;  // divided by: the mean of a constant row is that constant
    // every group of the workgroup makes the same number of turns (the sums hold barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < rows; r0 += step) {
        const int64_t r = r0 + wave / WPR;
        const bool live = r < rows;
        const int n = live ? cols : 0;
        const int64_t off = live ? r * cols * kSize<DT> : 0;
        float v[CH][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            widen8<DT>(load8<DT>(x + off, j, n), v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[0] += v[c][i];
        }
        row_sums<WPR>(sum, slots[0], wave);
        const float mu = sum[0] / n_cols;
        float sq[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[c][i] -= mu;
                sq[0] += j + i < n ? v[c][i] * v[c][i] : 0.0f;
            }
        }
        row_sums<WPR>(sq, slots[1], wave);
        const float rs = 1.0f / sqrtf(sq[0] / n_cols + eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            float w[8], b[8];
            weights8<WDT>(weight, j, cols, 1.0f, w);
            weights8<WDT>(bias, j, cols, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = __builtin_fmaf(v[c][i] * rs, w[i], b[i]);
            store8<DT>(y + off, j, n, w);
        }
        if (live && mean && threadIdx.x % (WPR * 64) == 0) {
            mean[r] = mu;
            rstd[r] = rs;
        }
    }
}

// Rows of any width: one workgroup of 16 waves a row, which it reads three times (the
// second and third time from cache).
template <int DT, int WDT>
__global__ __launch_bounds__(1024) void layer_norm_fwd_wide_kernel(const char *x, const char *weight,
                                                                   const char *bias, char *y, float *mean,
                                                                   float *rstd, int64_t rows, int cols, float eps)
{
    __shared__ float slots[2][1][16];
    const int wave = wave_in_block();
    const float n_cols = (float)cols;  // divided by: the mean of a constant row is that constant
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t off = r * cols * kSize<DT>;
        float f[8];
        float sum[1] = {0.0f}, sq[1] = {0.0f};
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
            for (int i = 0; i < 8; ++i)
                sq[0] += j + i < cols ? (f[i] - mu) * (f[i] - mu) : 0.0f;
        }
        row_sums<16>(sq, slots[1], wave);
        const float rs = 1.0f / sqrtf(sq[0] / n_cols + eps);
        for (int j = threadIdx.x * 8; j < cols; j += 8192) {
            float w[8], b[8];
            widen8<DT>(load8<DT>(x + off, j, cols), f);
            weights8<WDT>(weight, j, cols, 1.0f, w);
            weights8<WDT>(bias, j, cols, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __builtin_fmaf((f[i] - mu) * rs, w[i], b[i]);
            store8<DT>(y + off, j, cols, f);
        }
        if (mean && threadIdx.x == 0) {
            mean[r] = mu;
            rstd[r] = rs;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// A fixed number of workgroups of 16 waves walks the rows. Each lane owns its columns for
// the whole walk, so it adds their weight and bias gradients in registers, and a
// workgroup writes one partial row of each at its end; layer_norm_partials_kernel adds
// those. part: fp32 [gridDim.x][2][cols] or null.
template <int DT, int WDT, int WPR, int CH>
__global__ __launch_bounds__(1024) void layer_norm_bwd_kernel(const char *gy, const char *x, const char *weight,
                                                              const float *mean, const float *rstd, char *gx,
                                                              float *part, int64_t rows, int cols)
{
    constexpr int kGroups = 16 / WPR;
    __shared__ float slots[2][2][16];
    extern __shared__ float sums[];  // [2][cols]: only where several groups share a workgroup
    const int wave = wave_in_block();
    const int at = (int)threadIdx.x % (WPR * 64) * 8;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float n_cols = (float)cols;  // divided by: the mean of a constant row is that constant
    float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        weights8<WDT>(weight, at + c * WPR * 512, cols, 1.0f, w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[c][i] = db[c][i] = 0.0f;
    }
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < rows; r0 += step, turn ^= 1) {
        const int64_t r = r0 + wave / WPR;
        const bool live = r < rows;
        const int n = live ? cols : 0;
        const int64_t off = live ? r * cols * kSize<DT> : 0;
        const float mu = live ? mean[r] : 0.0f, rs = live ? rstd[r] : 0.0f;
        float g[CH][8], h[CH][8];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            widen8<DT>(load8<DT>(gy + off, j, n), g[c]);
            widen8<DT>(load8<DT>(x + off, j, n), h[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // past the row's end g is 0; h is kept 0 too, so an infinite statistic of
                // the row cannot put a NaN there
                h[c][i] = j + i < n ? (h[c][i] - mu) * rs : 0.0f;
                dw[c][i] = __builtin_fmaf(g[c][i], h[c][i], dw[c][i]);
                db[c][i] += g[c][i];
                g[c][i] = j + i < n ? g[c][i] * w[c][i] : 0.0f;
                s[0] += g[c][i];
                s[1] = __builtin_fmaf(g[c][i], h[c][i], s[1]);
            }
        }
        if (gx) {
            row_sums<WPR>(s, slots[turn], wave);
            const float a = s[0] / n_cols, b = s[1] / n_cols;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = (g[c][i] - a - h[c][i] * b) * rs;
                store8<DT>(gx + off, at + c * WPR * 512, n, o);
            }
        }
    }
    if (!part)
        return;
    // the groups' sums, in group order
    for (int k = kGroups - 1; k > 0; --k) {
        if (wave / WPR == k) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int j = at + c * WPR * 512;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i < cols) {
                        const bool first = k == kGroups - 1;
                        sums[j + i] = dw[c][i] + (first ? 0.0f : sums[j + i]);
                        sums[cols + j + i] = db[c][i] + (first ? 0.0f : sums[cols + j + i]);
                    }
            }
        }
        __syncthreads();
    }
    if (wave / WPR == 0) {
        char *pw = reinterpret_cast<char *>(part + (int64_t)blockIdx.x * 2 * cols);
        char *pb = pw + (int64_t)cols * 4;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = at + c * WPR * 512;
            if constexpr (kGroups > 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i < cols) {
                        dw[c][i] += sums[j + i];
                        db[c][i] += sums[cols + j + i];
                    }
            }
            store8<DT_F32>(pw, j, cols, dw[c]);
            store8<DT_F32>(pb, j, cols, db[c]);
        }
    }
}

// Rows of any width, grad_x only: one workgroup a row, which it reads twice.
template <int DT, int WDT>
__global__ __launch_bounds__(1024) void layer_norm_bwd_x_wide_kernel(const char *gy, const char *x,
                                                                     const char *weight, const float *mean,
                                                                     const float *rstd, char *gx, int64_t rows,
                                                                     int cols)
{
    __shared__ float slots[2][2][16];
    const int wave = wave_in_block();
    const float n_cols = (float)cols;  // divided by: the mean of a constant row is that constant
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

// Adds the partial rows: part [parts][2][cols] -> grad_weight, grad_bias. A workgroup takes
// 64 neighbouring values of the 2 cols; its 16 waves each add every 16th partial row, and
// the waves' sums are added in order. parts == 0 writes zeros.
template <int WDT>
__global__ __launch_bounds__(1024) void layer_norm_partials_kernel(const float *part, char *gw, char *gb, int parts,
                                                                   int cols)
{
    __shared__ float sums[16][64];
    const int wave = wave_in_block(), lane = lane_id();
    const int64_t j = (int64_t)blockIdx.x * 64 + lane;
    const int64_t n = 2 * (int64_t)cols;
    float t = 0.0f;
    if (j < n)
        for (int p = wave; p < parts; p += 16)
            t += part[p * n + j];
    sums[wave][lane] = t;
    __syncthreads();
    if (wave == 0 && j < n) {
        for (int w = 1; w < 16; ++w)
            t += sums[w][lane];
        char *out = j < cols ? gw : gb;
        if (out)
            store1<WDT>(out, j < cols ? j : j - cols, t);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kMaxCols = 1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 48;
constexpr int64_t kMaxGrid = 1 << 22;  // times 1024 threads: a dispatch counts work-items in 32 bits
constexpr int kBwdParts = 256;         // one workgroup a CU, so one partial row a CU

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
    while (wpr < 16 && cols > (int64_t)wpr * 1024)
        wpr *= 2;
    return 16 / wpr;
}

int bwd_parts(int64_t rows, int64_t cols)
{
    const int64_t groups = cols > 16384 ? 1 : bwd_groups(cols);
    const int64_t need = ceil_div(rows, groups);
    return (int)(need < kBwdParts ? need : kBwdParts);
}

template <int DT, int WDT, int WPR, int CH, int BLOCK>
block_status_t fwd_as(const Args &a)
{
    const int64_t blocks = ceil_div(a.rows, BLOCK / 64 / WPR);
    return launch(layer_norm_fwd_kernel<DT, WDT, WPR, CH, BLOCK>, dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid)),
                  dim3(BLOCK), 0, a.st, static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                  static_cast<const char *>(a.bias), static_cast<char *>(a.y), a.mean_out, a.rstd_out, a.rows, a.cols,
                  a.eps);
}

template <int DT, int WDT>
struct Fwd {
    static block_status_t run(const Args &a)
    {
        if (a.cols <= 512)
            return fwd_as<DT, WDT, 1, 1, 256>(a);
        if (a.cols <= 1024)
            return fwd_as<DT, WDT, 1, 2, 256>(a);
        if (a.cols <= 2048)
            return fwd_as<DT, WDT, 4, 1, 256>(a);
        if (a.cols <= 4096)
            return fwd_as<DT, WDT, 4, 2, 256>(a);
        if (a.cols <= 8192)
            return fwd_as<DT, WDT, 4, 4, 256>(a);
        if (a.cols <= 16384)
            return fwd_as<DT, WDT, 16, 2, 1024>(a);
        return launch(layer_norm_fwd_wide_kernel<DT, WDT>, dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)),
                      dim3(1024), 0, a.st, static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                      static_cast<const char *>(a.bias), static_cast<char *>(a.y), a.mean_out, a.rstd_out, a.rows,
                      a.cols, a.eps);
    }
};

template <int DT, int WDT, int WPR, int CH>
block_status_t bwd_as(const Args &a)
{
    constexpr int kGroups = 16 / WPR;
    const uint32_t lds = kGroups > 1 && a.part ? (uint32_t)a.cols * 8u : 0u;
    return launch(layer_norm_bwd_kernel<DT, WDT, WPR, CH>, dim3(bwd_parts(a.rows, a.cols)), dim3(1024), lds, a.st,
                  static_cast<const char *>(a.gy), static_cast<const char *>(a.x), static_cast<const char *>(a.weight),
                  a.mean, a.rstd, static_cast<char *>(a.gx), a.part, a.rows, a.cols);
}

template <int DT, int WDT>
struct Bwd {
    static block_status_t run(const Args &a)
    {
        if (a.cols <= 512)
            return bwd_as<DT, WDT, 1, 1>(a);
        if (a.cols <= 1024)
            return bwd_as<DT, WDT, 1, 2>(a);
        if (a.cols <= 2048)
            return bwd_as<DT, WDT, 2, 2>(a);
        if (a.cols <= 4096)
            return bwd_as<DT, WDT, 4, 2>(a);
        if (a.cols <= 8192)
            return bwd_as<DT, WDT, 8, 2>(a);
        if (a.cols <= 16384)
            return bwd_as<DT, WDT, 16, 2>(a);
        block_status_t s = BLOCK_OK;
        if (a.gx)
            s = launch(layer_norm_bwd_x_wide_kernel<DT, WDT>, dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)),
                       dim3(1024), 0, a.st, static_cast<const char *>(a.gy), static_cast<const char *>(a.x),
                       static_cast<const char *>(a.weight), a.mean, a.rstd, static_cast<char *>(a.gx), a.rows, a.cols);
        if (s == BLOCK_OK && a.part)
            s = launch(layer_norm_bwd_w_wide_kernel<DT>, dim3((unsigned)ceil_div(a.cols, 2048), bwd_parts(a.rows, a.cols)),
                       dim3(256), 0, a.st, static_cast<const char *>(a.gy), static_cast<const char *>(a.x), a.mean,
                       a.rstd, a.part, a.rows, a.cols);
        return s;
    }
};

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
    const dim3 grid((unsigned)ceil_div(2 * cols, 64));
    const int parts = rows > 0 ? bwd_parts(rows, cols) : 0;
    const float *part = static_cast<const float *>(workspace);
    char *gw = static_cast<char *>(grad_weight), *gb = static_cast<char *>(grad_bias);
    if (weight_dtype == BLOCK_BF16)
        return launch(layer_norm_partials_kernel<DT_BF16>, grid, dim3(1024), 0, stream, part, gw, gb, parts, (int)cols);
    if (weight_dtype == BLOCK_FP16)
        return launch(layer_norm_partials_kernel<DT_F16>, grid, dim3(1024), 0, stream, part, gw, gb, parts, (int)cols);
    return launch(layer_norm_partials_kernel<DT_F32>, grid, dim3(1024), 0, stream, part, gw, gb, parts, (int)cols);
}

}  // extern "C"
