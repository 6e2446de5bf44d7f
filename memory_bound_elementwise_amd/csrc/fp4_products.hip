// Products with weights in 4 bits (layout in fp4.h), for AMD Instinct MI355X (gfx950): y = act(x
// W^T + bias) + residual, and the expert layer of a few tokens. C ABI declared in
// block/moe_block.h.
//
// For a few rows of x the cost is reading W once. A wave reads tiles of 16 rows x 128 k in whole,
// straight into the registers from which the matrix instructions take them; a workgroup's waves
// split k, and their sums meet in shared memory.
//   linear  one workgroup 16 rows of W
//   up      one workgroup a (chosen expert, 16 columns of the activation); the activation times the
//           probability goes to the workspace as three bf16 terms, which keep its 24 bits
//   down    one workgroup a (chosen expert, 16 columns of the output); the terms are columns of
//           their own, and a pair's fp32 products go to the workspace
//   combine adds a token's pairs in slot order, so no atomics are needed and the bits never change
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "fp4.h"
#include "fp4_host.h"
#include "route_device.h"

namespace {

using namespace block;

// Offset of a lane that reads nothing: past the end of every resource, so the load returns zeros
// (tensors of these products stay below 2^31 bytes a resource).
constexpr uint32_t kNowhere = 0x80000000u;

constexpr int kWaves = 4;

// One matrix's row blocks for a wave: W's tiles and their scales.
struct Tiles {
    rsrc_t codes, scales;
};

__device__ __forceinline__ Tiles tiles_of(const uint8_t *codes, const uint8_t *scales, int64_t block, int k_tiles)
{
    return {make_rsrc(codes + block * k_tiles * kFp4Codes, (uint32_t)k_tiles * kFp4Codes),
            make_rsrc(scales + block * k_tiles * kFp4Scales, (uint32_t)k_tiles * kFp4Scales)};
}

// acc[i][g] += 16 rows of W (w[i]) times 16 columns (group g), over the k tiles first, first +
// stride, ... x: resource of the columns; col[g]: where column lane % 16 of the group starts in
// it, plus 16 (lane / 16) bytes, or kNowhere.
template <int RT, int G>
__device__ __forceinline__ void stream_products(f32x4 (&acc)[RT][G], const Tiles (&w)[RT], rsrc_t x,
                                                const uint32_t (&col)[G], int K, int first, int stride)
{
    struct Buf {
        u32x4 codes[RT], x[G][4];
        uint32_t scales[RT];
    };
    const int lane = lane_id(), k_tiles = (K + kFp4K - 1) / kFp4K;
    auto fetch = [&](Buf &buf, int t) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {  // a tile past the last reads zeros
            buf.codes[i] = __builtin_amdgcn_raw_buffer_load_b128(w[i].codes, lane * 16, t * kFp4Codes, kLoadAux);
            buf.scales[i] = __builtin_amdgcn_raw_buffer_load_b32(w[i].scales, lane % 16 * 4, t * kFp4Scales, 0);
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = t * kFp4K + j * 32;
                buf.x[g][j] = __builtin_amdgcn_raw_buffer_load_b128(x, k < K ? col[g] : kNowhere, k * 2, 0);
            }
    };
    auto multiply = [&](const Buf &buf) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const u32x4 a = fp4_widen(buf.codes[i][j], fp4_scale(buf.scales[i], j));
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[i][g] = mfma16<DT_BF16>(a, buf.x[g][j], acc[i][g]);
            }
    };
    Buf even, odd;
    fetch(even, first);
    for (int t = first; t < k_tiles; t += 2 * stride) {
        fetch(odd, t + stride);
        multiply(even);
        fetch(even, t + 2 * stride);
        multiply(odd);
    }
}

template <int RT, int G>
__device__ __forceinline__ void clear(f32x4 (&acc)[RT][G])
{
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g)
            acc[i][g] = f32x4{0, 0, 0, 0};
}

// The waves' sums, joined in order: joined[wave][i][g][lane], a barrier on each side.
template <int RT, int G>
__device__ __forceinline__ void share_sums(const f32x4 (&acc)[RT][G], f32x4 *joined)
{
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g)
            joined[((wave_in_block() * RT + i) * G + g) * 64 + lane_id()] = acc[i][g];
    __syncthreads();
}

// Row `row` of tile i times column c of group g.
template <int RT, int G>
__device__ __forceinline__ float joined_sum(const f32x4 *joined, int i, int g, int row, int c)
{
    float z = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        z += joined[((w * RT + i) * G + g) * 64 + row / 4 * 16 + c][row % 4];
    return z;
}

// ---------------------------------------------------------------------------
// Product with an epilogue
// ---------------------------------------------------------------------------
struct LinearArgs {
    const uint16_t *x;
    const uint8_t *codes, *scales;
    const uint16_t *bias, *residual;
    uint16_t *y;
    int m, n, k, act;
};

template <int G>
__global__ __launch_bounds__(kWaves * 64) void fp4_linear_kernel(LinearArgs a)
{
    __shared__ f32x4 joined[kWaves * G * 64];
    const int lane = lane_id(), k_tiles = (a.k + kFp4K - 1) / kFp4K;
    const Tiles w[1] = {tiles_of(a.codes, a.scales, blockIdx.x, k_tiles)};
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.m * (uint32_t)a.k * 2u);
    uint32_t col[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int row = g * 16 + lane % 16;
        col[g] = row < a.m ? (uint32_t)row * (uint32_t)a.k * 2u + lane / 16 * 16 : kNowhere;
    }
    f32x4 acc[1][G];
    clear(acc);
    stream_products<1, G>(acc, w, x, col, a.k, wave_in_block(), kWaves);
    share_sums(acc, joined);
    for (int i = threadIdx.x; i < G * 256; i += kWaves * 64) {
        const int c = i % 16, row = i / 16, col_n = blockIdx.x * 16 + c;
        if (row >= a.m || col_n >= a.n)
            continue;
        float z = joined_sum<1, G>(joined, 0, row / 16, c, row % 16);
        if (a.bias)
            z += load1<DT_BF16>(a.bias, col_n);
        z = activate(a.act, z);
        const int64_t at = (int64_t)row * a.n + col_n;
        if (a.residual)
            z += load1<DT_BF16>(a.residual, at);
        store1<DT_BF16>(a.y, at, z);
    }
}

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------
struct ExpertArgs {
    const uint16_t *x;
    const uint8_t *up_codes, *up_scales, *down_codes, *down_scales;
    const int *ids;
    const float *probs;
    const uint16_t *residual;
    char *y;
    const int *valid;
    uint16_t *h;  // [3][pairs][inter]
    float *z;     // [pairs][hidden]
    int tokens, hidden, inter, experts, top_k, by_pair;
    float limit;
};

// An fp32 value as the sum of three bf16: its first 8 bits, the next 8 and the rest (nothing is
// lost, but below 2^-109, where the last term runs out of exponents). Of an infinity or a NaN the
// first term is one and the others zero.
__device__ __forceinline__ void three_terms(float h, uint16_t (&term)[3])
{
    const uint32_t bits = __float_as_uint(h);
    const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
    const float first = __uint_as_float(bits & 0xffff0000u), rest = h - first;
    const float second = __uint_as_float(__float_as_uint(rest) & 0xffff0000u), third = rest - second;
    term[0] = (uint16_t)(bits >> 16) | (h != h ? 0x40 : 0);
    term[1] = finite ? (uint16_t)(__float_as_uint(second) >> 16) : 0;
    term[2] = finite ? (uint16_t)(__float_as_uint(third) >> 16) : 0;
}

// The workgroup's expert (blockIdx.y: a pair, which stands for its expert if no earlier one has
// the same, or an expert, whichever is fewer) and its pairs; returns their number.
__device__ __forceinline__ int expert_pairs(const ExpertArgs &a, int pairs, int &e, uint16_t *list, int &count)
{
    e = blockIdx.y;
    if (a.by_pair) {
        if (e >= pairs)
            return 0;
        e = a.ids[e];
        if (e < 0 || e >= a.experts)
            return 0;
    }
    if (wave_in_block() == 0) {
        const int n = list_pairs(a.ids, pairs, e, list);
        if (lane_id() == 0)
            count = n;
    }
    __syncthreads();
    const int n = count;
    return n == 0 || (a.by_pair && list[0] != (int)blockIdx.y) ? 0 : n;
}

template <int ACT, int G>
__device__ __forceinline__ void up_pass(const ExpertArgs &a, int e, const uint16_t *list, int n, f32x4 *joined)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;  // gate and up, or the one product
    const int lane = lane_id(), k_tiles = (a.hidden + kFp4K - 1) / kFp4K, blocks = a.inter / 16;
    Tiles w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        w[i] = tiles_of(a.up_codes, a.up_scales, ((int64_t)e * RT + i) * blocks + blockIdx.x, k_tiles);
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.hidden * 2u);
    uint32_t col[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 16 + lane % 16;
        col[g] = s < n ? (uint32_t)(list[s] / a.top_k) * (uint32_t)a.hidden * 2u + lane / 16 * 16 : kNowhere;
    }
    f32x4 acc[RT][G];
    clear(acc);
    stream_products<RT, G>(acc, w, x, col, a.hidden, wave_in_block(), kWaves);
    share_sums(acc, joined);
    const int64_t plane = (int64_t)a.tokens * a.top_k * a.inter;
    for (int i = threadIdx.x; i < G * 256; i += kWaves * 64) {
        const int row = i % 16, s = i / 16;
        if (s >= n)
            continue;
        float z[RT];
#pragma unroll
        for (int q = 0; q < RT; ++q)
            z[q] = joined_sum<RT, G>(joined, q, s / 16, row, s % 16);
        const int pair = list[s];
        uint16_t term[3];
        three_terms((ACT == ACT_SWIGLU ? swiglu(z[0], z[RT - 1], a.limit) : squared_relu(z[0])) * a.probs[pair], term);
        uint16_t *to = a.h + (int64_t)pair * a.inter + blockIdx.x * 16 + row;
#pragma unroll
        for (int q = 0; q < 3; ++q)
            to[q * plane] = term[q];
    }
}

// G: groups of 16 tokens that share one read of the weights; an expert with more tokens reads
// them again.
template <int ACT, int G>
__global__ __launch_bounds__(kWaves * 64) void fp4_up_kernel(ExpertArgs a)
{
    __shared__ f32x4 joined[kWaves * 2 * G * 64];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k;
    int e;
    const int n = expert_pairs(a, pairs, e, list, count);
    for (int p = 0; p < n; p += G * 16) {
        const int m = n - p < G * 16 ? n - p : G * 16;
        if (G == 1 || m <= 16)
            up_pass<ACT, 1>(a, e, list + p, m, joined);
        else if (G == 2 || m <= 32)
            up_pass<ACT, G < 2 ? 1 : 2>(a, e, list + p, m, joined);
        else
            up_pass<ACT, G>(a, e, list + p, m, joined);
    }
}

// A group holds the three terms of five pairs, columns 3 p + 0 .. 2.
constexpr int kPairs = 5;

template <int G>
__device__ __forceinline__ void down_pass(const ExpertArgs &a, int e, const uint16_t *list, int n, f32x4 *joined)
{
    const int lane = lane_id(), k_tiles = (a.inter + kFp4K - 1) / kFp4K;
    const Tiles w[1] = {tiles_of(a.down_codes, a.down_scales, (int64_t)e * (a.hidden / 16) + blockIdx.x, k_tiles)};
    const uint32_t pairs = (uint32_t)(a.tokens * a.top_k), row_bytes = (uint32_t)a.inter * 2u;
    const rsrc_t h = make_rsrc(a.h, 3u * pairs * row_bytes);
    uint32_t col[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int c = lane % 16, s = g * kPairs + c / 3;
        col[g] = c < 15 && s < n ? ((uint32_t)(c % 3) * pairs + list[s]) * row_bytes + lane / 16 * 16 : kNowhere;
    }
    f32x4 acc[1][G];
    clear(acc);
    stream_products<1, G>(acc, w, h, col, a.inter, wave_in_block(), kWaves);
    share_sums(acc, joined);
    for (int i = threadIdx.x; i < G * kPairs * 16; i += kWaves * 64) {
        const int row = i % 16, s = i / 16;
        if (s >= n)
            continue;
        float z = 0.0f;
#pragma unroll
        for (int q = 0; q < 3; ++q)
            z += joined_sum<1, G>(joined, 0, s / kPairs, row, s % kPairs * 3 + q);
        a.z[(int64_t)list[s] * a.hidden + blockIdx.x * 16 + row] = z;
    }
}

template <int G>
__global__ __launch_bounds__(kWaves * 64) void fp4_down_kernel(ExpertArgs a)
{
    __shared__ f32x4 joined[kWaves * G * 64];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k;
    int e;
    const int n = expert_pairs(a, pairs, e, list, count);
    for (int p = 0; p < n; p += G * kPairs) {
        const int m = n - p < G * kPairs ? n - p : G * kPairs;
        if (G == 1 || m <= kPairs)
            down_pass<1>(a, e, list + p, m, joined);
        else if (G == 2 || m <= 2 * kPairs)
            down_pass<G < 2 ? 1 : 2>(a, e, list + p, m, joined);
        else
            down_pass<G>(a, e, list + p, m, joined);
    }
}

// y = residual + a token's products in slot order. A lane takes four neighbouring columns.
template <int YDT>
__global__ __launch_bounds__(256) void fp4_combine_kernel(ExpertArgs a)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= (int64_t)live_tokens(a.valid, a.tokens) * a.hidden)
        return;
    const int t = (int)(i / a.hidden), c = (int)(i % a.hidden);
    f32x4 v = {0, 0, 0, 0};
    for (int j = 0; j < a.top_k; ++j) {
        const int pair = t * a.top_k + j, e = a.ids[pair];
        if (e >= 0 && e < a.experts)
            v += *reinterpret_cast<const f32x4 *>(a.z + (int64_t)pair * a.hidden + c);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float o = v[q];
        if (a.residual)
            o += load1<DT_BF16>(a.residual, i + q);
        store1<YDT>(a.y, i + q, o);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int kFewRows = 64;

bool good_linear(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && m <= (1 << 24) && n >= 8 && k >= 32 && n <= (1 << 20) && k <= (1 << 20) &&
           n * k <= ((int64_t)1 << 36) && m * n <= ((int64_t)1 << 36) && m * k <= ((int64_t)1 << 36);
}

struct ExpertSizes {
    int64_t tokens, hidden, inter;
    int experts, top_k;
};

block_status_t check_experts(const ExpertSizes &s, block_act_t act, float limit)
{
    if (s.tokens < 0 || s.hidden < 32 || s.inter < 32 || s.hidden > (1 << 16) || s.inter > (1 << 16) || s.experts < 1 ||
        s.experts > kMaxExperts || s.top_k < 1 || s.top_k > kMaxPairs || s.tokens > kMaxPairs ||
        s.tokens * s.top_k > kMaxPairs)
        return BLOCK_ERR_INVALID_ARG;
    if (act != BLOCK_ACT_SWIGLU && act != BLOCK_ACT_SQUARED_RELU)
        return BLOCK_ERR_INVALID_ARG;
    if (act == BLOCK_ACT_SWIGLU && !(limit > 0.0f))
        return BLOCK_ERR_INVALID_ARG;
    if (s.hidden % 32 || s.inter % 32)
        return BLOCK_ERR_ALIGNMENT;
    return BLOCK_OK;
}

// Workspace: the activations' terms, then the pairs' products.
int64_t h_bytes(const ExpertSizes &s) { return round_up(s.tokens * s.top_k * s.inter * 6, 16); }
int64_t expert_bytes(const ExpertSizes &s) { return h_bytes(s) + s.tokens * s.top_k * s.hidden * 4; }

// Groups of pairs that share a read of an expert's weights: enough for one and a half times the
// pairs an expert has on average.
int pair_groups(const ExpertSizes &s, int group)
{
    const int64_t some = ceil_div(3 * s.tokens * s.top_k, 2 * s.experts);
    const int64_t each = s.tokens < some ? s.tokens : some;
    return each <= group ? 1 : (each <= 2 * group ? 2 : 4);
}

template <int ACT>
block_status_t launch_up(const ExpertArgs &a, int groups, dim3 grid, hipStream_t st)
{
    const dim3 threads(kWaves * 64);
    if (groups == 1)
        return launch(fp4_up_kernel<ACT, 1>, grid, threads, 0, st, a);
    if (groups == 2)
        return launch(fp4_up_kernel<ACT, 2>, grid, threads, 0, st, a);
    return launch(fp4_up_kernel<ACT, 4>, grid, threads, 0, st, a);
}

block_status_t launch_down(const ExpertArgs &a, int groups, dim3 grid, hipStream_t st)
{
    const dim3 threads(kWaves * 64);
    if (groups == 1)
        return launch(fp4_down_kernel<1>, grid, threads, 0, st, a);
    if (groups == 2)
        return launch(fp4_down_kernel<2>, grid, threads, 0, st, a);
    return launch(fp4_down_kernel<4>, grid, threads, 0, st, a);
}

}  // namespace

extern "C" {

int64_t block_linear_act_fp4_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!good_linear(m, n, k) || k % 32 || n % 8 || m <= kFewRows)
        return 0;
    return round_up(n * k * 2, 16) + block_linear_act_workspace(m, n, k);
}

block_status_t block_linear_act_fp4(const uint16_t *x, const uint8_t *codes, const uint8_t *scales, const uint16_t *bias,
                                    const uint16_t *residual, uint16_t *y, int64_t m, int64_t n, int64_t k,
                                    block_act_t act, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (!good_linear(m, n, k) || act < BLOCK_ACT_NONE || act > BLOCK_ACT_SQUARED_RELU)
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
    const LinearArgs a = {x, codes, scales, bias, residual, y, (int)m, (int)n, (int)k, act};
    const dim3 grid((unsigned)s.row_tiles()), threads(kWaves * 64);
    if (m <= 16)
        return launch(fp4_linear_kernel<1>, grid, threads, 0, stream, a);
    if (m <= 32)
        return launch(fp4_linear_kernel<2>, grid, threads, 0, stream, a);
    return launch(fp4_linear_kernel<4>, grid, threads, 0, stream, a);
}

int64_t block_moe_experts_fp4_workspace(int64_t tokens, int64_t hidden, int64_t inter, int n_experts, int top_k)
{
    const ExpertSizes s = {tokens, hidden, inter, n_experts, top_k};
    return check_experts(s, BLOCK_ACT_SQUARED_RELU, 0.0f) == BLOCK_OK ? expert_bytes(s) : 0;
}

block_status_t block_moe_experts_fp4(const uint16_t *x, const uint8_t *up_codes, const uint8_t *up_scales,
                                     const uint8_t *down_codes, const uint8_t *down_scales, const int32_t *ids,
                                     const float *probs, const uint16_t *residual, void *y, block_dtype_t y_dtype,
                                     int64_t tokens, int64_t hidden, int64_t inter, int n_experts, int top_k,
                                     block_act_t act, float limit, const int32_t *valid_tokens, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream)
{
    const ExpertSizes s = {tokens, hidden, inter, n_experts, top_k};
    if (const block_status_t r = check_experts(s, act, limit))
        return r;
    if (y_dtype != BLOCK_BF16 && y_dtype != BLOCK_FP32)
        return BLOCK_ERR_INVALID_ARG;
    if (tokens == 0)
        return BLOCK_OK;
    const int64_t need = expert_bytes(s);
    if (!x || !up_codes || !up_scales || !down_codes || !down_scales || !ids || !probs || !y || !workspace ||
        workspace_bytes < need)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(up_codes, 16) || misaligned(up_scales, 16) || misaligned(down_codes, 16) ||
        misaligned(down_scales, 16) || misaligned(residual, 16) || misaligned(y, 16) || misaligned(ids, 4) ||
        misaligned(probs, 4) || misaligned(valid_tokens, 4) || misaligned(workspace, 16))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t n = tokens * hidden;
    const Fp4Shape up = {n_experts, act == BLOCK_ACT_SWIGLU ? 2 * inter : inter, hidden}, down = {n_experts, hidden, inter};
    if (any_overlap<2, 9>({{y, n * (y_dtype == BLOCK_FP32 ? 4 : 2)}, {workspace, need}},
                          {{x, n * 2},
                           {up_codes, up.codes()},
                           {up_scales, up.scales()},
                           {down_codes, down.codes()},
                           {down_scales, down.scales()},
                           {ids, tokens * top_k * 4},
                           {probs, tokens * top_k * 4},
                           {residual, n * 2},
                           {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    ExpertArgs a = {};
    a.x = x, a.up_codes = up_codes, a.up_scales = up_scales, a.down_codes = down_codes, a.down_scales = down_scales;
    a.ids = ids, a.probs = probs, a.residual = residual, a.y = static_cast<char *>(y), a.valid = valid_tokens;
    a.h = static_cast<uint16_t *>(workspace);
    a.z = reinterpret_cast<float *>(static_cast<char *>(workspace) + h_bytes(s));
    a.tokens = (int)tokens, a.hidden = (int)hidden, a.inter = (int)inter, a.experts = n_experts, a.top_k = top_k;
    a.limit = limit;
    const int64_t pairs = tokens * top_k;
    a.by_pair = pairs < n_experts;
    const unsigned each = (unsigned)(a.by_pair ? pairs : n_experts);
    const dim3 up_grid((unsigned)(inter / 16), each), down_grid((unsigned)(hidden / 16), each);
    const int groups = pair_groups(s, 16);
    if (const block_status_t r = act == BLOCK_ACT_SWIGLU ? launch_up<ACT_SWIGLU>(a, groups, up_grid, stream)
                                                         : launch_up<ACT_SQUARED_RELU>(a, groups, up_grid, stream))
        return r;
    if (const block_status_t r = launch_down(a, pair_groups(s, kPairs), down_grid, stream))
        return r;
    const dim3 all((unsigned)ceil_div(n, 1024));
    return y_dtype == BLOCK_FP32 ? launch(fp4_combine_kernel<DT_F32>, all, dim3(256), 0, stream, a)
                                 : launch(fp4_combine_kernel<DT_BF16>, all, dim3(256), 0, stream, a);
}

}  // extern "C"
