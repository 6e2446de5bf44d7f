// The router and the expert products of a few tokens, for AMD Instinct MI355X (gfx950).
// C ABI declared in block/moe_block.h.
//
// For a few tokens the cost is reading each chosen expert's weights once. Two kernels:
//   up    one workgroup a (chosen expert, 16 columns of the activation): its waves split the
//         hidden axis, the activation and the probability are applied to the joined sums,
//         and h goes to the workspace in fp32.
//   down  one workgroup 16 columns of the output: its waves take the chosen experts in turn
//         and leave each (token, slot)'s 16 values in LDS; a token's values are then added in
//         slot order, so no atomics are needed and the bits never change.
// A workgroup finds its experts and their tokens in ids itself: at most 1024 entries.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "block_host.h"
#include "gate.h"
#include "route_device.h"
#include "weight_stream.h"

namespace {

using namespace block;

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kRouteTile = 16;   // tokens and experts of a workgroup's tile
constexpr int kRouteStep = 32;   // k of one load: four octets, one a group of 16 lanes
constexpr int kRouteWaves = 16;  // waves that share a part of k

// partial[part][t][e]: a workgroup's tile of 16 tokens x 16 experts over one part of k, on the
// fp64 matrix cores. Products of two bf16 (or a bf16 and an fp32) are exact in fp64 and the
// sums are fp64. A lane loads octet lane / 16 of its row; the eight instructions that follow
// take one element of each lane's octet, so that k runs in the same order on both sides.
template <int RDT>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_kernel(const char *x, const char *router,
                                                                        double *partial, int tokens, int hidden,
                                                                        int experts, int part_k, const int *valid)
{
    __shared__ double joined[kRouteWaves][4][64];
    const int lane = lane_id(), wave = wave_in_block(), i = lane % 16, k8 = lane / 16 * 8;
    const int t0 = blockIdx.y * kRouteTile, e0 = blockIdx.x * kRouteTile;
    if (t0 >= live_tokens(valid, tokens))
        return;
    // past the last row: the last one again, not stored
    const int t = t0 + i < tokens ? t0 + i : tokens - 1, e = e0 + i < experts ? e0 + i : experts - 1;
    const char *xr = x + (int64_t)t * hidden * 2, *wr = router + (int64_t)e * hidden * kSize<RDT>;
    const int first = blockIdx.z * part_k, last = first + part_k < hidden ? first + part_k : hidden;
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
    constexpr int kAhead = 4;  // steps whose loads go out together
    for (int k = first + wave * kRouteStep; k < last; k += kAhead * kRouteWaves * kRouteStep) {
        Raw8<DT_BF16> xa[kAhead];
        Raw8<RDT> wa[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int at = k + u * kRouteWaves * kRouteStep + k8;
            const int from = at < last ? at : 0;
            xa[u].v[0] = *reinterpret_cast<const u32x4 *>(xr + from * 2);
#pragma unroll
            for (int v = 0; v < kSize<RDT> / 2; ++v)
                wa[u].v[v] = reinterpret_cast<const u32x4 *>(wr + (int64_t)from * kSize<RDT>)[v];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int at = k + u * kRouteWaves * kRouteStep;
            if (at >= last)
                break;
            if (at + kRouteStep > last && at + k8 >= last) {  // an octet past the part read the row's first: zeros
                xa[u] = Raw8<DT_BF16>{};
                wa[u] = Raw8<RDT>{};
            }
            float a[8], b[8];
            widen8<DT_BF16>(xa[u], a);
            widen8<RDT>(wa[u], b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)b[j], (double)a[j], acc, 0, 0, 0);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        joined[wave][r][lane] = acc[r];
    __syncthreads();
    // element r of lane l: expert 4 r + l / 16 of the tile, token l % 16; wave r finishes it
    if (wave >= 4)
        return;
    const int c = 4 * wave + lane / 16;
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w)
        sum += joined[w][wave][lane];
    if (t0 + i < tokens && e0 + c < experts)
        partial[((int64_t)blockIdx.z * tokens + t0 + i) * experts + e0 + c] = sum;
}

// The same for up to kRouteFew tokens, where a matrix instruction of 16 would idle: the octet's
// products in the vector unit, the four octets of an expert joined across the wave.
constexpr int kRouteFew = 4;

template <int RDT>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_few_kernel(const char *x, const char *router,
                                                                            double *partial, int tokens, int hidden,
                                                                            int experts, int part_k, const int *valid)
{
    __shared__ double joined[kRouteWaves][kRouteFew][16];
    const int lane = lane_id(), wave = wave_in_block(), i = lane % 16, k8 = lane / 16 * 8;
    const int e0 = blockIdx.x * kRouteTile, live = live_tokens(valid, tokens);
    if (live == 0)
        return;
    const int e = e0 + i < experts ? e0 + i : experts - 1;  // past the last: the last one again, not stored
    const char *wr = router + (int64_t)e * hidden * kSize<RDT>;
    const int first = blockIdx.z * part_k, last = first + part_k < hidden ? first + part_k : hidden;
    double acc[kRouteFew] = {};
    constexpr int kAhead = 2;  // steps whose loads go out together
    for (int k = first + wave * kRouteStep; k < last; k += kAhead * kRouteWaves * kRouteStep) {
        Raw8<DT_BF16> xa[kAhead][kRouteFew];
        Raw8<RDT> wa[kAhead];
        bool in[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int at = k + u * kRouteWaves * kRouteStep + k8;
            in[u] = at < last;  // an octet past the part: the row's first instead, not counted
            const int from = in[u] ? at : 0;
#pragma unroll
            for (int v = 0; v < kSize<RDT> / 2; ++v)
                wa[u].v[v] = reinterpret_cast<const u32x4 *>(wr + (int64_t)from * kSize<RDT>)[v];
#pragma unroll
            for (int t = 0; t < kRouteFew; ++t)
                xa[u][t].v[0] = *reinterpret_cast<const u32x4 *>(x + ((int64_t)(t < live ? t : 0) * hidden + from) * 2);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (k + u * kRouteWaves * kRouteStep >= last)
                break;
            float b[8];
            widen8<RDT>(wa[u], b);
#pragma unroll
            for (int t = 0; t < kRouteFew; ++t) {
                if (t >= live)
                    break;
                float a[8];
                widen8<DT_BF16>(xa[u][t], a);
                double sum = 0.0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum = __builtin_fma((double)a[j], (double)b[j], sum);
                acc[t] += in[u] ? sum : 0.0;
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kRouteFew; ++t) {
        double v = acc[t];
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (lane < 16)
            joined[wave][t][i] = v;
    }
    __syncthreads();
    if (wave > 0)
        return;
    const int t = lane / 16;  // one token a quarter of the wave
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w)
        sum += joined[w][t][i];
    if (t < live && e0 + i < experts)
        partial[((int64_t)blockIdx.z * tokens + t) * experts + e0 + i] = sum;
}

// One workgroup a token, a thread an expert: its logit is the sum of its parts in order, its
// rank the number of experts before it (a larger logit, or an equal one and a lower index).
// Counting against all others costs less than top_k reductions over the wave one after the
// other (64 experts, top 8: 4.7 us so).
__global__ __launch_bounds__(kMaxExperts) void route_choose_kernel(const double *partial, int *ids, float *probs,
                                                                   int tokens, int experts, int parts, int top_k,
                                                                   int renormalize, const int *valid)
{
    __shared__ uint64_t keys[kMaxExperts];
    __shared__ double sums[kMaxExperts / 64];
    __shared__ int holder[kMaxExperts];
    __shared__ int tied;
    __shared__ double top;
    const int t = blockIdx.x, e = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    if (t >= live_tokens(valid, tokens))
        return;
    const double *mine = partial + (int64_t)t * experts + (e < experts ? e : 0);
    const int64_t part = (int64_t)tokens * experts;
    const double v = sum_parts(mine, part, parts);
    const uint64_t key = order_key(v);
    keys[e] = key;
    if (e == 0)
        tied = 0;
    __syncthreads();
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < experts; ++j)
        rank += keys[j] > key;
    // equal logits got one rank: whoever finds another expert there has company
    if (e < experts)
        holder[rank] = e;
    __syncthreads();
    if (e < experts && holder[rank] != e)
        tied = 1;
    __syncthreads();
    if (tied)
        for (int j = 0; j < e && j < experts; ++j)
            rank += keys[j] == key;
    if (e >= experts)
        rank = experts;
    if (rank == 0)
        top = v;
    __syncthreads();
    const double w = e < experts ? exp(v - top) : 0.0;
    double sum = wave_sum64(renormalize && rank >= top_k ? 0.0 : w);
    if (lane == 0)
        sums[wave] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < (int)blockDim.x / 64; ++i)
        sum += sums[i];
    if (rank < top_k) {
        ids[(int64_t)t * top_k + rank] = e;
        probs[(int64_t)t * top_k + rank] = (float)(w / sum);
    }
}

// The same choice by one wave for a token of up to 64 experts (the same bits): lane = expert,
// keys: 64 of the wave's own. Slots beyond top_k lanes are not written.
__device__ __forceinline__ void choose_in_wave(const double *partial, int t, int tokens, int experts, int parts,
                                               int top_k, int renormalize, uint64_t *keys, int *ids, float *probs)
{
    const int e = lane_id();
    const double *mine = partial + (int64_t)t * experts + (e < experts ? e : 0);
    const int64_t part = (int64_t)tokens * experts;
    const double v = sum_parts(mine, part, parts);
    const uint64_t key = order_key(v);
    keys[e] = key;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < experts; ++j)
        rank += keys[j] > key || (keys[j] == key && j < e);
    if (e >= experts)
        rank = experts;
    const int first = __builtin_ctzll(__ballot(rank == 0));
    const double w = e < experts ? exp(v - of_lane(v, first)) : 0.0;
    const double sum = wave_sum64(renormalize && rank >= top_k ? 0.0 : w);
    if (rank < top_k) {
        ids[t * top_k + rank] = e;
        probs[t * top_k + rank] = (float)(w / sum);
    }
}

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------
struct UpArgs {
    const uint16_t *x, *w;
    const int *ids;
    const float *probs;
    float *h;  // [pairs][inter]
    const int *valid;
    int tokens, hidden, inter, experts, top_k, by_pair;
    float limit;
    // set where the choice of experts is made here (by every workgroup for itself; the first
    // one writes it out): the router's partial logits
    const double *partial;
    int parts, renormalize;
    int *ids_out;
    float *probs_out;
};

// The choice is made in the up kernel for up to this many tokens (one a wave) and experts
// (one a lane), and workgroups of that kernel: each of them then takes about 1.5 us longer,
// against a kernel of its own of 2 to 3.6 us and its launch. (Where the workgroups come in
// several rounds they pay it in each: one token of 7168 x 2048, 1024 workgroups, +4.2 us.)
constexpr int kChooseTokens = 4, kChooseExperts = 64, kChooseGroups = 512;

constexpr int kUpWaves = 4;

template <int ACT, int G>
__device__ __forceinline__ void up_pass(const UpArgs &a, const float *probs, int e, int i0, const uint16_t *list, int n,
                                        u32x4 *shared)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;  // gate and up, or the one product
    const int lane = lane_id(), wave = wave_in_block();
    const int there = a.inter - i0 < 16 ? a.inter - i0 : 16;
    const uint32_t row_bytes = (uint32_t)a.hidden * 2u;
    rsrc_t w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        w[r] = make_rsrc(a.w + (((int64_t)e * RT + r) * a.inter + i0) * a.hidden, (uint32_t)there * row_bytes);
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.tokens * row_bytes);
    uint32_t col[2 * G];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int s = g * 16 + p * 8 + lane / 8;
            col[2 * g + p] = s < n ? (uint32_t)(list[s] / a.top_k) * row_bytes + lane % 8 * 16 : kNowhere;
        }
    f32x4 acc[RT][G];
    clear(acc);
    stream_products<DT_BF16, RT, G, false>(acc, w, row_bytes, x, col, a.hidden, wave * kLineK,
                                           kUpWaves * kLineK, shared + wave * kStage<RT, G, false>);
    __syncthreads();  // the sums take the place of the stages
    f32x4 *joined = reinterpret_cast<f32x4 *>(shared);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < G; ++g)
            joined[((wave * RT + r) * G + g) * 64 + lane] = acc[r][g];
    __syncthreads();
    // wave q finishes element q of each lane's four
    const int i = i0 + lane / 16 * 4 + wave;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float z[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            z[r] = 0.0f;
#pragma unroll
            for (int q = 0; q < kUpWaves; ++q)
                z[r] += joined[((q * RT + r) * G + g) * 64 + lane][wave];
        }
        const int s = g * 16 + lane % 16;
        if (s < n && i < a.inter) {
            const int pair = list[s];
            const float v = (ACT == ACT_SWIGLU ? swiglu(z[0], z[RT - 1], a.limit) : squared_relu(z[0])) * probs[pair];
            a.h[(int64_t)pair * a.inter + i] = v + 0.0f;  // no -0: three_terms
        }
    }
    __syncthreads();
}

// blockIdx.y: a pair (by_pair: it stands for its expert if no earlier pair has the same), or
// an expert, whichever is fewer. G: groups of 16 tokens that share one read of the weights;
// an expert with more tokens reads them again.
template <int ACT, int G, bool CHOOSE>
__global__ __launch_bounds__(kUpWaves * 64) void moe_up_kernel(UpArgs a)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;
    __shared__ u32x4 shared[kUpWaves * kStage<RT, G, false>];  // the waves' stages, then their sums
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    const int live = live_tokens(a.valid, a.tokens), pairs = live * a.top_k;
    const int *ids = a.ids;
    const float *probs = a.probs;
    if constexpr (CHOOSE) {
        __shared__ uint64_t keys[kChooseTokens][64];
        __shared__ int chosen[kChooseTokens * 64];
        __shared__ float weights[kChooseTokens * 64];
        static_assert(kChooseTokens == kUpWaves, "a token a wave");
        const int t = wave_in_block();
        if (t < live)
            choose_in_wave(a.partial, t, a.tokens, a.experts, a.parts, a.top_k, a.renormalize, keys[t], chosen, weights);
        __syncthreads();
        if (blockIdx.x == 0 && blockIdx.y == 0 && (int)threadIdx.x < pairs) {
            a.ids_out[threadIdx.x] = chosen[threadIdx.x];
            a.probs_out[threadIdx.x] = weights[threadIdx.x];
        }
        ids = chosen;
        probs = weights;
    }
    int e = blockIdx.y;
    if (a.by_pair) {
        if (e >= pairs)
            return;
        e = ids[e];
        if (e < 0 || e >= a.experts)
            return;
    }
    if (wave_in_block() == 0) {
        const int n = list_pairs(ids, pairs, e, list);
        if (lane_id() == 0)
            count = n;
    }
    __syncthreads();
    const int n = count;
    if (n == 0 || (a.by_pair && list[0] != (int)blockIdx.y))
        return;
    const int i0 = blockIdx.x * 16;
    for (int p = 0; p < n; p += G * 16) {
        const int m = n - p < G * 16 ? n - p : G * 16;
        if (G == 1 || m <= 16)
            up_pass<ACT, 1>(a, probs, e, i0, list + p, m, shared);
        else if (G == 2 || m <= 32)
            up_pass<ACT, G < 2 ? 1 : 2>(a, probs, e, i0, list + p, m, shared);
        else
            up_pass<ACT, G>(a, probs, e, i0, list + p, m, shared);
    }
}

struct DownArgs {
    const float *h;  // [pairs][inter]
    const uint16_t *w, *residual;
    const int *ids;
    char *y;
    const int *valid;
    int tokens, hidden, inter, experts, top_k, parts;
};

template <int YDT>
__device__ __forceinline__ void finish_row(const DownArgs &a, int64_t at, float v)
{
    if (a.residual)
        v += load1<DT_BF16>(a.residual, at);
    store1<YDT>(a.y, at, v);
}

// Waves of a workgroup of the down products: fewer where their stages in shared memory are larger.
template <int G>
constexpr int kDownWaves = G == 4 ? 4 : 8;

// A lane's columns of h: load i of the wave that is `wave`-th of SHARE takes pairs 4 (wave + i SHARE) ..+4.
template <int LOADS>
__device__ __forceinline__ void h_columns(const DownArgs &a, const uint16_t *list, int n, int wave, int share,
                                          uint32_t (&col)[LOADS])
{
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int s = (wave + i * share) * 4 + lane / 16;
        col[i] = s < n ? (uint32_t)list[s] * (uint32_t)a.inter * 4u + lane % 16 * 16 : kNowhere;
    }
}

// A group is 8 pairs, whose products take two columns each (stream_products), joined after the sums.
template <int G>
__device__ __forceinline__ void down_pass(const DownArgs &a, const rsrc_t (&w)[1], const uint16_t *list, int n, int part,
                                          float *sums, u32x4 *stage)
{
    const int lane = lane_id();
    const rsrc_t h = make_rsrc(a.h, (uint32_t)(a.tokens * a.top_k) * (uint32_t)a.inter * 4u);
    uint32_t col[2 * G];
    h_columns(a, list, n, 0, 1, col);
    f32x4 acc[1][G];
    clear(acc);
    stream_products<DT_BF16, 1, G, true>(acc, w, (uint32_t)a.inter * 2u, h, col, a.inter, part * kLineK,
                                         a.parts * kLineK, stage);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        f32x4 v = acc[0][g];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[r] += dpp<0x128>(v[r]);  // row_ror:8: the other column of the pair
        const int s = g * 8 + lane % 8;
        if (s < n && lane % 16 < 8)
            *reinterpret_cast<f32x4 *>(sums + (list[s] * a.parts + part) * 16 + lane / 16 * 4) = v;
    }
}

template <int YDT, int G>
__global__ __launch_bounds__(kDownWaves<G> * 64) void moe_down_kernel(DownArgs a)
{
    constexpr int W = kDownWaves<G>;
    extern __shared__ f32x4 dynamic[];  // [pairs][parts][16] fp32
    __shared__ int ids[kMaxPairs];
    __shared__ uint16_t lists[W][kMaxPairs];
    __shared__ u32x4 stages[W * kStage<1, G, true>];
    float *sums = reinterpret_cast<float *>(dynamic);
    const int wave = wave_in_block(), tid = threadIdx.x;
    const int live = live_tokens(a.valid, a.tokens), pairs = live * a.top_k;
    for (int p = tid; p < pairs; p += W * 64) {
        const int e = a.ids[p];
        ids[p] = e >= 0 && e < a.experts ? e : -1;
    }
    __syncthreads();
    const int c0 = blockIdx.x * 16;
    const int there = a.hidden - c0 < 16 ? a.hidden - c0 : 16;
    uint16_t *list = lists[wave];
    // a pair stands for its expert if no earlier pair has the same
    for (int u = wave; u < pairs * a.parts; u += W) {
        const int p = u / a.parts, part = u % a.parts;
        const int e = __builtin_amdgcn_readfirstlane(ids[p]);
        if (e < 0)
            continue;
        const int n = list_pairs(ids, pairs, e, list);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (__builtin_amdgcn_readfirstlane(list[0]) != p)
            continue;
        const rsrc_t w[1] = {
            make_rsrc(a.w + ((int64_t)e * a.hidden + c0) * a.inter, (uint32_t)there * (uint32_t)a.inter * 2u)};
        u32x4 *stage = stages + wave * kStage<1, G, true>;
        for (int q = 0; q < n; q += G * 8) {
            const int m = n - q < G * 8 ? n - q : G * 8;
            if (G == 1 || m <= 8)
                down_pass<1>(a, w, list + q, m, part, sums, stage);
            else if (G == 2 || m <= 16)
                down_pass<G < 2 ? 1 : 2>(a, w, list + q, m, part, sums, stage);
            else
                down_pass<G>(a, w, list + q, m, part, sums, stage);
        }
    }
    __syncthreads();
    for (int i = tid; i < live * 16; i += W * 64) {
        const int t = i / 16, c = c0 + i % 16;
        if (c >= a.hidden)
            continue;
        float v = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int p = t * a.top_k + j;
            if (ids[p] < 0)
                continue;
            for (int s = 0; s < a.parts; ++s)
                v += sums[(p * a.parts + s) * 16 + i % 16];
        }
        finish_row<YDT>(a, (int64_t)t * a.hidden + c, v);
    }
}

// The down product where the chosen experts' tokens are many: h (fp32, every pair's) is
// then as large a stream as the weights if each workgroup of 16 columns reads all of it. Here
// a wave takes 32 columns, a workgroup of four or eight waves 128 or 256 of them and every
// gridDim.y-th chosen expert; the waves walk the same h together and share its loads where an
// expert has more than eight tokens (stream_products). A wave adds up all its experts' products
// in its own LDS rows, in the order of their first pair, and writes one partial row of y a
// token; moe_combine_kernel adds the shares in order.
constexpr int kManyTokens = 128, kManyPairs = 128;
constexpr int kManyWaves = 1024;
constexpr int kManyTiles = 2, kManyCols = 16 * kManyTiles;  // a wave's columns

// Rows of eight pairs' sums added to their tokens'. Slots of one token (an id that a token
// has twice) follow each other, as the list ascends.
__device__ __forceinline__ void add_to_tokens(const f32x4 &v, int token, bool live, float *mine)
{
    const int lane = lane_id();
    float *at = mine + token * kManyCols + lane / 16 * 4;
    const int before = __shfl_up(token, 1);
    const bool twice = live && lane % 16 > 0 && before == token;
    if (__ballot(twice) == 0) {
        if (live)
            *reinterpret_cast<f32x4 *>(at) += v;
        return;
    }
    for (int j = 0; j < 8; ++j) {
        if (live && lane % 16 == j)
            *reinterpret_cast<f32x4 *>(at) += v;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

template <int G, int W>
__device__ __forceinline__ void down_many_pass(const DownArgs &a, const rsrc_t (&w)[kManyTiles], const rsrc_t &h,
                                               const uint16_t *list, int n, float *mine, u32x4 *stage, u32x4 *terms,
                                               int set_chunks)
{
    const int lane = lane_id();
    constexpr int kShare = G == 1 ? 1 : W;
    uint32_t col[kOwnLoads<G, kShare>];
    h_columns(a, list, n, kShare > 1 ? wave_in_block() : 0, kShare, col);
    int token[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 8 + lane % 8;
        token[g] = list[s < n ? s : n - 1] / a.top_k;
    }
    f32x4 acc[kManyTiles][G];
    clear(acc);
    stream_products<DT_BF16, kManyTiles, G, true, kShare>(acc, w, (uint32_t)a.inter * 2u, h, col, a.inter, 0, kLineK, stage,
                                                     terms, set_chunks);
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = 0; i < kManyTiles; ++i) {
            f32x4 v = acc[i][g];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] += dpp<0x128>(v[r]);  // row_ror:8: the other column of the pair
            add_to_tokens(v, token[g], g * 8 + lane % 8 < n && lane % 16 < 8, mine + i * 16);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

template <int YDT, int G, int W>
__global__ __launch_bounds__(W * 64) void moe_down_many_kernel(DownArgs a, float *partial)
{
    extern __shared__ f32x4 dynamic[];  // [waves][tokens][kManyCols] fp32
    __shared__ int ids[kMaxPairs];
    __shared__ int first[kMaxExperts], count[kMaxExperts];
    __shared__ uint16_t units[kMaxPairs], starts[kMaxPairs], list[kMaxPairs];
    __shared__ u32x4 stages[W * kStage<kManyTiles, 1, true>], terms[G > 1 ? 2 * G * kTerms : 1];
    __shared__ int unit_count;
    u32x4 *stage = stages + wave_in_block() * kStage<kManyTiles, 1, true>;
    const int lane = lane_id(), wave = wave_in_block(), tid = threadIdx.x;
    const int live = live_tokens(a.valid, a.tokens), pairs = live * a.top_k;
    float *mine = reinterpret_cast<float *>(dynamic) + wave * a.tokens * kManyCols;
    for (int e = tid; e < a.experts; e += W * 64) {
        first[e] = kMaxPairs;
        count[e] = 0;
    }
    for (int i = lane; i < live * (kManyCols / 4); i += 64)
        reinterpret_cast<f32x4 *>(mine)[i] = f32x4{0, 0, 0, 0};
    __syncthreads();
    for (int p = tid; p < pairs; p += W * 64) {
        const int e = a.ids[p];
        const bool ok = e >= 0 && e < a.experts;
        ids[p] = ok ? e : -1;
        if (ok) {
            atomicMin(&first[e], p);
            atomicAdd(&count[e], 1);
        }
    }
    __syncthreads();
    if (wave == 0) {  // the pairs that are their expert's first, and where its list starts
        int n = 0, start = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const bool is = p < pairs && ids[p] >= 0 && first[ids[p]] == p;
            const uint64_t m = __ballot(is);
            int sum = is ? count[ids[p]] : 0;
            const int own = sum;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int up = __shfl_up(sum, d);
                sum += lane >= d ? up : 0;
            }
            if (is) {
                const int at = n + __popcll(m & (((uint64_t)1 << lane) - 1));
                units[at] = (uint16_t)p;
                starts[at] = (uint16_t)(start + sum - own);
            }
            n += __popcll(m);
            start += __shfl(sum, 63);
        }
        if (lane == 0)
            unit_count = n;
    }
    __syncthreads();
    const int n_units = unit_count, step = gridDim.y;
    for (int u = blockIdx.y + wave * step; u < n_units; u += W * step)
        list_pairs(ids, pairs, ids[units[u]], list + starts[u]);
    __syncthreads();
    const int c0 = (blockIdx.x * W + wave) * kManyCols;  // past the end: no rows of W, but its part of h
    const rsrc_t h = make_rsrc(a.h, (uint32_t)(a.tokens * a.top_k) * (uint32_t)a.inter * 4u);
    for (int u = blockIdx.y; u < n_units; u += step) {
        const int e = __builtin_amdgcn_readfirstlane(ids[units[u]]);
        const int n = __builtin_amdgcn_readfirstlane(count[e]);
        const uint16_t *l = list + starts[u];
        rsrc_t w[kManyTiles];
#pragma unroll
        for (int i = 0; i < kManyTiles; ++i) {
            const int c = c0 + 16 * i, there = a.hidden - c < 16 ? (a.hidden - c > 0 ? a.hidden - c : 0) : 16;
            w[i] = make_rsrc(a.w + ((int64_t)e * a.hidden + (there ? c : 0)) * a.inter,
                             (uint32_t)there * (uint32_t)a.inter * 2u);
        }
        for (int p = 0; p < n; p += G * 8) {
            const int m = n - p < G * 8 ? n - p : G * 8;
            if (G == 1 || m <= 8)
                down_many_pass<1, W>(a, w, h, l + p, m, mine, stage, terms, G * kTerms);
            else if (G == 2 || m <= 16)
                down_many_pass<G < 2 ? 1 : 2, W>(a, w, h, l + p, m, mine, stage, terms, G * kTerms);
            else
                down_many_pass<G, W>(a, w, h, l + p, m, mine, stage, terms, G * kTerms);
        }
    }
    for (int i = lane; i < live * kManyCols; i += 64) {
        const int t = i / kManyCols, c = c0 + i % kManyCols;
        if (c >= a.hidden)
            continue;
        const int64_t at = (int64_t)t * a.hidden + c;
        if (step > 1)
            partial[(int64_t)blockIdx.y * a.tokens * a.hidden + at] = mine[i];
        else
            finish_row<YDT>(a, at, mine[i]);
    }
}

// y = residual + the partial rows in order. A lane takes four neighbouring columns.
template <int YDT>
__global__ __launch_bounds__(256) void moe_combine_kernel(DownArgs a, const float *partial, int parts)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, all = (int64_t)a.tokens * a.hidden;
    if (i >= (int64_t)live_tokens(a.valid, a.tokens) * a.hidden)
        return;
    f32x4 v = {0, 0, 0, 0};
    for (int p = 0; p < parts; p += 2) {  // a power of two, at least 2; two loads at a time
        const f32x4 a0 = *reinterpret_cast<const f32x4 *>(partial + p * all + i);
        const f32x4 a1 = *reinterpret_cast<const f32x4 *>(partial + (p + 1) * all + i);
        v = v + a0 + a1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        finish_row<YDT>(a, i + j, v[j]);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct RouteSizes {
    int64_t tokens, hidden;
    int experts;
};

bool good_route(const RouteSizes &s)
{
    return s.tokens >= 0 && s.tokens <= (1 << 19) && s.hidden >= 8 && s.hidden <= (1 << 20) && s.experts >= 1 &&
           s.experts <= kMaxExperts && s.tokens * s.experts <= (1 << 25);
}

// k of a part, and the parts: a workgroup of 16 waves a CU, and no part shorter than two steps
// a wave. (Few parts: whoever chooses adds them up. Four waves a workgroup, so 28 parts of one
// token's 7168 x 64, took 5.1 us for that.)
int route_part(const RouteSizes &s)
{
    const int64_t tiles = ceil_div(s.tokens, kRouteTile) * ceil_div(s.experts, kRouteTile);
    const int64_t wanted = tiles < 256 ? 256 / tiles : 1;
    const int64_t k = round_up(ceil_div(s.hidden, wanted), kRouteStep);
    const int64_t least = 2 * kRouteWaves * kRouteStep;
    return (int)(k < least ? least : k);
}

int64_t route_parts(const RouteSizes &s) { return ceil_div(s.hidden, route_part(s)); }

int64_t route_bytes(const RouteSizes &s)
{
    return s.tokens > 0 ? round_up(route_parts(s) * s.tokens * s.experts * 8, 16) : 0;
}

block_status_t route_logits(const uint16_t *x, const void *router, block_dtype_t rdt, const RouteSizes &s,
                            const int *valid, void *ws, hipStream_t st)
{
    double *partial = static_cast<double *>(ws);
    const char *xc = reinterpret_cast<const char *>(x), *rc = static_cast<const char *>(router);
    const dim3 grid((unsigned)ceil_div(s.experts, kRouteTile), (unsigned)ceil_div(s.tokens, kRouteTile),
                    (unsigned)route_parts(s)),
        threads(kRouteWaves * 64);
    auto run = [&](auto kernel) {
        return launch(kernel, grid, threads, 0, st, xc, rc, partial, (int)s.tokens, (int)s.hidden, s.experts,
                      route_part(s), valid);
    };
    if (s.tokens <= kRouteFew)
        return rdt == BLOCK_FP32 ? run(route_logits_few_kernel<DT_F32>) : run(route_logits_few_kernel<DT_BF16>);
    return rdt == BLOCK_FP32 ? run(route_logits_kernel<DT_F32>) : run(route_logits_kernel<DT_BF16>);
}

block_status_t route(const uint16_t *x, const void *router, block_dtype_t rdt, int *ids, float *probs,
                     const RouteSizes &s, int top_k, int renormalize, const int *valid, void *ws, hipStream_t st)
{
    if (const block_status_t r = route_logits(x, router, rdt, s, valid, ws, st))
        return r;
    return launch(route_choose_kernel, dim3((unsigned)s.tokens), dim3((unsigned)round_up(s.experts, 64)), 0, st,
                  static_cast<const double *>(ws), ids, probs, (int)s.tokens, s.experts, (int)route_parts(s), top_k,
                  renormalize, valid);
}

struct ExpertSizes {
    int64_t tokens, hidden, inter;
    int experts, top_k;
};

block_status_t check_experts(const ExpertSizes &s, block_act_t act, float limit)
{
    if (s.tokens < 0 || s.hidden < 8 || s.inter < 8 || s.hidden > (1 << 16) || s.inter > (1 << 16) || s.experts < 1 ||
        s.experts > kMaxExperts || s.top_k < 1 || s.top_k > kMaxPairs || s.tokens > kMaxPairs ||
        s.tokens * s.top_k > kMaxPairs)
        return BLOCK_ERR_INVALID_ARG;
    if (act != BLOCK_ACT_SWIGLU && act != BLOCK_ACT_SQUARED_RELU)
        return BLOCK_ERR_INVALID_ARG;
    if (act == BLOCK_ACT_SWIGLU && !(limit > 0.0f))
        return BLOCK_ERR_INVALID_ARG;
    if (s.hidden % 8 || s.inter % 8)
        return BLOCK_ERR_ALIGNMENT;
    return BLOCK_OK;
}

// Workgroups that share the chosen experts of one block of output columns in the down product,
// or 0 for the form of a few pairs.
int down_shares(const ExpertSizes &s);

struct ExpertSpace {
    int64_t h, all;  // bytes: h, then the partial rows of y
};

ExpertSpace expert_space(const ExpertSizes &s)
{
    const int64_t h = round_up(s.tokens * s.top_k * s.inter * 4, 16), shares = down_shares(s);
    return {h, h + (shares > 1 ? shares * s.tokens * s.hidden * 4 : 0)};
}

// Parts the down product of one expert is cut into, so that a workgroup's waves all have
// work when few experts are reached.
int down_parts(const ExpertSizes &s)
{
    const int64_t pairs = s.tokens * s.top_k;
    const int64_t units = pairs < s.experts ? pairs : s.experts;
    int parts = 1;
    while (units * parts < 8 && pairs * parts * 2 <= kMaxPairs && parts * 4 * kLineK <= s.inter)
        parts *= 2;
    return parts;
}

int down_shares(const ExpertSizes &s)
{
    const int64_t pairs = s.tokens * s.top_k;
    if (s.tokens > kManyTokens || pairs < kManyPairs)
        return 0;
    const int64_t units = pairs < s.experts ? pairs : s.experts;
    int shares = 1;
    while (shares < 16 && shares * 2 <= units && ceil_div(s.hidden, kManyCols) * shares < kManyWaves)
        shares *= 2;
    return shares;
}

// Groups of tokens that share a read of an expert's weights: enough for one and a half times
// the tokens an expert has on average. An expert with more reads its weights again, but
// registers for more would cost waves in flight.
int token_groups(const ExpertSizes &s, int group)
{
    const int64_t some = ceil_div(3 * s.tokens * s.top_k, 2 * s.experts);
    const int64_t each = s.tokens < some ? s.tokens : some;
    return each <= group ? 1 : (each <= 2 * group ? 2 : 4);
}

template <int ACT>
block_status_t launch_up(const UpArgs &u, int groups, dim3 grid, hipStream_t st)
{
    const dim3 threads(kUpWaves * 64);
    if (u.partial)
        return launch(moe_up_kernel<ACT, 1, true>, grid, threads, 0, st, u);
    if (groups == 1)
        return launch(moe_up_kernel<ACT, 1, false>, grid, threads, 0, st, u);
    if (groups == 2)
        return launch(moe_up_kernel<ACT, 2, false>, grid, threads, 0, st, u);
    return launch(moe_up_kernel<ACT, 4, false>, grid, threads, 0, st, u);
}

template <int YDT, int G>
block_status_t launch_few(const DownArgs &d, dim3 grid, uint32_t lds, hipStream_t st)
{
    constexpr int W = kDownWaves<G>;
    // stages, ids, the waves' lists, the pairs' sums (at most kMaxPairs times their parts)
    static_assert(W * kStage<1, G, true> * 16 + kMaxPairs * 4 + W * kMaxPairs * 2 + kMaxPairs * 64 <= 160 * 1024,
                  "shared memory of a workgroup");
    return launch(moe_down_kernel<YDT, G>, grid, dim3(W * 64), lds, st, d);
}

template <int YDT>
block_status_t launch_down(const DownArgs &d, int groups, dim3 grid, uint32_t lds, hipStream_t st)
{
    if (groups == 1)
        return launch_few<YDT, 1>(d, grid, lds, st);
    if (groups == 2)
        return launch_few<YDT, 2>(d, grid, lds, st);
    return launch_few<YDT, 4>(d, grid, lds, st);
}

// Shared memory of a workgroup: each wave has a stage and a row of kManyCols sums a token, so
// more than 64 tokens leave room for four waves.
int many_waves(const ExpertSizes &s, int groups) { return groups == 4 || s.tokens > 64 ? 4 : 8; }

template <int YDT, int G, int W>
block_status_t launch_many(const DownArgs &d, dim3 grid, float *partial, hipStream_t st)
{
    // stages, the lists of pairs (18.1 KB), the sums
    constexpr int kStatic = (W * kStage<kManyTiles, 1, true> + (G > 1 ? 2 * G * kTerms : 1)) * 16 + 18 * 1024 + 128;
    constexpr int kSums = W * (W == 8 ? 64 : kManyTokens) * kManyCols * 4;
    static_assert(kStatic + kSums <= 160 * 1024, "shared memory of a workgroup");
    return launch(moe_down_many_kernel<YDT, G, W>, grid, dim3(W * 64), (uint32_t)(W * d.tokens * kManyCols * 4), st, d,
                  partial);
}

template <int YDT>
block_status_t launch_down_many(const DownArgs &d, int groups, int waves, int shares, dim3 grid, float *partial,
                                hipStream_t st)
{
    block_status_t r;
    if (groups == 4)
        r = launch_many<YDT, 4, 4>(d, grid, partial, st);
    else if (groups == 2)
        r = waves == 8 ? launch_many<YDT, 2, 8>(d, grid, partial, st) : launch_many<YDT, 2, 4>(d, grid, partial, st);
    else
        r = waves == 8 ? launch_many<YDT, 1, 8>(d, grid, partial, st) : launch_many<YDT, 1, 4>(d, grid, partial, st);
    if (r || shares == 1)
        return r;
    return launch(moe_combine_kernel<YDT>, dim3((unsigned)ceil_div((int64_t)d.tokens * d.hidden, 1024)), dim3(256), 0,
                  st, d, partial, shares);
}

// A choice of experts still to be made, in the up kernel.
struct Choice {
    const double *partial;
    int parts, renormalize;
    int *ids;
    float *probs;
};

block_status_t experts(const uint16_t *x, const uint16_t *w_up, const uint16_t *w_down, const int *ids,
                       const float *probs, const Choice *choice, const uint16_t *residual, void *y, block_dtype_t ydt,
                       const ExpertSizes &s, block_act_t act, float limit, const int *valid, void *ws, hipStream_t st)
{
    UpArgs u = {};
    if (choice) {
        u.partial = choice->partial, u.parts = choice->parts, u.renormalize = choice->renormalize;
        u.ids_out = choice->ids, u.probs_out = choice->probs;
    }
    u.x = x, u.w = w_up, u.ids = ids, u.probs = probs, u.h = static_cast<float *>(ws), u.valid = valid;
    u.tokens = (int)s.tokens, u.hidden = (int)s.hidden, u.inter = (int)s.inter, u.experts = s.experts;
    u.top_k = s.top_k, u.limit = limit;
    const int64_t pairs = s.tokens * s.top_k;
    u.by_pair = pairs < s.experts;
    const dim3 grid((unsigned)ceil_div(s.inter, 16), (unsigned)(u.by_pair ? pairs : s.experts));
    const int up_groups = token_groups(s, 16);
    if (const block_status_t r = act == BLOCK_ACT_SWIGLU ? launch_up<ACT_SWIGLU>(u, up_groups, grid, st)
                                                         : launch_up<ACT_SQUARED_RELU>(u, up_groups, grid, st))
        return r;
    DownArgs d = {};
    d.h = u.h, d.w = w_down, d.residual = residual, d.ids = ids, d.y = static_cast<char *>(y), d.valid = valid;
    d.tokens = u.tokens, d.hidden = u.hidden, d.inter = u.inter, d.experts = u.experts, d.top_k = u.top_k;
    const int groups = token_groups(s, 8), shares = down_shares(s);
    if (shares > 0) {
        const int waves = many_waves(s, groups);
        const dim3 tiles((unsigned)ceil_div(s.hidden, kManyCols * waves), (unsigned)shares);
        float *partial = reinterpret_cast<float *>(static_cast<char *>(ws) + expert_space(s).h);
        return ydt == BLOCK_FP32 ? launch_down_many<DT_F32>(d, groups, waves, shares, tiles, partial, st)
                                 : launch_down_many<DT_BF16>(d, groups, waves, shares, tiles, partial, st);
    }
    d.parts = down_parts(s);
    const uint32_t lds = (uint32_t)(pairs * d.parts * 64);
    const dim3 tiles((unsigned)ceil_div(s.hidden, 16));
    return ydt == BLOCK_FP32 ? launch_down<DT_F32>(d, groups, tiles, lds, st)
                             : launch_down<DT_BF16>(d, groups, tiles, lds, st);
}

bool good_choice(int top_k, int experts) { return top_k >= 1 && top_k <= experts && top_k <= 64; }

}  // namespace

extern "C" {

int64_t block_moe_route_workspace(int64_t tokens, int64_t hidden, int n_experts)
{
    const RouteSizes s = {tokens, hidden, n_experts};
    return good_route(s) ? route_bytes(s) : 0;
}

block_status_t block_moe_route(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype, int32_t *ids,
                               float *probs, int64_t tokens, int64_t hidden, int n_experts, int top_k, int renormalize,
                               const int32_t *valid_tokens, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream)
{
    const RouteSizes s = {tokens, hidden, n_experts};
    if (!good_route(s) || !good_choice(top_k, n_experts) ||
        (router_dtype != BLOCK_BF16 && router_dtype != BLOCK_FP32))
        return BLOCK_ERR_INVALID_ARG;
    if (hidden % 8)
        return BLOCK_ERR_ALIGNMENT;
    if (tokens == 0)
        return BLOCK_OK;
    const int64_t need = route_bytes(s), wsize = router_dtype == BLOCK_FP32 ? 4 : 2;
    if (!x || !router_weight || !ids || !probs || !workspace || workspace_bytes < need)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(router_weight, 16) || misaligned(ids, 4) || misaligned(probs, 4) ||
        misaligned(valid_tokens, 4) || misaligned(workspace, 16))
        return BLOCK_ERR_ALIGNMENT;
    if (any_overlap<3, 3>({{ids, tokens * top_k * 4}, {probs, tokens * top_k * 4}, {workspace, need}},
                          {{x, tokens * hidden * 2}, {router_weight, n_experts * hidden * wsize}, {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    return route(x, router_weight, router_dtype, ids, probs, s, top_k, renormalize, valid_tokens, workspace, stream);
}

block_status_t block_moe_route_gated(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype,
                                     const float *bias, int32_t *ids, float *probs, int64_t tokens, int64_t hidden,
                                     int n_experts, int top_k, block_scores_t scores, int groups, int top_groups,
                                     int group_top, int renormalize, float scale, const int32_t *valid_tokens,
                                     void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    const RouteSizes s = {tokens, hidden, n_experts};
    const GateRule rule = {top_k, (int)scores, groups, top_groups, group_top, renormalize, scale};
    if (!good_route(s) || !good_gate(rule, n_experts) || (router_dtype != BLOCK_BF16 && router_dtype != BLOCK_FP32))
        return BLOCK_ERR_INVALID_ARG;
    if (hidden % 8)
        return BLOCK_ERR_ALIGNMENT;
    if (tokens == 0)
        return BLOCK_OK;
    const int64_t need = route_bytes(s), wsize = router_dtype == BLOCK_FP32 ? 4 : 2;
    if (!x || !router_weight || !ids || !probs || !workspace || workspace_bytes < need)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(router_weight, 16) || misaligned(bias, 4) || misaligned(ids, 4) ||
        misaligned(probs, 4) || misaligned(valid_tokens, 4) || misaligned(workspace, 16))
        return BLOCK_ERR_ALIGNMENT;
    if (any_overlap<3, 4>({{ids, tokens * top_k * 4}, {probs, tokens * top_k * 4}, {workspace, need}},
                          {{x, tokens * hidden * 2},
                           {router_weight, n_experts * hidden * wsize},
                           {bias, n_experts * (int64_t)4},
                           {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    if (const block_status_t r = route_logits(x, router_weight, router_dtype, s, valid_tokens, workspace, stream))
        return r;
    const GateArgs a = {workspace, bias, ids, probs, valid_tokens, (int)tokens, n_experts, (int)route_parts(s), rule};
    return gate_of_parts(a, stream);
}

int64_t block_moe_experts_workspace(int64_t tokens, int64_t hidden, int64_t inter, int n_experts, int top_k)
{
    const ExpertSizes s = {tokens, hidden, inter, n_experts, top_k};
    return check_experts(s, BLOCK_ACT_SQUARED_RELU, 0.0f) == BLOCK_OK ? expert_space(s).all : 0;
}

block_status_t block_moe_experts(const uint16_t *x, const uint16_t *w_up, const uint16_t *w_down, const int32_t *ids,
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
    const int64_t need = expert_space(s).all;
    if (!x || !w_up || !w_down || !ids || !probs || !y || !workspace || workspace_bytes < need)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(w_up, 16) || misaligned(w_down, 16) || misaligned(residual, 16) ||
        misaligned(y, 16) || misaligned(ids, 4) || misaligned(probs, 4) || misaligned(valid_tokens, 4) ||
        misaligned(workspace, 16))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t n = tokens * hidden, ups = act == BLOCK_ACT_SWIGLU ? 2 * inter : inter;
    if (any_overlap<2, 7>({{y, n * (y_dtype == BLOCK_FP32 ? 4 : 2)}, {workspace, need}},
                          {{x, n * 2},
                           {w_up, n_experts * ups * hidden * 2},
                           {w_down, n_experts * inter * hidden * 2},
                           {ids, tokens * top_k * 4},
                           {probs, tokens * top_k * 4},
                           {residual, n * 2},
                           {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    return experts(x, w_up, w_down, ids, probs, nullptr, residual, y, y_dtype, s, act, limit, valid_tokens, workspace,
                   stream);
}

int64_t block_moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter, int n_experts, int top_k)
{
    return block_moe_route_workspace(tokens, hidden, n_experts) + block_moe_experts_workspace(tokens, hidden, inter, n_experts, top_k);
}

block_status_t block_moe_layer(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype,
                               const uint16_t *w_up, const uint16_t *w_down, const uint16_t *residual, void *y,
                               block_dtype_t y_dtype, int32_t *ids, float *probs, int64_t tokens, int64_t hidden,
                               int64_t inter, int n_experts, int top_k, int renormalize, block_act_t act, float limit,
                               const int32_t *valid_tokens, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream)
{
    const RouteSizes rs = {tokens, hidden, n_experts};
    const ExpertSizes s = {tokens, hidden, inter, n_experts, top_k};
    if (!good_route(rs) || !good_choice(top_k, n_experts) ||
        (router_dtype != BLOCK_BF16 && router_dtype != BLOCK_FP32) || (y_dtype != BLOCK_BF16 && y_dtype != BLOCK_FP32))
        return BLOCK_ERR_INVALID_ARG;
    if (const block_status_t r = check_experts(s, act, limit))
        return r;
    if (tokens == 0)
        return BLOCK_OK;
    const int64_t route_need = route_bytes(rs), need = route_need + expert_space(s).all;
    if (!x || !router_weight || !w_up || !w_down || !ids || !probs || !y || !workspace || workspace_bytes < need)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(router_weight, 16) || misaligned(w_up, 16) || misaligned(w_down, 16) ||
        misaligned(residual, 16) || misaligned(y, 16) || misaligned(ids, 4) || misaligned(probs, 4) ||
        misaligned(valid_tokens, 4) || misaligned(workspace, 16))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t n = tokens * hidden, ups = act == BLOCK_ACT_SWIGLU ? 2 * inter : inter;
    if (any_overlap<4, 6>({{y, n * (y_dtype == BLOCK_FP32 ? 4 : 2)},
                           {workspace, need},
                           {ids, tokens * top_k * 4},
                           {probs, tokens * top_k * 4}},
                          {{x, n * 2},
                           {w_up, n_experts * ups * hidden * 2},
                           {w_down, n_experts * inter * hidden * 2},
                           {router_weight, n_experts * hidden * (router_dtype == BLOCK_FP32 ? 4 : 2)},
                           {residual, n * 2},
                           {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    void *space = static_cast<char *>(workspace) + route_need;
    const int64_t pairs = tokens * top_k;
    if (tokens <= kChooseTokens && n_experts <= kChooseExperts &&
        ceil_div(inter, 16) * (pairs < n_experts ? pairs : n_experts) <= kChooseGroups) {
        if (const block_status_t r = route_logits(x, router_weight, router_dtype, rs, valid_tokens, workspace, stream))
            return r;
        const Choice c = {static_cast<const double *>(workspace), (int)route_parts(rs), renormalize, ids, probs};
        return experts(x, w_up, w_down, ids, probs, &c, residual, y, y_dtype, s, act, limit, valid_tokens, space, stream);
    }
    if (const block_status_t r = route(x, router_weight, router_dtype, ids, probs, rs, top_k, renormalize,
                                       valid_tokens, workspace, stream))
        return r;
    return experts(x, w_up, w_down, ids, probs, nullptr, residual, y, y_dtype, s, act, limit, valid_tokens, space,
                   stream);
}

}  // extern "C"
