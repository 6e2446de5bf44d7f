// The router and the expert products of a few tokens, for AMD Instinct MI355X (gfx950).
// C ABI declared in block/moe_block.h.
//
// For a few tokens the cost is reading each chosen expert's weights once. Two kernels:
//   up    one workgroup a (chosen expert, 16 columns of the activation): its waves split the
//         hidden axis, the activation and the probability are applied to the joined sums,
//         and h goes to the workspace as two bf16 terms.
//   down  one workgroup 16 columns of the output: its waves take the chosen experts in turn
//         and leave each (token, slot)'s 16 values in LDS; a token's values are then added in
//         slot order, so no atomics are needed and the bits never change.
// A workgroup finds its experts and their tokens in ids itself: at most 1024 entries.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "block_host.h"
#include "weight_stream.h"

namespace {

using namespace block;

constexpr int kMaxPairs = 1024;    // tokens * top_k
constexpr int kMaxExperts = 1024;
constexpr int kPass = 64;          // pairs of one expert that share a read of its weights

__device__ __forceinline__ int live_tokens(const int *valid, int tokens)
{
    if (!valid)
        return tokens;
    const int v = *valid;
    return v < 0 ? 0 : (v < tokens ? v : tokens);
}

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------
__device__ __forceinline__ double wave_sum64(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2)
        v += __shfl_xor(v, m);
    return v;
}

// logits[t][e]: one wave a (token, expert). Products of two bf16 (or a bf16 and an fp32) are
// exact in fp64 and the sums are fp64.
template <int RDT>
__global__ __launch_bounds__(256) void route_logits_kernel(const char *x, const char *router, double *logits,
                                                           int tokens, int hidden, int experts, const int *valid)
{
    const int64_t at = (int64_t)blockIdx.x * 4 + wave_in_block();
    const int t = (int)(at / experts), e = (int)(at % experts);
    if (t >= live_tokens(valid, tokens))
        return;
    const char *xr = x + (int64_t)t * hidden * 2, *wr = router + (int64_t)e * hidden * kSize<RDT>;
    double sum = 0.0;
    for (int j = lane_id() * 8; j < hidden; j += 512) {
        float a[8], b[8];
        widen8<DT_BF16>(load8<DT_BF16>(xr, j, hidden), a);
        widen8<RDT>(load8<RDT>(wr, j, hidden), b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fma((double)a[i], (double)b[i], sum);
    }
    sum = wave_sum64(sum);
    if (lane_id() == 0)
        logits[at] = sum;
}

// A double as an unsigned integer in the same order; +0 and -0 alike, NaN above all, and
// nothing at 0 (which marks an expert already chosen).
__device__ __forceinline__ uint64_t order_key(double v)
{
    if (v != v)
        return ~(uint64_t)0;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return b >> 63 ? ~b : b | (uint64_t)1 << 63;
}

// One wave a token; lane l holds experts l, l + 64, ... (PER of them). top_k times, the
// largest remaining key, the lowest index first.
template <int PER>
__global__ __launch_bounds__(64) void route_choose_kernel(const double *logits, int *ids, float *probs, int tokens,
                                                          int experts, int top_k, int renormalize, const int *valid)
{
    const int t = blockIdx.x, lane = lane_id();
    if (t >= live_tokens(valid, tokens))
        return;
    const double *row = logits + (int64_t)t * experts;
    double v[PER];
    uint64_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < experts ? row[e] : 0.0;
        key[i] = e < experts ? order_key(v[i]) : 0;
    }
    int chosen = 0;      // lane j keeps slot j
    double logit = 0.0, top = 0.0;
    for (int j = 0; j < top_k; ++j) {
        uint64_t best = 0;
        double value = 0.0;
        int e = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                value = v[i];
                e = lane + 64 * i;
            }
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const uint64_t b2 = __shfl_xor(best, m);
            const double v2 = __shfl_xor(value, m);
            const int e2 = __shfl_xor(e, m);
            if (b2 > best || (b2 == best && e2 < e)) {
                best = b2;
                value = v2;
                e = e2;
            }
        }
        if (lane == j) {
            chosen = e;
            logit = value;
        }
        if (j == 0)
            top = value;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == lane + 64 * i)
                key[i] = 0;
    }
    const float mine = lane < top_k ? expf((float)(logit - top)) : 0.0f;
    float sum = mine;
    if (!renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += lane + 64 * i < experts ? expf((float)(v[i] - top)) : 0.0f;
    }
    sum = wave_sum(sum);
    if (lane < top_k) {
        ids[(int64_t)t * top_k + lane] = chosen;
        probs[(int64_t)t * top_k + lane] = mine / sum;
    }
}

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------
// The pairs (token * top_k + slot) below `pairs` whose id is e, in increasing order, into
// list; returns their number. One wave, all lanes.
__device__ __forceinline__ int list_pairs(const int *ids, int pairs, int e, uint16_t *list)
{
    const int lane = lane_id();
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
        const bool is = p0 + lane < pairs && ids[p0 + lane] == e;
        const uint64_t m = __ballot(is);
        if (is)
            list[n + __popcll(m & (((uint64_t)1 << lane) - 1))] = (uint16_t)(p0 + lane);
        n += __popcll(m);
    }
    return n;
}

// h as a sum of two bf16: the first cut off after 8 bits, the second the rest rounded to 8,
// so h keeps 16 bits (one bf16 alone would cost about what the output's own rounding
// costs). An infinity or NaN is the first term alone.
__device__ __forceinline__ void split_bf16(float h, uint16_t &hi, uint16_t &lo)
{
    const unsigned b = __float_as_uint(h);
    if ((b & 0x7f800000u) == 0x7f800000u) {
        hi = (uint16_t)pack_bf16x2(h, h);
        lo = 0;
        return;
    }
    hi = (uint16_t)(b >> 16);
    const float rest = h - __uint_as_float(b & 0xffff0000u);
    lo = (uint16_t)pack_bf16x2(rest, rest);
}

// Where h[pair][i] is in the workspace: rows of inter, eight first terms and then their
// eight second terms in turn, so that both are one lane's neighbouring 16 bytes.
__device__ __forceinline__ int64_t h_at(int64_t pair, int inter, int i)
{
    return pair * 2 * inter + (i / 8) * 16 + i % 8;
}

struct UpArgs {
    const uint16_t *x, *w;
    const int *ids;
    const float *probs;
    uint16_t *h;
    const int *valid;
    int tokens, hidden, inter, experts, top_k, by_pair;
    float limit;
};

template <int ACT, int G>
__device__ __forceinline__ void up_pass(const UpArgs &a, int e, int i0, const uint16_t *list, int n, f32x4 *joined)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;  // gate and up, or the one product
    const int lane = lane_id(), wave = wave_in_block();
    const int k8 = lane / 16 * 8;
    const uint16_t *w[RT], *b[1][G];
    const int row = i0 + lane % 16 < a.inter ? i0 + lane % 16 : a.inter - 1;  // past the end: read again, not stored
#pragma unroll
    for (int r = 0; r < RT; ++r)
        w[r] = a.w + ((int64_t)e * RT * a.inter + (int64_t)r * a.inter + row) * a.hidden + k8;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 16 + lane % 16;
        b[0][g] = a.x + (int64_t)(list[s < n ? s : n - 1] / a.top_k) * a.hidden + k8;
    }
    f32x4 acc[RT][G];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < G; ++g)
            acc[r][g] = f32x4{0, 0, 0, 0};
    stream_products<DT_BF16, RT, G, 1>(acc, w, b, 1, a.hidden, wave * kStreamStep, 4 * kStreamStep);
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
            for (int q = 0; q < 4; ++q)
                z[r] += joined[((q * RT + r) * G + g) * 64 + lane][wave];
        }
        const int s = g * 16 + lane % 16;
        if (s < n && i < a.inter) {
            const int pair = list[s];
            const float v = (ACT == ACT_SWIGLU ? swiglu(z[0], z[RT - 1], a.limit) : squared_relu(z[0])) * a.probs[pair];
            uint16_t hi, lo;
            split_bf16(v, hi, lo);
            uint16_t *at = a.h + h_at(pair, a.inter, i);
            at[0] = hi;
            at[8] = lo;
        }
    }
    __syncthreads();
}

// blockIdx.y: a pair (by_pair: it stands for its expert if no earlier pair has the same), or
// an expert, whichever is fewer.
template <int ACT>
__global__ __launch_bounds__(256) void moe_up_kernel(UpArgs a)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;
    __shared__ f32x4 joined[4 * RT * (kPass / 16) * 64];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k;
    int e = blockIdx.y;
    if (a.by_pair) {
        if (e >= pairs)
            return;
        e = a.ids[e];
        if (e < 0 || e >= a.experts)
            return;
    }
    if (wave_in_block() == 0) {
        const int n = list_pairs(a.ids, pairs, e, list);
        if (lane_id() == 0)
            count = n;
    }
    __syncthreads();
    const int n = count;
    if (n == 0 || (a.by_pair && list[0] != (int)blockIdx.y))
        return;
    const int i0 = blockIdx.x * 16;
    for (int p = 0; p < n; p += kPass) {
        const int m = n - p < kPass ? n - p : kPass;
        if (m <= 16)
            up_pass<ACT, 1>(a, e, i0, list + p, m, joined);
        else if (m <= 32)
            up_pass<ACT, 2>(a, e, i0, list + p, m, joined);
        else
            up_pass<ACT, 4>(a, e, i0, list + p, m, joined);
    }
}

struct DownArgs {
    const uint16_t *h, *w, *residual;
    const int *ids;
    char *y;
    const int *valid;
    int tokens, hidden, inter, experts, top_k, parts;
};

template <int G>
__device__ __forceinline__ void down_pass(const DownArgs &a, const uint16_t *w, const uint16_t *list, int n, int part,
                                          float *sums)
{
    const int lane = lane_id(), k8 = lane / 16 * 8;
    const uint16_t *wr[1] = {w}, *b[2][G];
    f32x4 acc[1][G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 16 + lane % 16;
        b[0][g] = a.h + h_at(list[s < n ? s : n - 1], a.inter, k8);
        b[1][g] = b[0][g] + 8;
        acc[0][g] = f32x4{0, 0, 0, 0};
    }
    stream_products<DT_BF16, 1, G, 2>(acc, wr, b, 2, a.inter, part * kStreamStep, a.parts * kStreamStep);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 16 + lane % 16;
        if (s < n)
            *reinterpret_cast<f32x4 *>(sums + (list[s] * a.parts + part) * 16 + lane / 16 * 4) = acc[0][g];
    }
}

template <int YDT>
__global__ __launch_bounds__(256) void moe_down_kernel(DownArgs a)
{
    extern __shared__ f32x4 dynamic[];  // [pairs][parts][16] fp32
    __shared__ int ids[kMaxPairs];
    __shared__ int first[kMaxExperts];
    __shared__ uint16_t units[kMaxPairs];
    __shared__ uint16_t lists[4][kMaxPairs];
    __shared__ int unit_count;
    float *sums = reinterpret_cast<float *>(dynamic);
    const int lane = lane_id(), wave = wave_in_block(), tid = threadIdx.x;
    const int live = live_tokens(a.valid, a.tokens), pairs = live * a.top_k;
    for (int e = tid; e < a.experts; e += 256)
        first[e] = kMaxPairs;
    __syncthreads();
    for (int p = tid; p < pairs; p += 256) {
        const int e = a.ids[p];
        const bool ok = e >= 0 && e < a.experts;
        ids[p] = ok ? e : -1;
        if (ok)
            atomicMin(&first[e], p);
    }
    __syncthreads();
    if (wave == 0) {  // the pairs that are their expert's first
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const bool is = p < pairs && ids[p] >= 0 && first[ids[p]] == p;
            const uint64_t m = __ballot(is);
            if (is)
                units[n + __popcll(m & (((uint64_t)1 << lane) - 1))] = (uint16_t)p;
            n += __popcll(m);
        }
        if (lane == 0)
            unit_count = n;
    }
    __syncthreads();
    const int n_units = unit_count;
    const int c0 = blockIdx.x * 16;
    const int row = c0 + lane % 16 < a.hidden ? c0 + lane % 16 : a.hidden - 1;
    uint16_t *list = lists[wave];
    for (int u = wave; u < n_units * a.parts; u += 4) {
        const int e = __builtin_amdgcn_readfirstlane(ids[units[u / a.parts]]), part = u % a.parts;
        const int n = list_pairs(ids, pairs, e, list);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const uint16_t *w = a.w + ((int64_t)e * a.hidden + row) * a.inter + lane / 16 * 8;
        for (int p = 0; p < n; p += kPass) {
            const int m = n - p < kPass ? n - p : kPass;
            if (m <= 16)
                down_pass<1>(a, w, list + p, m, part, sums);
            else if (m <= 32)
                down_pass<2>(a, w, list + p, m, part, sums);
            else
                down_pass<4>(a, w, list + p, m, part, sums);
        }
    }
    __syncthreads();
    for (int i = tid; i < live * 16; i += 256) {
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
        const int64_t at = (int64_t)t * a.hidden + c;
        if (a.residual)
            v += load1<DT_BF16>(a.residual, at);
        store1<YDT>(a.y, at, v);
    }
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
    return s.tokens >= 0 && s.tokens <= (1 << 20) && s.hidden >= 8 && s.hidden <= (1 << 20) && s.experts >= 1 &&
           s.experts <= kMaxExperts && s.tokens * s.experts <= (1 << 25);
}

int64_t route_bytes(const RouteSizes &s) { return round_up(s.tokens * s.experts * 8, 16); }

template <int PER>
block_status_t choose(const double *logits, int *ids, float *probs, const RouteSizes &s, int top_k, int renormalize,
                      const int *valid, hipStream_t st)
{
    return launch(route_choose_kernel<PER>, dim3((unsigned)s.tokens), dim3(64), 0, st, logits, ids, probs,
                  (int)s.tokens, s.experts, top_k, renormalize, valid);
}

block_status_t route(const uint16_t *x, const void *router, block_dtype_t rdt, int *ids, float *probs,
                     const RouteSizes &s, int top_k, int renormalize, const int *valid, void *ws, hipStream_t st)
{
    double *logits = static_cast<double *>(ws);
    const char *xc = reinterpret_cast<const char *>(x), *rc = static_cast<const char *>(router);
    const dim3 grid((unsigned)ceil_div(s.tokens * s.experts, 4));
    block_status_t r;
    if (rdt == BLOCK_FP32)
        r = launch(route_logits_kernel<DT_F32>, grid, dim3(256), 0, st, xc, rc, logits, (int)s.tokens, (int)s.hidden,
                   s.experts, valid);
    else
        r = launch(route_logits_kernel<DT_BF16>, grid, dim3(256), 0, st, xc, rc, logits, (int)s.tokens, (int)s.hidden,
                   s.experts, valid);
    if (r)
        return r;
    if (s.experts <= 64)
        return choose<1>(logits, ids, probs, s, top_k, renormalize, valid, st);
    if (s.experts <= 256)
        return choose<4>(logits, ids, probs, s, top_k, renormalize, valid, st);
    return choose<16>(logits, ids, probs, s, top_k, renormalize, valid, st);
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

int64_t expert_bytes(int64_t tokens, int top_k, int64_t inter) { return tokens * top_k * inter * 4; }

// Parts the down product of one expert is cut into, so that a workgroup's four waves all
// have work when few experts are reached.
int down_parts(const ExpertSizes &s)
{
    const int64_t pairs = s.tokens * s.top_k;
    const int64_t units = pairs < s.experts ? pairs : s.experts;
    int parts = 1;
    while (units * parts < 8 && pairs * parts * 2 <= kMaxPairs && parts * 2 * kStreamStep <= s.inter)
        parts *= 2;
    return parts;
}

block_status_t experts(const uint16_t *x, const uint16_t *w_up, const uint16_t *w_down, const int *ids,
                       const float *probs, const uint16_t *residual, void *y, block_dtype_t ydt, const ExpertSizes &s,
                       block_act_t act, float limit, const int *valid, void *ws, hipStream_t st)
{
    UpArgs u = {};
    u.x = x, u.w = w_up, u.ids = ids, u.probs = probs, u.h = static_cast<uint16_t *>(ws), u.valid = valid;
    u.tokens = (int)s.tokens, u.hidden = (int)s.hidden, u.inter = (int)s.inter, u.experts = s.experts;
    u.top_k = s.top_k, u.limit = limit;
    const int64_t pairs = s.tokens * s.top_k;
    u.by_pair = pairs < s.experts;
    const dim3 grid((unsigned)ceil_div(s.inter, 16), (unsigned)(u.by_pair ? pairs : s.experts));
    block_status_t r;
    if (act == BLOCK_ACT_SWIGLU)
        r = launch(moe_up_kernel<ACT_SWIGLU>, grid, dim3(256), 0, st, u);
    else
        r = launch(moe_up_kernel<ACT_SQUARED_RELU>, grid, dim3(256), 0, st, u);
    if (r)
        return r;
    DownArgs d = {};
    d.h = u.h, d.w = w_down, d.residual = residual, d.ids = ids, d.y = static_cast<char *>(y), d.valid = valid;
    d.tokens = u.tokens, d.hidden = u.hidden, d.inter = u.inter, d.experts = u.experts, d.top_k = u.top_k;
    d.parts = down_parts(s);
    const uint32_t lds = (uint32_t)(pairs * d.parts * 64);
    const dim3 tiles((unsigned)ceil_div(s.hidden, 16));
    if (ydt == BLOCK_FP32)
        return launch(moe_down_kernel<DT_F32>, tiles, dim3(256), lds, st, d);
    return launch(moe_down_kernel<DT_BF16>, tiles, dim3(256), lds, st, d);
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

int64_t block_moe_experts_workspace(int64_t tokens, int top_k, int64_t inter)
{
    if (tokens < 0 || tokens > kMaxPairs || top_k < 1 || top_k > kMaxPairs || inter < 0 || inter > (1 << 16))
        return 0;
    return expert_bytes(tokens, top_k, inter);
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
    const int64_t need = expert_bytes(tokens, top_k, inter);
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
    return experts(x, w_up, w_down, ids, probs, residual, y, y_dtype, s, act, limit, valid_tokens, workspace, stream);
}

int64_t block_moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter, int n_experts, int top_k)
{
    return block_moe_route_workspace(tokens, hidden, n_experts) + block_moe_experts_workspace(tokens, top_k, inter);
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
    const int64_t route_need = route_bytes(rs), need = route_need + expert_bytes(tokens, top_k, inter);
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
    if (const block_status_t r = route(x, router_weight, router_dtype, ids, probs, rs, top_k, renormalize,
                                       valid_tokens, workspace, stream))
        return r;
    return experts(x, w_up, w_down, ids, probs, residual, y, y_dtype, s, act, limit, valid_tokens,
                   static_cast<char *>(workspace) + route_need, stream);
}

}  // extern "C"
