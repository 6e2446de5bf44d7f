// The gate: scores of a token's experts, the choice among them and their weights, and its
// gradient, for AMD Instinct MI355X (gfx950). C ABI declared in block/moe_block.h.
//
// A token's experts lie spread over L lanes of a wave, V a lane (expert i L + l in lane l), so a
// wave holds 64 / L tokens. Scores are formed in fp64, as the choice is made between neighbouring
// values; what has to be seen by other lanes goes through the wave's own shared memory, and no
// kernel here has a barrier.
//
// Few tokens of up to 256 experts take 2.8 to 5.7 us: a launch, a chain of exchanges for groups (1.3)
// and one for each slot (0.15); of 512 experts up to 10.4. Many are bound by vector instructions, not
// by memory: with 256 experts in 8 groups of which 4 are kept, top 8, a wave of two tokens issues 1400
// of them, and 6720 tokens (13.8 us for 6.9 MB) leave some of the 1024 SIMDs four waves and others
// three. (Sixteen lanes a token 13.9 us, a wave each 14.6; the same choice in fp32 where its gaps
// certify it 1196 instructions and 13.8; the winner's index found in the scalar unit 14.0.)
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "gate.h"
#include "gate_math.h"
#include "route_device.h"

namespace {

using namespace block;

constexpr int kWavesHere = 4;
constexpr int SRC_PARTS = 3;  // beside the DT_ codes: fp64 partial sums

// What order_key was made of.
__device__ __forceinline__ double of_key(uint64_t k)
{
    return __builtin_bit_cast(double, k >> 63 ? k & ~((uint64_t)1 << 63) : ~k);
}

template <typename T>
__device__ __forceinline__ T larger(T a, T b)
{
    return a > b ? a : b;
}

template <int kCtrl>
__device__ __forceinline__ unsigned dpp32(unsigned v)
{
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
}

// What the lane in the other row of 16 of each pair of rows holds, or in the other half of the wave.
// (One instruction swaps the odd rows of one register with the even rows of another.)
template <int kLanes>
__device__ __forceinline__ unsigned other_row(unsigned v)
{
    const auto s = kLanes == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (lane_id() & kLanes) ? s[0] : s[1];
}

// Over the L = 16, 32 or 64 lanes of a token, the same in each of them.
template <int L>
__device__ __forceinline__ unsigned lanes_max(unsigned v)
{
    v = larger(v, dpp32<0xB1>(v));
    v = larger(v, dpp32<0x4E>(v));
    v = larger(v, dpp32<0x141>(v));
    v = larger(v, dpp32<0x140>(v));
    if constexpr (L >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = larger(s[0], s[1]);
    }
    if constexpr (L == 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = larger(s[0], s[1]);
    }
    return v;
}

// The largest key: its upper half, then the lower halves of those that share it.
template <int L>
__device__ __forceinline__ uint64_t lanes_max(uint64_t v)
{
    const unsigned hi = lanes_max<L>((unsigned)(v >> 32));
    return (uint64_t)hi << 32 | lanes_max<L>((unsigned)(v >> 32) == hi ? (unsigned)v : 0u);
}

template <int kLanes>
__device__ __forceinline__ double other_row(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t hi = other_row<kLanes>((unsigned)(b >> 32)), lo = other_row<kLanes>((unsigned)b);
    return __builtin_bit_cast(double, hi << 32 | lo);
}

template <int L>
__device__ __forceinline__ double lanes_sum(double v)
{
    v += dpp64<0xB1>(v);
    v += dpp64<0x4E>(v);
    v += dpp64<0x141>(v);
    v += dpp64<0x140>(v);
    if constexpr (L >= 32)
        v += other_row<16>(v);
    if constexpr (L == 64)
        v += other_row<32>(v);
    return v;
}

// The wave's accesses to its shared memory stay in order; this keeps the compiler from moving
// them across.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// 1 / d to a step or so, for d that neither overflows nor underflows.
__device__ __forceinline__ double reciprocal(double d)
{
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
    return __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
}

__device__ __forceinline__ double sigmoid(double v)
{
    const double e = exp_below(-__builtin_fabs(v)), q = reciprocal(1.0 + e);
    return v < 0.0 ? e * q : q;
}

// The logits at row + at[i]. Loads go out together, of partial sums those of several parts (a
// logit after the other, one token's 256 took 1.2 us more); the parts are added in
// order.
template <int SRC, int N>
__device__ __forceinline__ void logits_at(const GateArgs &a, int64_t row, const int (&at)[N], double (&v)[N])
{
    if constexpr (SRC == SRC_PARTS) {
        constexpr int kTogether = N > 8 ? 2 : (N > 4 ? 4 : 8);
        const double *from = static_cast<const double *>(a.logits) + row;
        const int64_t part = (int64_t)a.tokens * a.experts;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = 0.0;
        for (int s = 0; s < a.parts; s += kTogether) {
            double p[kTogether][N];
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    p[j][i] = from[(s + j < a.parts ? s + j : 0) * part + at[i]];
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] += s + j < a.parts ? p[j][i] : 0.0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = (double)load1<SRC>(a.logits, row + at[i]);
    }
}

// What a softmax takes from all of its logits: the largest, and one over the sum of e^(v - largest).
struct Softmax {
    double largest, share;
    __device__ __forceinline__ double operator()(double v) const
    {
        return largest == -INFINITY ? 0.0 : exp_below(v - largest) * share;
    }
};

// e = e^(v - largest) over a token's lanes, all zeros where every logit is -inf. top: of the order keys.
template <int L, int V>
__device__ __forceinline__ Softmax softmax_parts(const double (&v)[V], uint64_t top, double (&e)[V])
{
    const double m = of_key(lanes_max<L>(top));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        e[i] = m == -INFINITY ? 0.0 : exp_below(v[i] - m);
        sum += e[i];
    }
    sum = lanes_sum<L>(sum);
    return {m, sum == 0.0 ? 0.0 : reciprocal(sum)};  // a sum is 0, or at least 1
}

// s = softmax(v) over a token's lanes.
template <int L, int V>
__device__ __forceinline__ void softmax(const double (&v)[V], double (&s)[V])
{
    uint64_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        top = larger(top, order_key(v[i]));
    const double q = softmax_parts<L, V>(v, top, s).share;
#pragma unroll
    for (int i = 0; i < V; ++i)
        s[i] *= q;
}

// A token's room in its wave's shared memory.
struct Room {
    uint64_t *table;  // an entry an expert
    uint64_t *worth;  // an entry a group
};

// Lanes of a token that look through one group together: a power of two.
template <int L>
__device__ __forceinline__ int lanes_a_group(int groups)
{
    return groups >= L ? 1 : L >> (32 - __builtin_clz(groups - 1));
}

// The choice, in fp64: lane l gets the experts of slots l, L + l, ... and their scores. v: the
// logits, -inf past the last expert.
//
// Without a bias (BIASED false) experts are ranked by their logits: the scores have the same order, but
// run out of exponents (the softmax's) or come to 1 (the sigmoid's) and then tie. Scores are formed for
// the chosen ones alone, and for the worth of a group that is a sum of two.
template <int L, int V, int Q, bool BIASED>
__device__ __forceinline__ void choose(const GateRule &r, int experts, int l, const double (&v)[V], const float (&bias)[V],
                                       const Room &room, int (&id)[Q], double (&p)[Q])
{
    constexpr int T = 64 / L;
    double s[V];
    uint64_t key[V];  // of the rank; 0, below every number's, for what cannot be chosen
    Softmax all = {0.0, 0.0};
    const auto score_of = [&](double x) __attribute__((always_inline)) {
        return r.scores == BLOCK_SCORES_SIGMOID ? sigmoid(x) : all(x);
    };
    if constexpr (BIASED) {
        if (r.scores == BLOCK_SCORES_SIGMOID) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] = sigmoid(v[i]);
        } else {
            softmax<L, V>(v, s);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = i * L + l < experts ? order_key(v[i] == -INFINITY ? v[i] : s[i] + (double)bias[i]) : 0;
    } else {
        uint64_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = order_key(v[i]);
            top = larger(top, key[i]);
            key[i] = i * L + l < experts ? key[i] : 0;
        }
        if (r.scores != BLOCK_SCORES_SIGMOID) {
            all = softmax_parts<L, V>(v, top, s);
            if (__any(all.share != all.share)) {  // a NaN, or an infinity: all scores are NaN but of masked experts
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = all.share != all.share && key[i] > order_key(-INFINITY) ? ~(uint64_t)0 : key[i];
            }
        }
    }
    if (r.groups > 1) {
        const int size = experts / r.groups;
        const unsigned inverse = ((1u << 20) + size - 1) / size;  // e / size = e inverse / 2^20 for e, size <= 1024
#pragma unroll
        for (int i = 0; i < V; ++i)
            room.table[i * L + l] = key[i];
        wave_fence();
        const int each = lanes_a_group<L>(r.groups);
        for (int g0 = 0; g0 < r.groups; g0 += L / each) {
            const int g = g0 + l / each;
            uint64_t first_key = 0, second_key = 0;
            const int from = g < r.groups ? g * size : 0;
            constexpr int kTogether = 4;  // loads that go out together
            for (int m0 = l % each; m0 < size; m0 += kTogether * each) {
                uint64_t k[kTogether];
#pragma unroll
                for (int i = 0; i < kTogether; ++i) {
                    const int m = m0 + i * each;
                    k[i] = room.table[from + (m < size ? m : 0)];
                    k[i] = m < size ? k[i] : 0;
                }
#pragma unroll
                for (int i = 0; i < kTogether; ++i) {
                    second_key = larger(second_key, k[i] < first_key ? k[i] : first_key);
                    first_key = larger(first_key, k[i]);
                }
            }
            for (int d = 1; d < each; d *= 2) {
                const uint64_t f = __shfl_xor(first_key, d), q = __shfl_xor(second_key, d);
                second_key = larger(larger(second_key, q), f < first_key ? f : first_key);
                first_key = larger(first_key, f);
            }
            double w = of_key(first_key);
            if (r.group_top == 2) {
                double other = of_key(second_key);
                if (!BIASED) {
                    w = w == -INFINITY ? w : score_of(w);
                    other = other == -INFINITY ? other : score_of(other);
                }
                w += other;
            }
            if (g < r.groups && l % each == 0)
                room.worth[g] = order_key(w);
        }
        wave_fence();
        uint64_t kept = 0;  // a bit a group
        for (int g0 = 0; g0 < r.groups; g0 += L) {
            const int g = g0 + l < r.groups ? g0 + l : 0;
            const uint64_t own = room.worth[g];
            int before = 0;
#pragma unroll 8
            for (int o = 0; o < r.groups; ++o)
                before += room.worth[o] > own || (room.worth[o] == own && o < g);
            const uint64_t lanes = __ballot(g0 + l < r.groups && before < r.top_groups) >> (lane_id() & (64 - L));
            kept |= (L == 64 ? lanes : lanes & (((uint64_t)1 << (L & 63)) - 1)) << g0;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned e = i * L + l, g = e * inverse >> 20;
            const unsigned word = g < 32 ? (unsigned)kept : (unsigned)(kept >> 32);
            key[i] = word >> g % 32 & 1 ? key[i] : 0;  // experts past the last one have 0 already
        }
        wave_fence();
    }
    if (!BIASED && r.groups == 1) {  // where the chosen ones' logits are found
#pragma unroll
        for (int i = 0; i < V; ++i)
            room.table[i * L + l] = key[i];
    }
    // The upper halves of the keys decide where the largest is there once for each token of the wave;
    // otherwise the lower halves of those that share it, then the index. (The comparisons serve twice,
    // and are counted in the scalar unit: 13,440 x 256 20.5 -> 19.7 us.)
    unsigned hi[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        hi[i] = (unsigned)(key[i] >> 32);
#pragma unroll
    for (int q = 0; q < Q; ++q)
        id[q] = 0;
    for (int j = 0; j < r.top_k; ++j) {
        unsigned best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            best = larger(best, hi[i]);
        best = lanes_max<L>(best);
        unsigned from_end = 0;  // the lowest expert of the best, counted from the end
        int count = 0;  // as each token has one at least, one each if there are T
        bool is[V];
#pragma unroll
        for (int i = V - 1; i >= 0; --i) {
            is[i] = hi[i] == best;
            from_end = is[i] ? (unsigned)(kGateExperts - (i * L + l)) : from_end;
            count += __popcll(__ballot(is[i]));
        }
        int e;
        if (count != T) {
            unsigned low = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                low = larger(low, is[i] ? (unsigned)key[i] : 0u);
            low = lanes_max<L>(low);
            from_end = 0;
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                from_end = is[i] && (unsigned)key[i] == low ? (unsigned)(kGateExperts - (i * L + l)) : from_end;
            e = kGateExperts - (int)lanes_max<L>(from_end);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hi[i] = i * L + l == e ? 0u : hi[i];
        } else {
            e = kGateExperts - (int)lanes_max<L>(from_end);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hi[i] = is[i] ? 0u : hi[i];
        }
#pragma unroll
        for (int q = 0; q < Q; ++q)
            id[q] = q * L + l == j ? e : id[q];
    }
    wave_fence();
    double *score = reinterpret_cast<double *>(room.table);
    if constexpr (BIASED) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            score[i * L + l] = s[i];
        wave_fence();
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        p[q] = 0.0;
        if (q * L < r.top_k) {
            const double x = BIASED ? score[id[q]] : score_of(of_key(room.table[id[q]]));
            p[q] = q * L + l < r.top_k ? x : 0.0;
        }
    }
}

// Whether a sum of chosen scores is so small that some of them have lost digits or are gone, and their
// shares are better had from their logits. (Sigmoid scores that are all 0 have shares of 0.)
__device__ __forceinline__ bool near_the_end(int scores, double sum)
{
    return sum < 0x1p-840 && (scores == BLOCK_SCORES_SOFTMAX || sum > 0.0);
}

template <int SRC, int L, int V, bool BIASED>
__global__ __launch_bounds__(kWavesHere * 64) void gate_kernel(GateArgs a)
{
    constexpr int T = 64 / L;
    __shared__ uint64_t tables[kWavesHere][T][L * V];
    __shared__ uint64_t worths[kWavesHere][T][kGateGroups];
    const GateRule r = a.rule;
    const int lane = lane_id(), wave = wave_in_block(), l = lane % L, tl = lane / L;
    const int first = ((int)blockIdx.x * kWavesHere + wave) * T, live = live_tokens(a.valid, a.tokens);
    if (first >= live)
        return;
    const bool mine = first + tl < live;
    const int t = mine ? first + tl : first;  // past the last token: the first one again, not stored
    uint64_t *table = tables[wave][tl], *worth = worths[wave][tl];
    const int64_t row = (int64_t)t * a.experts;

    // Loads without branches, past the last expert of the first one again: all of them are on their way
    // together, and what follows is no chain of branches either. (With a condition around each
    // load, 6720 x 256 took 14.7 us.)
    int at[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        at[i] = i * L + l < a.experts ? i * L + l : 0;
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        bias[i] = BIASED ? a.bias[at[i]] : 0.0f;
    double v[V];
    logits_at<SRC, V>(a, row, at, v);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = i * L + l < a.experts ? v[i] : -INFINITY;
    constexpr int Q = kGateSlots / L;
    int id[Q];  // lane l has slots l, L + l, ...
    double p[Q];
    const Room room = {table, worth};
    choose<L, V, Q, BIASED>(r, a.experts, l, v, bias, room, id, p);
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
        sum += p[q];
    if (r.renormalize) {
        sum = lanes_sum<L>(sum);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            p[q] = sum == 0.0 ? 0.0 : p[q] / sum;
        // Chosen for their bias, hundreds below the largest logit, or sigmoid scores that are e^logit: from
        // the chosen logits alone, as in the gradient, where the scores run out of exponents (fp32
        // weights reach down to 2^-149).
        if (__any(near_the_end(r.scores, sum))) {
            double x[Q], own[Q];
            logits_at<SRC, Q>(a, row, id, x);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                x[q] = q * L + l < r.top_k ? x[q] : -INFINITY;
            softmax<L, Q>(x, own);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                p[q] = near_the_end(r.scores, sum) ? own[q] : p[q];
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = q * L + l;
        if (mine && j < r.top_k) {
            a.ids[(int64_t)t * r.top_k + j] = id[q];
            a.probs[(int64_t)t * r.top_k + j] = (float)(p[q] * (double)r.scale);
        }
    }
}

// v as fp32, but so that its rounding to DT is v's own. fp32's nearest number to v may be the middle
// between two of DT, on whose one side v lies. For bf16 that is seen in its bits, once in 2^16 values,
// and a step to that side will do; for fp16, whose subnormals have other middles, v is cut off to fp32 and
// its last bit set where anything was lost. (bf16 by cutting off too: 50,000 x 256, softmax of all
// 30.3 -> 32.1 us; the nearest fp32 of fp16's conversion from fp64 took 40.0, this takes 32.4.)
template <int DT, int V>
__device__ __forceinline__ void round_once(const double (&v)[V], float (&f)[V])
{
    bool middle = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f[i] = (float)v[i];
        middle |= DT == DT_BF16 && (uint16_t)__float_as_uint(f[i]) == 0x8000;
    }
    if (DT == DT_F32 || (DT == DT_BF16 && !__any(middle)))
        return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t bits = __float_as_uint(f[i]);
        const double d = (double)f[i];
        const bool lost = d != v[i], past = __builtin_fabs(d) > __builtin_fabs(v[i]);
        if (DT == DT_F16)
            f[i] = __uint_as_float(lost ? (bits - (past ? 1 : 0)) | 1 : bits);
        else if (lost && (uint16_t)bits == 0x8000)
            f[i] = __uint_as_float(past ? bits - 1 : bits + 1);
    }
}

struct GateGradArgs {
    const void *logits;
    const int *ids;
    const float *grad_probs;
    void *grad_logits;
    const int *valid;
    int tokens, experts, top_k, scores, renormalize;
    float scale;
};

// Gradient of the logits. With g_j = scale grad_probs_j and the chosen scores s_j:
//     renormalised: p_j = s_j / sum s, v_j = p_j (g_j - sum g p), otherwise v_j = g_j s_j;
//     sigmoid: v_j (1 - s_j) goes to expert ids_j. softmax: v_j does, and without
//     renormalisation (DENSE) every expert loses s sum v.
// Only DENSE reads logits that were not chosen. The gradient is a stream of stores: 6720 x 256 fp32
// 6.2 us for 6.9 MB, of which a launch and the chain ids, logits, stores take most.
template <int DT, int L, int V, bool DENSE>
__global__ __launch_bounds__(kWavesHere * 64) void gate_grad_kernel(GateGradArgs a)
{
    constexpr int T = 64 / L, Q = kGateSlots / L;
    __shared__ double tables[kWavesHere][T][L * V];
    __shared__ double values[kWavesHere][T][kGateSlots];
    __shared__ int slots[kWavesHere][T][kGateSlots];
    const int lane = lane_id(), wave = wave_in_block(), l = lane % L, tl = lane / L;
    const int first = ((int)blockIdx.x * kWavesHere + wave) * T, live = live_tokens(a.valid, a.tokens);
    if (first >= live)
        return;
    const bool mine = first + tl < live;
    const int t = mine ? first + tl : first;
    double *table = tables[wave][tl], *value = values[wave][tl];
    int *slot = slots[wave][tl];
    const int64_t row = (int64_t)t * a.experts;

    double s[V];
    if constexpr (DENSE) {
        double v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = (double)load1<DT>(a.logits, row + (i * L + l < a.experts ? i * L + l : 0));
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = i * L + l < a.experts ? v[i] : -INFINITY;
        softmax<L, V>(v, s);
#pragma unroll
        for (int i = 0; i < V; ++i)
            table[i * L + l] = s[i];
        wave_fence();
    }
    int id[Q];
    double x[Q], g[Q];  // the slot's logit (DENSE: score), its gradient
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = q * L + l, at = j < a.top_k ? j : 0;
        const int e = a.ids[(int64_t)t * a.top_k + at];
        g[q] = (double)a.scale * (double)a.grad_probs[(int64_t)t * a.top_k + at];
        id[q] = j < a.top_k && e >= 0 && e < a.experts ? e : -1;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = id[q] < 0 ? 0 : id[q];
        x[q] = DENSE ? table[e] : (double)load1<DT>(a.logits, row + e);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        x[q] = id[q] < 0 ? -INFINITY : x[q];
        g[q] = id[q] < 0 ? 0.0 : g[q];
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i)
        table[i * L + l] = 0.0;
    double out[Q], dot = 0.0;
    if constexpr (DENSE) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            out[q] = id[q] < 0 ? 0.0 : g[q] * x[q];
            dot += out[q];
        }
        dot = lanes_sum<L>(dot);
    } else {
        double p[Q];
        if (a.scores == BLOCK_SCORES_SIGMOID) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                p[q] = q * L < a.top_k ? sigmoid(x[q]) : 0.0;
        } else {
            softmax<L, Q>(x, p);
        }
        if (a.renormalize) {
            double sum = 0.0;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                sum += p[q];
            sum = lanes_sum<L>(sum);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                p[q] = sum == 0.0 ? 0.0 : p[q] / sum;
            if (a.scores == BLOCK_SCORES_SIGMOID && __any(near_the_end(a.scores, sum))) {
                double own[Q];
                softmax<L, Q>(x, own);
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    p[q] = near_the_end(a.scores, sum) ? own[q] : p[q];
            }
#pragma unroll
            for (int q = 0; q < Q; ++q)
                dot += id[q] < 0 ? 0.0 : g[q] * p[q];
            dot = lanes_sum<L>(dot);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            out[q] = p[q] * (g[q] - dot);
            if (a.scores == BLOCK_SCORES_SIGMOID && q * L < a.top_k)
                out[q] *= sigmoid(-x[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        slot[q * L + l] = id[q];
        value[q * L + l] = out[q];
    }
    wave_fence();
    // a lane adds to its own experts alone, in the order of the slots, so that the same id twice
    // is neither a race nor a choice of order
    for (int j = 0; j < a.top_k; ++j) {
        const int e = slot[j];
        if (e >= 0 && e % L == l)
            table[e] += value[j];
    }
    wave_fence();
    double grad[V];
    float once[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        grad[i] = table[i * L + l] - (DENSE ? s[i] * dot : 0.0);
    round_once<DT, V>(grad, once);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * L + l;
        if (mine && e < a.experts)
            store1<DT>(a.grad_logits, row + e, once[i]);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Up to so many tokens take a wave each, more share one by two or, with up to 64 experts, by four: a
// wave of its own has the shorter way to the answer, shared ones spend fewer instructions a
// token. (us, own and shared, softmax, top 8: 1024 tokens of 64 experts 3.8 and 4.7, of 256 4.9 and 6.1;
// 2048 tokens 4.1 and 4.8, 5.5 and 6.2; 4096 tokens 5.6 and 4.8, 7.5 and 6.9. The gradient's, of every logit:
// 3.2 and 3.7, 3.9 and 4.5; 3.5 and 3.7, 4.5 and 4.7; 4.2 and 3.8, 5.8 and 5.6.)
constexpr int kFewTokens = 2048;

unsigned groups_of(int64_t tokens, int lanes) { return (unsigned)ceil_div(tokens, kWavesHere * (64 / lanes)); }

template <int SRC, bool BIASED>
block_status_t run_gate(const GateArgs &a, hipStream_t st)
{
    const dim3 threads(kWavesHere * 64);
    const unsigned few = groups_of(a.tokens, 64);
    if (a.experts <= 64)
        return a.tokens <= kFewTokens
                   ? launch(gate_kernel<SRC, 64, 1, BIASED>, dim3(few), threads, 0, st, a)
                   : launch(gate_kernel<SRC, 16, 4, BIASED>, dim3(groups_of(a.tokens, 16)), threads, 0, st, a);
    if (a.experts <= 256)
        return a.tokens <= kFewTokens
                   ? launch(gate_kernel<SRC, 64, 4, BIASED>, dim3(few), threads, 0, st, a)
                   : launch(gate_kernel<SRC, 32, 8, BIASED>, dim3(groups_of(a.tokens, 32)), threads, 0, st, a);
    return launch(gate_kernel<SRC, 64, 16, BIASED>, dim3(few), threads, 0, st, a);
}

template <int SRC>
block_status_t run_gate(const GateArgs &a, hipStream_t st)
{
    return a.bias ? run_gate<SRC, true>(a, st) : run_gate<SRC, false>(a, st);
}

template <int DT, bool DENSE>
block_status_t run_gate_grad(const GateGradArgs &a, hipStream_t st)
{
    const dim3 threads(kWavesHere * 64);
    const unsigned few = groups_of(a.tokens, 64);
    if (a.experts <= 64)
        return a.tokens <= kFewTokens
                   ? launch(gate_grad_kernel<DT, 64, 1, DENSE>, dim3(few), threads, 0, st, a)
                   : launch(gate_grad_kernel<DT, 16, 4, DENSE>, dim3(groups_of(a.tokens, 16)), threads, 0, st, a);
    if (a.experts <= 256)
        return a.tokens <= kFewTokens
                   ? launch(gate_grad_kernel<DT, 64, 4, DENSE>, dim3(few), threads, 0, st, a)
                   : launch(gate_grad_kernel<DT, 32, 8, DENSE>, dim3(groups_of(a.tokens, 32)), threads, 0, st, a);
    return launch(gate_grad_kernel<DT, 64, 16, DENSE>, dim3(few), threads, 0, st, a);
}

template <int DT>
block_status_t run_gate_grad(const GateGradArgs &a, hipStream_t st)
{
    return a.scores == BLOCK_SCORES_SOFTMAX && !a.renormalize ? run_gate_grad<DT, true>(a, st)
                                                              : run_gate_grad<DT, false>(a, st);
}

bool good_tokens(int64_t tokens) { return tokens >= 0 && tokens <= (1 << 24); }

int64_t size_of(block_dtype_t dt) { return dt == BLOCK_FP32 ? 4 : 2; }

bool good_dtype(block_dtype_t dt) { return dt == BLOCK_BF16 || dt == BLOCK_FP16 || dt == BLOCK_FP32; }

}  // namespace

namespace block {

block_status_t gate_of_parts(const GateArgs &a, hipStream_t stream) { return run_gate<SRC_PARTS>(a, stream); }

}  // namespace block

extern "C" {

block_status_t block_moe_gate_fwd(const void *logits, block_dtype_t logits_dtype, const float *bias, int32_t *ids,
                                  float *probs, int64_t tokens, int experts, int top_k, block_scores_t scores,
                                  int groups, int top_groups, int group_top, int renormalize, float scale,
                                  const int32_t *valid_tokens, hipStream_t stream)
{
    const GateRule rule = {top_k, (int)scores, groups, top_groups, group_top, renormalize, scale};
    if (!good_tokens(tokens) || !good_gate(rule, experts) || !good_dtype(logits_dtype))
        return BLOCK_ERR_INVALID_ARG;
    if (tokens == 0)
        return BLOCK_OK;
    if (!logits || !ids || !probs)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(probs, 4) ||
        misaligned(valid_tokens, 4))
        return BLOCK_ERR_ALIGNMENT;
    if (any_overlap<2, 3>({{ids, tokens * top_k * 4}, {probs, tokens * top_k * 4}},
                          {{logits, tokens * experts * size_of(logits_dtype)}, {bias, experts * (int64_t)4}, {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    const GateArgs a = {logits, bias, ids, probs, valid_tokens, (int)tokens, experts, 1, rule};
    if (logits_dtype == BLOCK_FP32)
        return run_gate<DT_F32>(a, stream);
    return logits_dtype == BLOCK_BF16 ? run_gate<DT_BF16>(a, stream) : run_gate<DT_F16>(a, stream);
}

block_status_t block_moe_gate_bwd(const void *logits, block_dtype_t logits_dtype, const int32_t *ids,
                                  const float *grad_probs, void *grad_logits, int64_t tokens, int experts, int top_k,
                                  block_scores_t scores, int renormalize, float scale, const int32_t *valid_tokens,
                                  hipStream_t stream)
{
    if (!good_tokens(tokens) || experts < 1 || experts > kGateExperts || top_k < 1 || top_k > kGateSlots ||
        !good_gate_scores((int)scores, scale) || !good_dtype(logits_dtype))
        return BLOCK_ERR_INVALID_ARG;
    if (tokens == 0)
        return BLOCK_OK;
    if (!logits || !ids || !grad_probs || !grad_logits)
        return BLOCK_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(ids, 4) || misaligned(grad_probs, 4) || misaligned(grad_logits, 16) ||
        misaligned(valid_tokens, 4))
        return BLOCK_ERR_ALIGNMENT;
    const int64_t all = tokens * experts * size_of(logits_dtype), pairs = tokens * top_k * 4;
    if (any_overlap<1, 4>({{grad_logits, all}}, {{logits, all}, {ids, pairs}, {grad_probs, pairs}, {valid_tokens, 4}}))
        return BLOCK_ERR_INVALID_ARG;
    const GateGradArgs a = {logits, ids, grad_probs, grad_logits, valid_tokens, (int)tokens, experts, top_k,
                            (int)scores, renormalize, scale};
    if (logits_dtype == BLOCK_FP32)
        return run_gate_grad<DT_F32>(a, stream);
    return logits_dtype == BLOCK_BF16 ? run_gate_grad<DT_BF16>(a, stream) : run_gate_grad<DT_F16>(a, stream);
}

}  // extern "C"
