// The expert layer of a few tokens with weights in 4 bits (layout in fp4.h), for AMD Instinct MI355X
// (gfx950). C ABI declared in block/moe_block.h.
//
// y = residual + sum over a token's slots of down (act(up x) p), sums fp32. For a few tokens the cost is
// reading each chosen expert's weights once: 187 MB for one token of 8 of 64 experts, hidden 7168, inter
// 2048 (up 21.4 us, 5.8 TB/s; down 15.8, 3.9 TB/s), 1.5 GB for 64 tokens (162, 6.2 TB/s; 115, 4.3;
// combine 5.3).
//   up       one workgroup a (chosen expert, block of columns of the activation); the activation
//            times the probability goes to the workspace as three bf16 terms, which keep its 24 bits
//   down     the terms are columns of their own. For a few pairs one workgroup 16 columns of
//            the output, all experts: their sums meet in shared memory. Otherwise units of an
//            expert and a block of columns of the output, and a pair's fp32 products go to the workspace
//   combine  adds a token's pairs in slot order, so no atomics are needed and the bits never change
// Workgroups of few columns split k among their waves; where there are more, the waves have rows of W of
// their own and share the columns instead.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "fp4_host.h"
#include "fp4_stream.h"
#include "route_device.h"

namespace {

using namespace block;

constexpr int kWaves = 4;

template <int RT, int G>
__device__ __forceinline__ void clear(f32x4 (&acc)[RT][G])
{
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g)
            acc[i][g] = f32x4{0, 0, 0, 0};
}

struct ExpertArgs {
    const uint16_t *x;
    const uint8_t *up_codes, *up_scales, *down_codes, *down_scales;
    const int *ids;
    const float *probs;
    const uint16_t *residual;
    char *y;
    const int *valid;
    uint16_t *h;  // [3][pairs][inter]
    float *z;     // [parts][pairs][hidden]
    int tokens, hidden, inter, experts, top_k, by_pair;
    int part_bits;  // of parts, a power of two
    float limit;
};

// An fp32 value as the sum of three bf16: its first 8 bits, the next 8 and the rest (nothing is
// lost, but below 2^-109, where the last term runs out of exponents; what is below 2^-133 is 0). Of
// an infinity or a NaN the first term is one and the others zero.
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

// Four neighbours' terms, one plane after the other.
__device__ __forceinline__ void store_terms(const f32x4 &h, uint16_t *to, int64_t plane)
{
    uint16_t t[4][3];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        three_terms(h[r], t[r]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        *reinterpret_cast<u32x2 *>(to + q * plane) =
            u32x2{t[0][q] | (uint32_t)t[1][q] << 16, t[2][q] | (uint32_t)t[3][q] << 16};
}

// The workgroup's expert: blockIdx.y is a pair, which stands for its expert if no earlier one has the
// same, or an expert, whichever is fewer. -1: none.
__device__ __forceinline__ int own_expert(const ExpertArgs &a, int pairs)
{
    int e = blockIdx.y;
    if (a.by_pair) {
        e = e < pairs ? a.ids[e] : -1;
        if (e >= a.experts)
            e = -1;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// The pairs (token * top_k + slot) below `pairs` whose id is e, in increasing order, into list;
// returns their number, or 0 where an earlier workgroup has them. W waves look through ids
// together, 64 pairs a chunk. counts: of the chunks.
template <int W>
__device__ __forceinline__ int expert_pairs(const ExpertArgs &a, int pairs, int e, uint16_t *list, int (&counts)[kMaxPairs / 64])
{
    constexpr int kOwn = kMaxPairs / 64 / W;
    const int lane = lane_id(), wave = wave_in_block(), chunks = (pairs + 63) / 64;
    uint64_t found[kOwn];
    int id[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int p = (wave + i * W) * 64 + lane;
        id[i] = p < pairs ? a.ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        found[i] = __ballot(id[i] == e);
        if (lane == 0)
            counts[wave + i * W] = __popcll(found[i]);
    }
    sync_shared();
    int n = 0;
    for (int c = 0; c < chunks; ++c) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (c == wave + i * W && id[i] == e)
                list[n + __popcll(found[i] & (((uint64_t)1 << lane) - 1))] = (uint16_t)(c * 64 + lane);
        n += counts[c];
    }
    sync_shared();
    return n == 0 || (a.by_pair && list[0] != (int)blockIdx.y) ? 0 : __builtin_amdgcn_readfirstlane(n);
}

// The same by one wave for up to 64 pairs: id holds the lane's pair's. The list is the wave's own.
__device__ __forceinline__ int list_few(int id, int e, uint16_t *list)
{
    const uint64_t found = __ballot(id == e);
    const int lane = lane_id();
    if (id == e)
        list[__popcll(found & (((uint64_t)1 << lane) - 1))] = (uint16_t)lane;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return __popcll(found);
}

// The lane's pair's id, -1 for none or one outside the experts (up to 64 pairs).
__device__ __forceinline__ int few_ids(const ExpertArgs &a, int pairs)
{
    const int lane = lane_id(), id = lane < pairs ? a.ids[lane] : -1;
    return id >= 0 && id < a.experts ? id : -1;
}

// FEW: up to 64 pairs. Up to 4 NX tokens of an expert share one read of its weights; an expert with
// more reads them again. What one token costs beyond its weights is one chain of loads: ids, then
// (tiles are sent for before the pairs are looked through) tiles and x. (Eight waves a workgroup 24.2
// us, four steps in flight 22.2, seven 22.7, for 21.4.)
template <int ACT, int NX, bool FEW>
__global__ __launch_bounds__(kWaves * 64) void fp4_up_kernel(ExpertArgs a)
{
    constexpr int RT = ACT == ACT_SWIGLU ? 2 : 1;  // gate and up, or the one product
    constexpr int kStages = kWaves * NX * 64, kSums = kWaves * RT * 64;
    __shared__ u32x4 shared[kStages > kSums ? kStages : kSums];  // the waves' stages, then their sums
    __shared__ uint16_t lists[FEW ? kWaves * 64 : kMaxPairs];
    __shared__ int counts[kMaxPairs / 64];
    const int lane = lane_id(), wave = wave_in_block();
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k;
    int id = -1, e;
    if constexpr (FEW) {
        id = few_ids(a, pairs);
        e = a.by_pair ? ((int)blockIdx.y < pairs ? __builtin_amdgcn_readlane(id, blockIdx.y) : -1) : (int)blockIdx.y;
    } else {
        e = own_expert(a, pairs);
    }
    if (e < 0)
        return;
    const int k_tiles = (a.hidden + kFp4K - 1) / kFp4K, blocks = a.inter / 16;
    Tiles w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        w[i] = tiles_of(a.up_codes, a.up_scales, ((int64_t)e * RT + i) * blocks + blockIdx.x, k_tiles);
    Stream<RT, NX, 2> stream;
    stream.start(w, wave, kWaves);
    uint16_t *list = lists;
    int n;
    if constexpr (FEW) {
        list += wave * 64;
        n = list_few(id, e, list);
        if (n == 0 || (a.by_pair && list[0] != (int)blockIdx.y))
            return;  // all of the workgroup: no barrier is behind or ahead of it
    } else {
        n = expert_pairs<kWaves>(a, pairs, e, list, counts);
    }
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.hidden * 2u);
    const int64_t plane = (int64_t)a.tokens * a.top_k * a.inter;
    for (int p = 0; p < n; p += 4 * NX) {
        uint32_t col[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int s = p + 4 * i + lane / 16;
            col[i] = s < n ? (uint32_t)(list[s] / a.top_k) * (uint32_t)a.hidden * 2u + lane % 16 * 16 : kNowhere;
        }
        f32x4 acc[RT] = {};
        if (p > 0) {
            __syncthreads();  // the sums have been read
            stream.start(w, wave, kWaves);
        }
        stream.run(acc, w, x, col, a.hidden, wave, kWaves, shared + wave * NX * 64);
        __syncthreads();
        f32x4 *joined = reinterpret_cast<f32x4 *>(shared);
#pragma unroll
        for (int i = 0; i < RT; ++i)
            joined[(wave * RT + i) * 64 + lane] = acc[i];
        __syncthreads();
        const int row = threadIdx.x % 16, s = p + threadIdx.x / 16;
        if (s >= n || (int)threadIdx.x / 16 >= 4 * NX)
            continue;
        float z[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            z[i] = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q)
                z[i] += joined[(q * RT + i) * 64 + row / 4 * 16 + (s - p)][row % 4];
        }
        const int pair = list[s];
        uint16_t term[3];
        three_terms((ACT == ACT_SWIGLU ? swiglu(z[0], z[RT - 1], a.limit) : squared_relu(z[0])) * a.probs[pair], term);
        uint16_t *to = a.h + (int64_t)pair * a.inter + blockIdx.x * 16 + row;
#pragma unroll
        for (int q = 0; q < 3; ++q)
            to[q * plane] = term[q];
    }
}

// Up products where experts have many tokens: a workgroup takes one expert and kManyWaves times two
// row tiles, which walk k together (Walk), so that x is read once for all of them. A wave has gate
// and up of 16 columns of the activation, or 32 columns of one product. Bound by the stream of weights:
// 64 tokens, 7168 x 2048, 64 experts 162 us. (Four steps in flight 164; weights kept in the caches
// 180; without the scales' loads 150.)
constexpr int kManyWaves = 8;

template <int G>
using UpWalk = Walk<2, G, kManyWaves, 2, false>;

template <int ACT, int G>
__device__ __forceinline__ void up_many_pass(const ExpertArgs &a, UpWalk<G> &walk, typename UpWalk<G>::Ends &ends, int c0,
                                             const uint16_t *list, int n, u32x4 *xs)
{
    constexpr int W = kManyWaves;
    const int lane = lane_id(), wave = wave_in_block();
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.hidden * 2u);
#pragma unroll
    for (int i = 0; i < UpWalk<G>::kLoads; ++i) {
        const int s = 4 * (wave + i * W) + lane / 16;
        ends.col[i] = s < n ? (uint32_t)(list[s] / a.top_k) * (uint32_t)a.hidden * 2u + lane % 16 * 16 : kNowhere;
    }
    f32x4 acc[2][G];
    clear(acc);
    ends.K = a.hidden;
    walk.start_columns(x, ends);
    walk.run(acc, x, ends, ends, (n + 15) / 16, xs);
    if (c0 >= a.inter)
        return;
    const int64_t plane = (int64_t)a.tokens * a.top_k * a.inter;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int s = g * 16 + lane % 16;
        if (s >= n)
            continue;
        const int pair = list[s];
        const float p = a.probs[pair];
        uint16_t *to = a.h + (int64_t)pair * a.inter + c0 + lane / 16 * 4;
        if constexpr (ACT == ACT_SWIGLU) {
            f32x4 h;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                h[r] = swiglu(acc[0][g][r], acc[1][g][r], a.limit) * p;
            store_terms(h, to, plane);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 h;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    h[r] = squared_relu(acc[i][g][r]) * p;
                store_terms(h, to + 16 * i, plane);
            }
        }
    }
}

template <int ACT, int G>
__global__ __launch_bounds__(kManyWaves * 64, G == 1 ? 8 : 4) void fp4_up_many_kernel(ExpertArgs a)
{
    __shared__ u32x4 xs[2 * G * 256];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int counts[kMaxPairs / 64];
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k, e = own_expert(a, pairs);
    if (e < 0)
        return;
    constexpr int kCols = ACT == ACT_SWIGLU ? 16 : 32;
    const int c0 = (blockIdx.x * kManyWaves + wave_in_block()) * kCols, blocks = a.inter / 16;
    const int k_tiles = c0 < a.inter ? (a.hidden + kFp4K - 1) / kFp4K : 0;  // past the end: none, but its part of x
    typename UpWalk<G>::Ends ends;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        ends.w.block[i] = tiles_of(a.up_codes, a.up_scales,
                             k_tiles == 0 ? 0 : (ACT == ACT_SWIGLU ? ((int64_t)e * 2 + i) * blocks : (int64_t)e * blocks + i) + c0 / 16,
                             k_tiles);
    UpWalk<G> walk;
    walk.start_tiles(ends);  // on their way while the pairs are looked for
    const int n = expert_pairs<kManyWaves>(a, pairs, e, list, counts);
    for (int p = 0; p < n; p += G * 16) {
        const int m = n - p < G * 16 ? n - p : G * 16;
        if (p > 0) {
            sync_shared();  // what is in xs has been read
            walk.start_tiles(ends);
        }
        up_many_pass<ACT, G>(a, walk, ends, c0, list + p, m, xs);
    }
}

// A group of 16 columns holds the three terms of five pairs, columns 3 p + 0 .. 2. The sum of a
// pair's three is then in the lane of the first.
constexpr int kPairs = 5;

// An infinite weight, or activation, makes the first terms' sum infinite or NaN as the product of the
// whole would be; the further terms may be zeros, which times an infinity would make a NaN of it.
__device__ __forceinline__ f32x4 join_terms(const f32x4 &v)
{
    f32x4 z;
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // row_shl: what the next lane and the one behind it hold
        const float all = v[r] + dpp<0x101>(v[r]) + dpp<0x102>(v[r]);
        z[r] = __builtin_isinf(v[r]) ? v[r] : all;
    }
    return z;
}

// Where column c of the group that starts at pair s0 of the list starts in h, or kNowhere.
__device__ __forceinline__ uint32_t term_column(const ExpertArgs &a, const uint16_t *list, int n, int s0, int c)
{
    const int s = s0 + c / 3;
    const uint32_t pairs = (uint32_t)(a.tokens * a.top_k);
    return c < 3 * kPairs && s < n ? ((uint32_t)(c % 3) * pairs + list[s]) * (uint32_t)a.inter * 2u : kNowhere;
}

__device__ __forceinline__ rsrc_t terms_of(const ExpertArgs &a)
{
    return make_rsrc(a.h, 3u * (uint32_t)(a.tokens * a.top_k) * (uint32_t)a.inter * 2u);
}

// Down product of up to 64 pairs: a workgroup takes 16 columns of the output, its waves the chosen
// experts in turn, each in `parts` parts of k so that all have work; the pairs' sums meet in
// shared memory and are added in slot order. NX 1: a pair at a time, 4: five. One token's eight
// experts are one round of 3.5 waves a SIMD, whose start and end are half of its 15.8 us. (Six or
// eight steps in flight 17.3, sixteen waves a workgroup 18.2.)
constexpr int kFewWaves = 8, kFewPairs = 64;

template <int YDT, int NX>
__global__ __launch_bounds__(kFewWaves * 64) void fp4_down_few_kernel(ExpertArgs a, int parts)
{
    constexpr int kTogether = NX == 1 ? 1 : kPairs;
    __shared__ u32x4 stages[kFewWaves * NX * 64];
    __shared__ f32x4 sums[kFewPairs * 4];  // [pair][part][16]
    __shared__ uint16_t lists[kFewWaves * 64];
    __shared__ int ids[kFewPairs];
    const int lane = lane_id(), wave = wave_in_block();
    const int live = live_tokens(a.valid, a.tokens), pairs = live * a.top_k;
    const int id = few_ids(a, pairs), k_tiles = (a.inter + kFp4K - 1) / kFp4K;
    const rsrc_t h = terms_of(a);
    uint16_t *list = lists + wave * 64;
    if (wave == 0)
        ids[lane] = id;
    // The token that the thread adds up at the end and the next one, with their part of the residual
    const int c = threadIdx.x % 16, first = threadIdx.x / 16;
    constexpr int kTokensHere = kFewWaves * 4, kTurns = kFewPairs / kTokensHere;
    float residual[kTurns] = {};
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int t = first + i * kTokensHere;
            residual[i] = load1<DT_BF16>(a.residual, (int64_t)(t < a.tokens ? t : 0) * a.hidden + blockIdx.x * 16 + c);
        }
    }
    for (int u = wave; u < pairs * parts; u += kFewWaves) {
        const int p = u / parts, part = u % parts, e = __builtin_amdgcn_readlane(id, p);
        if (e < 0 || (int)__builtin_ctzll(__ballot(id == e)) != p)
            continue;  // none, or an earlier pair stands for its expert
        const Tiles w[1] = {tiles_of(a.down_codes, a.down_scales, (int64_t)e * (a.hidden / 16) + blockIdx.x, k_tiles)};
        Stream<1, NX, NX == 1 ? 4 : 2> stream;
        stream.start(w, part, parts);
        const int n = list_few(id, e, list);
        for (int s0 = 0; s0 < n; s0 += kTogether) {
            uint32_t col[NX];
#pragma unroll
            for (int i = 0; i < NX; ++i)
                col[i] = NX == 1 && lane / 16 == 3 ? kNowhere
                                                   : term_column(a, list, n, s0, 4 * i + lane / 16) + lane % 16 * 16;
            if (s0 > 0)
                stream.start(w, part, parts);
            f32x4 acc[1] = {};
            stream.run(acc, w, h, col, a.inter, part, parts, stages + wave * NX * 64);
            const f32x4 z = join_terms(acc[0]);
            const int c = lane % 16, s = s0 + c / 3;
            if (c % 3 == 0 && c < 3 * kTogether && s < n)
                sums[(list[s] * parts + part) * 4 + lane / 16] = z;
        }
    }
    __syncthreads();
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn) {
        const int t = first + turn * kTokensHere;
        if (t >= live)
            return;
        float v = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int p = t * a.top_k + j;
            if (ids[p] < 0)
                continue;
            for (int i = 0; i < parts; ++i)
                v += sums[(p * parts + i) * 4 + c / 4][c % 4];
        }
        store1<YDT>(a.y, (int64_t)t * a.hidden + blockIdx.x * 16 + c, v + residual[turn]);
    }
}

// Down products where experts have many tokens: units of one expert, up to G * 5 of its pairs, eight
// waves of two row tiles (256 columns of the output) and one of `parts` parts of k. A workgroup takes every gridDim.x-th unit,
// and its walk over one ends by sending for the next one's first steps: k is short here (2048: 16
// steps). Its pairs' terms come from cache, 12 KB a pair and unit beside the unit's 278 KB of weights.
// 64 tokens, 7168 x 2048, 64 experts: 115 us in a trace, 105 at best; when that was 107, a workgroup a
// unit took 126, and the weights' stream and the stores of z alone 93. (Four waves of four tiles 115,
// four of two 158, sixteen of one 141, four steps in flight 118.)
constexpr int kDownWaves = 8, kDownTiles = 2;

template <int G>
__global__ __launch_bounds__(kDownWaves * 64, 4) void fp4_down_many_kernel(ExpertArgs a)
{
    using DownWalk = Walk<kDownTiles, G, kDownWaves, 2, true>;
    constexpr int kThreads = kDownWaves * 64, kOnce = G * kPairs;  // pairs of a unit
    __shared__ u32x4 xs[2 * G * 256];
    __shared__ uint16_t loose[kMaxPairs], list[kMaxPairs];
    __shared__ uint16_t unit_at[kMaxPairs], unit_end[kMaxPairs], unit_expert[kMaxPairs];
    __shared__ int start[kMaxExperts];  // first counts, then where an expert's next pair goes
    __shared__ int unit_count;
    const int lane = lane_id(), wave = wave_in_block(), tid = threadIdx.x;
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k;
    for (int e = tid; e < a.experts; e += kThreads)
        start[e] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int e = a.ids[p];
        if (e >= 0 && e < a.experts)
            atomicAdd(&start[e], 1);
    }
    __syncthreads();
    if (wave == 0) {  // where each expert's pairs start, and its units
        int at = 0, units = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int n = e0 + lane < a.experts ? start[e0 + lane] : 0, own = (n + kOnce - 1) / kOnce;
            int sum = n, count = own;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int s = __shfl_up(sum, d), c = __shfl_up(count, d);
                sum += lane >= d ? s : 0;
                count += lane >= d ? c : 0;
            }
            const int first = at + sum - n;
            if (e0 + lane < a.experts)
                start[e0 + lane] = first;
            for (int i = 0; i < own; ++i) {
                const int u = units + count - own + i;
                unit_expert[u] = (uint16_t)(e0 + lane);
                unit_at[u] = (uint16_t)(first + i * kOnce);
                unit_end[u] = (uint16_t)(first + (i + 1) * kOnce < first + n ? first + (i + 1) * kOnce : first + n);
            }
            at += __shfl(sum, 63);
            units += __shfl(count, 63);
        }
        if (lane == 0)
            unit_count = units;
    }
    __syncthreads();
    // The pairs by expert, each expert's in any order at first, then in increasing order: workgroups
    // share an expert's pairs, so all of them have to cut the same list.
    for (int p = tid; p < pairs; p += kThreads) {
        const int e = a.ids[p];
        if (e >= 0 && e < a.experts)
            loose[atomicAdd(&start[e], 1)] = (uint16_t)p;
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int e = a.ids[p];
        if (e < 0 || e >= a.experts)
            continue;
        const int first = e > 0 ? start[e - 1] : 0, end = start[e];  // its end is where the next one starts
        int before = 0;
#pragma unroll 8
        for (int i = first; i < end; ++i)
            before += loose[i] < p;
        list[first + before] = (uint16_t)p;
    }
    __syncthreads();

    const int blocks = a.hidden / 16, row_units = (blocks + kDownWaves * kDownTiles - 1) / (kDownWaves * kDownTiles);
    const int parts = 1 << a.part_bits, each = row_units * parts, units = unit_count * each, k_tiles = (a.inter + kFp4K - 1) / kFp4K;
    const int part_tiles = (k_tiles + parts - 1) >> a.part_bits;
    const rsrc_t h = terms_of(a);
    auto block_of = [&](int u) { return ((u % each >> a.part_bits) * kDownWaves + wave) * kDownTiles; };
    auto ends_of = [&](typename DownWalk::Ends &ends, int u) {
        const bool there = u < units;  // past the last one: nothing is loaded
        const int at = there ? u / each : 0;
        const int e = __builtin_amdgcn_readfirstlane(unit_expert[at]), b0 = block_of(u);
        const int from = __builtin_amdgcn_readfirstlane(unit_at[at]), n = __builtin_amdgcn_readfirstlane(unit_end[at]) - from;
        const int rows = !there || b0 >= blocks ? 0 : (blocks - b0 < kDownTiles ? blocks - b0 : kDownTiles);
        const int t0 = (u & (parts - 1)) * part_tiles, left = k_tiles - t0;  // parts are no more than would leave one empty
        ends.w = run_of(a.down_codes, a.down_scales, rows ? (int64_t)e * blocks + b0 : 0, k_tiles, rows, t0,
                        left < part_tiles ? left : part_tiles);
        ends.K = left <= part_tiles ? a.inter - t0 * kFp4K : part_tiles * kFp4K;
#pragma unroll
        for (int i = 0; i < DownWalk::kLoads; ++i) {
            const int c = 4 * (wave + i * kDownWaves) + lane / 16;
            ends.col[i] = there ? term_column(a, list + from, n, c / 16 * kPairs, c % 16) + t0 * kFp4K * 2 + lane % 16 * 16 : kNowhere;
        }
    };
    int u = blockIdx.x;
    if (u >= units)
        return;
    typename DownWalk::Ends ends, next;
    DownWalk walk;
    ends_of(ends, u);
    walk.start_tiles(ends);
    walk.start_columns(h, ends);
    for (; u < units; u += gridDim.x) {
        const int at = u / each, b0 = block_of(u);
        const int from = __builtin_amdgcn_readfirstlane(unit_at[at]), n = __builtin_amdgcn_readfirstlane(unit_end[at]) - from;
        ends_of(next, u + gridDim.x);
        f32x4 acc[kDownTiles][G];
        clear(acc);
        walk.run(acc, h, ends, next, (n + kPairs - 1) / kPairs, xs);
        float *to = a.z + (int64_t)(u & (parts - 1)) * a.tokens * a.top_k * a.hidden + b0 * 16 + lane / 16 * 4;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int c = lane % 16, s = g * kPairs + c / 3;
#pragma unroll
            for (int i = 0; i < kDownTiles; ++i) {
                const f32x4 z = join_terms(acc[i][g]);
                if (c < 15 && c % 3 == 0 && s < n && b0 + i < blocks)
                    *reinterpret_cast<f32x4 *>(to + (int64_t)list[from + s] * a.hidden + i * 16) = z;
            }
        }
        ends = next;
    }
}

// y = residual + a token's products in slot order. A lane takes four neighbouring columns.
template <int YDT>
__global__ __launch_bounds__(256) void fp4_combine_kernel(ExpertArgs a)
{
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;  // up to 2^26
    if (i >= live_tokens(a.valid, a.tokens) * a.hidden)
        return;
    const int t = i / a.hidden, c = i % a.hidden;
    const u32x2 residual = a.residual ? *reinterpret_cast<const u32x2 *>(a.residual + i) : u32x2{0, 0};
    f32x4 v = {0, 0, 0, 0};
    constexpr int kTogether = 8;  // loads that go out together
    const int parts = 1 << a.part_bits, all = a.top_k * parts;  // a slot's parts follow each other
    const int64_t plane = (int64_t)a.tokens * a.top_k * a.hidden;
    for (int j0 = 0; j0 < all; j0 += kTogether) {
        f32x4 z[kTogether];
        bool in[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            const int item = j0 + j < all ? j0 + j : 0, pair = t * a.top_k + (item >> a.part_bits), e = a.ids[pair];
            in[j] = j0 + j < all && e >= 0 && e < a.experts;
            // unwritten where the id is none
            z[j] = *reinterpret_cast<const f32x4 *>(a.z + (item & (parts - 1)) * plane + (int64_t)pair * a.hidden + c);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
            if (in[j])
                v += z[j];
    }
    if (a.residual)
        v += f32x4{bf16_lo(residual[0]), bf16_hi(residual[0]), bf16_lo(residual[1]), bf16_hi(residual[1])};
    if constexpr (YDT == DT_F32)
        *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.y) + i) = v;
    else
        *reinterpret_cast<u32x2 *>(reinterpret_cast<uint16_t *>(a.y) + i) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
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

// Groups of pairs that share a read of an expert's weights: enough for one and a half times the
// pairs an expert has on average. (Enough for the average, and for twice it: up, 128 tokens, 7168 x
// 2048, 64 experts, top 8, 264 and 185 us for 185; down, 32 tokens, 113 and 99 for 101.)
int pair_groups(const ExpertSizes &s, int group)
{
    const int64_t some = ceil_div(3 * s.tokens * s.top_k, 2 * s.experts);
    const int64_t each = s.tokens < some ? s.tokens : some;
    return each <= group ? 1 : (each <= 2 * group ? 2 : (each <= 3 * group ? 3 : 4));
}

// Whether the up product's workgroups take many rows of W, whose waves share the columns, or 16 rows,
// whose waves split k: the former for more tokens than a few, where that leaves two workgroups a CU, or
// one for every other CU where experts may have so many tokens that the latter read their weights
// again. (us, shared and split k: 7168 x 2048, 8 of 64 experts, 2 tokens 43.9 and 39.7, 4 tokens 67.8
// and 66.5, 8 tokens, 1024 workgroups, of which 736 found an expert, 123.6 and 127.0, 64 tokens 160 and
// 211; 8 tokens, 2048 x 8192, 4 of 8, 512 workgroups 27.7 and 33.8; 4096 x 4096, 2 of 8, 256
// workgroups, 12 tokens 34.8 and 28.5, 64 tokens 37.4 and 48.6; 128 tokens, 2048 x 1408, 8 of 16, 176
// workgroups 55.4 and 69.9; 100 tokens, 4096 x 512, 2 of 8, 32 workgroups 36.1 and 17.6.)
bool up_shares(const ExpertArgs &a, int columns, unsigned experts)
{
    const bool many = a.tokens * a.top_k > kFewPairs;
    return (a.tokens > 4 || many) && ceil_div(a.inter, kManyWaves * columns) * experts >= (many ? 128 : 512);
}

// Experts that may have a token, times the blocks of rows of their down product.
int64_t down_units(const ExpertSizes &s)
{
    const int64_t pairs = s.tokens * s.top_k;
    return ceil_div(s.hidden, kDownWaves * kDownTiles * 16) * (pairs < s.experts ? pairs : s.experts);
}

// Whether the down product goes expert by expert, with a combine behind it, or in one kernel, 16 columns
// of the output a workgroup: the former for more pairs than the latter holds, where there are units
// for every CU, and where the latter's waves have several long turns. (us, with 4 to 5 for the combine
// not added, and in one: 2 tokens, 7168 x 2048, 8 of 64 experts 29.1 and 38.2; 2 of 8 experts of 4096 x
// 4096, 4 tokens 17.1 and 18.4, 8 tokens 18.4 and 30.6, 32 tokens 31.8 and 58.8; 4 tokens, 4 of 8 of 2048 x
// 8192 18.3 and 42.9; 16 tokens, 4 of 16 of 1024 x 512 7.9 and 12.9, of 1024 x 1024 10.5 and 18.1.)
bool down_by_expert(const ExpertSizes &s)
{
    const int64_t pairs = s.tokens * s.top_k;
    return pairs > kFewPairs || (s.tokens > 1 && down_units(s) >= 256) || (pairs > kFewWaves && pairs * s.inter >= (1 << 16));
}

// Parts of k of the down product by expert: more where the units are fewer than two a CU, of eight steps
// at least. (us, in one and in parts: 4096 x 14336, 2 of 8 experts, 16 tokens 89 and 54.5, 64 tokens 125
// and 82.5, 128 tokens 166 and 132; 8 tokens, 2048 x 8192, 4 of 8 48.8 and 19.7; 64 tokens, 4096 x 2048, 2
// of 8 23.6 and 21.4.)
int down_part_bits(const ExpertSizes &s)
{
    const int64_t steps = ceil_div(s.inter, kFp4K);
    int bits = 0;
    while (down_by_expert(s) && bits < 3 && down_units(s) << (bits + 1) <= 512 && steps >= 16 << bits)
        ++bits;
    return bits;
}

// Workspace: the activations' terms, then the pairs' products.
int64_t h_bytes(const ExpertSizes &s) { return round_up(s.tokens * s.top_k * s.inter * 6, 16); }
int64_t expert_bytes(const ExpertSizes &s) { return h_bytes(s) + (s.tokens * s.top_k * s.hidden * 4 << down_part_bits(s)); }

template <int ACT>
block_status_t launch_up(const ExpertArgs &a, int groups, unsigned each, hipStream_t st)
{
    constexpr int kCols = ACT == ACT_SWIGLU ? 16 : 32;
    if (up_shares(a, kCols, each)) {
        const dim3 grid((unsigned)ceil_div(a.inter, kManyWaves * kCols), each), threads(kManyWaves * 64);
        if (groups == 1)
            return launch(fp4_up_many_kernel<ACT, 1>, grid, threads, 0, st, a);
        if (groups == 2)
            return launch(fp4_up_many_kernel<ACT, 2>, grid, threads, 0, st, a);
        return launch(fp4_up_many_kernel<ACT, 4>, grid, threads, 0, st, a);
    }
    const dim3 grid((unsigned)(a.inter / 16), each), threads(kWaves * 64);
    if (a.tokens * a.top_k > kFewPairs)
        return launch(fp4_up_kernel<ACT, 4, false>, grid, threads, 0, st, a);
    return a.tokens <= 4 ? launch(fp4_up_kernel<ACT, 1, true>, grid, threads, 0, st, a)
                         : launch(fp4_up_kernel<ACT, 4, true>, grid, threads, 0, st, a);
}

// Parts of k of the down product of few pairs: as many as still leave a wave one turn. (One token, two
// experts, 4096 x 8192: 17.3 us in one part, 9.2 in four.)
int few_parts(const ExpertArgs &a)
{
    const int pairs = a.tokens * a.top_k;
    int parts = 1;
    while (pairs * parts * 2 <= kFewWaves && parts * 2 * kFp4K <= a.inter)
        parts *= 2;
    return parts;
}

template <int YDT>
block_status_t launch_down(const ExpertArgs &a, const ExpertSizes &s, unsigned each, hipStream_t st)
{
    const int pairs = a.tokens * a.top_k, groups = pair_groups(s, kPairs);
    block_status_t r;
    if (down_by_expert(s)) {
        // as many workgroups as fit, and of these as many as have the same number of units
        const int64_t units = ceil_div(a.hidden, kDownWaves * kDownTiles * 16) * (each + pairs / (groups * kPairs)) << a.part_bits;
        const int64_t fit = 256 * 2;
        const dim3 grid((unsigned)ceil_div(units, ceil_div(units, fit))), threads(kDownWaves * 64);
        if (groups == 1)
            r = launch(fp4_down_many_kernel<1>, grid, threads, 0, st, a);
        else if (groups == 2)
            r = launch(fp4_down_many_kernel<2>, grid, threads, 0, st, a);
        else if (groups == 3)
            r = launch(fp4_down_many_kernel<3>, grid, threads, 0, st, a);
        else
            r = launch(fp4_down_many_kernel<4>, grid, threads, 0, st, a);
    } else {
        const dim3 grid((unsigned)(a.hidden / 16)), threads(kFewWaves * 64);
        return a.tokens == 1 ? launch(fp4_down_few_kernel<YDT, 1>, grid, threads, 0, st, a, few_parts(a))
                             : launch(fp4_down_few_kernel<YDT, 4>, grid, threads, 0, st, a, few_parts(a));
    }
    return r ? r : launch(fp4_combine_kernel<YDT>, dim3((unsigned)ceil_div((int64_t)a.tokens * a.hidden, 1024)), dim3(256), 0, st, a);
}

}  // namespace

extern "C" {

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
    a.limit = limit, a.part_bits = down_part_bits(s);
    const int64_t pairs = tokens * top_k;
    a.by_pair = pairs < n_experts;
    const unsigned each = (unsigned)(a.by_pair ? pairs : n_experts);
    const int groups = pair_groups(s, 16);
    if (const block_status_t r = act == BLOCK_ACT_SWIGLU ? launch_up<ACT_SWIGLU>(a, groups, each, stream)
                                                         : launch_up<ACT_SQUARED_RELU>(a, groups, each, stream))
        return r;
    return y_dtype == BLOCK_FP32 ? launch_down<DT_F32>(a, s, each, stream) : launch_down<DT_BF16>(a, s, each, stream);
}

}  // extern "C"
