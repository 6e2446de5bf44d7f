// Device helpers shared by the router, the gate and the expert layers of libmoe_block.so.
#ifndef MBE_ROUTE_DEVICE_H
#define MBE_ROUTE_DEVICE_H

#include "block_device.h"

namespace block {

constexpr int kMaxPairs = 1024;    // tokens * top_k
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ int live_tokens(const int *valid, int tokens)
{
    if (!valid)
        return tokens;
    const int v = *valid;
    return v < 0 ? 0 : (v < tokens ? v : tokens);
}

// A double as an unsigned integer in the same order; +0 and -0 alike, NaN above all.
__device__ __forceinline__ uint64_t order_key(double v)
{
    if (v != v)
        return ~(uint64_t)0;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return b >> 63 ? ~b : b | (uint64_t)1 << 63;
}

template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ double dpp64(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)b, kCtrl, kRowMask, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), kCtrl, kRowMask, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)(unsigned)hi << 32 | (unsigned)lo);
}

// The value that lane `from` (the same in all lanes) holds.
__device__ __forceinline__ double of_lane(double v, int from)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)b, from);
    const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(b >> 32), from);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// wave_sum in fp64. The softmax stays in fp64 until its weights are rounded: with the difference
// of two logits rounded to fp32 a weight e^-d was off by d steps.
__device__ __forceinline__ double wave_sum64(double v)
{
    v += dpp64<0xB1>(v);
    v += dpp64<0x4E>(v);
    v += dpp64<0x141>(v);
    v += dpp64<0x140>(v);
    v += dpp64<0x142, 0xa>(v);
    v += dpp64<0x143, 0xc>(v);
    return of_lane(v, 63);
}

// The sum of a logit's parts in order, eight loads at a time (a loop of single loads waits
// for each: 3 us for seven).
__device__ __forceinline__ double sum_parts(const double *mine, int64_t part, int parts)
{
    double v = 0.0;
    for (int s = 0; s < parts; s += 8) {
        double p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = mine[(s + i < parts ? s + i : 0) * part];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += s + i < parts ? p[i] : 0.0;
    }
    return v;
}

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

}  // namespace block

#endif  // MBE_ROUTE_DEVICE_H
