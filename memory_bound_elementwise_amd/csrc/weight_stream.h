// The inner loop of products whose cost is reading a weight matrix once: a few rows of x
// against many rows of W (gfx950 matrix cores).
#ifndef MBE_WEIGHT_STREAM_H
#define MBE_WEIGHT_STREAM_H

#include "block_math.h"

namespace block {

constexpr int kStreamUnroll = 4;                   // matrix instructions (of 32 k) a step
constexpr int kStreamStep = 32 * kStreamUnroll;    // k of one step of a wave

// acc[i][g] += W rows of tile i times the x rows of group g, over k = first, first + stride,
// ... (a step is kStreamStep k; k at and past K count as zeros). w[i], b[s][g]: where the
// lane's own row starts, already moved to its k octet (8 (lane / 16) elements in). Weights
// go straight from memory to the registers that feed the matrix cores: each is used by one
// wave only, so shared memory would add a trip and save none. The next step's loads are
// issued before this step's products. S sources of b share the accumulator (a value held as
// a sum of S 16-bit terms).
template <int DT, int RT, int G, int S>
__device__ __forceinline__ void stream_products(f32x4 (&acc)[RT][G], const uint16_t *const (&w)[RT],
                                                const uint16_t *const (&b)[S][G], int bscale, int K, int first,
                                                int stride)
{
    constexpr int U = kStreamUnroll;
    const int k8 = lane_id() / 16 * 8;
    u32x4 wa[RT][U], xa[S][G][U];
    auto fetch = [&](int k0) {
        const bool whole = k0 + kStreamStep <= K;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 32 * u;
            // past K: read the row's start instead, and drop it
            const bool in = whole || k + k8 < K;
            const int at = in ? k : -k8;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(w[i] + at);
                wa[i][u] = in ? v : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(b[s][g] + at * bscale);
                    xa[s][g][u] = in ? v : u32x4{0, 0, 0, 0};
                }
        }
    };
    if (first >= K)
        return;
    fetch(first);
    for (int k0 = first; k0 < K;) {
        u32x4 wc[RT][U], xc[S][G][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wc[i][u] = wa[i][u];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    xc[s][g][u] = xa[s][g][u];
        }
        k0 += stride;
        if (k0 < K)
            fetch(k0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        acc[i][g] = mfma16<DT>(wc[i][u], xc[s][g][u], acc[i][g]);
    }
}

}  // namespace block

#endif  // MBE_WEIGHT_STREAM_H
