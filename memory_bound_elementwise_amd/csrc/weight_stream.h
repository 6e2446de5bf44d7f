// The inner loop of products whose cost is reading a weight matrix once: a few rows of x
// against many rows of W (gfx950 matrix cores).
#ifndef MBE_WEIGHT_STREAM_H
#define MBE_WEIGHT_STREAM_H

#include "block_math.h"

namespace block {

constexpr int kLineK = 64;  // 16-bit elements of a 128-byte line

// Offset of a lane that reads nothing: past the end of every resource, so the load returns
// zeros (tensors of these products stay below 2^31 bytes a resource).
constexpr uint32_t kNowhere = 0x80000000u;

// Shared memory of one wave: 128 bytes of each of 16 rows a tile, and of the columns 128 bytes
// of 16 or 256 of 8 a group.
template <int RT, int G>
constexpr int kStage = (RT + G) * 128;  // in 16-byte chunks

// acc[i][g] += 16 rows of W (tile i) times the 16 columns of group g, over k = first, first +
// stride, ... (a step is 64 k; k at and past K count as zeros). All in bytes:
//   w[i]      resource of tile i: its rows that exist, row_bytes apart (others read zeros)
//   x, col    resource of the columns, and where the lane's part of them starts in it:
//     TERMS 1   column 16 g + 8 p + lane / 8, at its octet lane % 8, in col[g][p]
//     TERMS 2   pair 8 g + 4 p + lane / 16, at its octet lane % 16 / 2 and term lane % 2; the
//               terms of a value are two columns, j and j + 8 of pair j, and eight first
//               terms lie before their eight second ones
// stage: kStage<RT, G> chunks of shared memory of the wave's own; the wave needs no barrier.
//
// What bounds it is the rate of the address unit, then memory. The matrix operand's own
// shape (lane 16 q + i holds row i) sends neighbouring lanes to different lines: such a load
// took 64 cycles a CU where one of contiguous lanes takes 16, and the two loads of rows that
// 16 lanes share made it the limit (470 MB: 5.9 TB/s, and 3.8 with 8 tokens an expert). So
// rows are read eight at a time, 128 bytes each, 8 neighbouring lanes a line, which may then
// bypass the caches (nontemporal, 6.8 TB/s), and turn into operands on the way through
// shared memory. Two steps of loads are in flight a wave; 12 to 16 waves a CU make that the
// 64 KB that cover 2 us of latency. (Three or four steps: up product of one token 70 -> 71.5
// us, down 40 -> 44; one step: 74, 41.)
template <int DT, int RT, int G, int TERMS>
__device__ __forceinline__ void stream_products(f32x4 (&acc)[RT][G], const rsrc_t (&w)[RT], uint32_t row_bytes,
                                                rsrc_t x, const uint32_t (&col)[G][2], int K, int first, int stride,
                                                u32x4 *stage)
{
    struct Buf {
        u32x4 w[RT][2], x[G][2];
    };
    const int lane = lane_id();
    const int row = lane / 8, chunk = lane % 8;
    const uint32_t row0 = row * row_bytes + chunk * 16, row1 = row0 + 8 * row_bytes;
    const int kw = chunk * 8, kx = TERMS == 1 ? kw : lane % 16 / 2 * 8;
    auto fetch = [&](Buf &buf, int k) {
        const bool in = k < K - kw, inx = k < K - kx;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            buf.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(w[i], in ? row0 : kNowhere, k * 2, kLoadAux);
            buf.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(w[i], in ? row1 : kNowhere, k * 2, kLoadAux);
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int p = 0; p < 2; ++p)
                buf.x[g][p] = __builtin_amdgcn_raw_buffer_load_b128(x, inx ? col[g][p] : kNowhere, k * 2 * TERMS, 0);
    };
    // chunk c of a row lies at c ^ (row % 8), so that eight lanes that read one chunk of eight
    // rows, or write a row, fall into different banks
    u32x4 *const xs = stage + RT * 128;
    const int put_w = row * 8 + (chunk ^ row);
    const int put_x0 = TERMS == 1 ? put_w : lane / 16 * 16 + (lane % 16 ^ lane / 16);
    const int put_x1 = TERMS == 1 ? put_w + 64 : 64 + lane / 16 * 16 + (lane % 16 ^ (4 + lane / 16));
    const int i16 = lane % 16, q = lane / 16;
    int get_w[2], get_x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        get_w[h] = i16 * 8 + ((4 * h + q) ^ i16 % 8);
        get_x[h] = TERMS == 1 ? get_w[h] : i16 % 8 * 16 + (((4 * h + q) * 2 + i16 / 8) ^ i16 % 8);
    }
    auto multiply = [&](const Buf &buf) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            stage[i * 128 + put_w] = buf.w[i][0];
            stage[i * 128 + 64 + put_w] = buf.w[i][1];
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            xs[g * 128 + put_x0] = buf.x[g][0];
            xs[g * 128 + put_x1] = buf.x[g][1];
        }
        // the lanes of a wave run together and its accesses to shared memory stay in order;
        // the fence keeps the compiler from moving them across
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 b[G];
#pragma unroll
            for (int g = 0; g < G; ++g)
                b[g] = xs[g * 128 + get_x[h]];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const u32x4 a = stage[i * 128 + get_w[h]];
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[i][g] = mfma16<DT>(a, b[g], acc[i][g]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    constexpr int DEPTH = 2;
    Buf buf[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        fetch(buf[d], first + d * stride);
    for (int k = first; k < K;) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            multiply(buf[d]);
            fetch(buf[d], k + DEPTH * stride);  // past K: loads nothing
            k += stride;
        }
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

}  // namespace block

#endif  // MBE_WEIGHT_STREAM_H
