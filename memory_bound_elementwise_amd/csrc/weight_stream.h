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

// Shared memory of one wave, in 16-byte chunks: 128 bytes of each of 16 rows a tile, and of the
// columns 128 bytes of 16 a group, or (WIDE) three terms of 8 for one group at a time. Waves that
// share their columns have two sets of every group's terms together, and a stage for rows each.
constexpr int kTerms = 192;
template <int G, int SHARE>
constexpr int kOwnLoads = (2 * G + SHARE - 1) / SHARE;  // a wave's loads of columns a step
template <int RT, int G, bool WIDE>
constexpr int kStage = RT * 128 + (WIDE ? kTerms : G * 128);

// The largest number of eight bits below |v|, with v's sign; +0 for +0.
__device__ __forceinline__ float eight_bits_below(float v)
{
    return __uint_as_float(__builtin_elementwise_sub_sat(__float_as_uint(v), 1u) & 0xffff0000u);
}

// An fp32 value (not -0) as three bf16, h = 2 a + b + c, each in the upper half of its word: 2 a its
// first 8 bits, b the next 8, c the rest, so nothing is lost (but below 2^-102, where c runs out
// of exponents). Each is cut off below the value, not at it, so that none is zero unless h is: a
// zero term times an infinite weight would make a NaN of an infinity. All have h's sign. Of an
// infinity c is one, of a NaN all three are.
__device__ __forceinline__ void three_terms(float h, unsigned &a, unsigned &b, unsigned &c)
{
    const float first = eight_bits_below(h), rest = h - first, second = eight_bits_below(rest);
    a = __float_as_uint(first * 0.5f);
    b = __float_as_uint(second);
    c = __float_as_uint(rest - second);
}

// Four values' terms, four 16-bit words each.
__device__ __forceinline__ void three_terms(const u32x4 &h, u32x2 (&term)[3])
{
    unsigned t[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        three_terms(__uint_as_float(h[i]), t[0][i], t[1][i], t[2][i]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        term[k] = u32x2{__builtin_amdgcn_perm(t[k][1], t[k][0], 0x07060302u),
                        __builtin_amdgcn_perm(t[k][3], t[k][2], 0x07060302u)};
}

// acc[i][g] += 16 rows of W (tile i) times the columns of group g, over k = first, first +
// stride, ... (a step is 64 k; k at and past K count as zeros). All in bytes:
//   w[i]      resource of tile i: its rows that exist, row_bytes apart (others read zeros)
//   x, col    resource of the columns, and where the lane's part of them starts in it:
//     16-bit  16 columns a group, two loads: column 8 i + lane / 8, at its octet lane % 8, in col[i]
//     WIDE    8 columns of fp32 a group, two loads: column 4 i + lane / 16, at its four lane % 16.
//             They become three bf16 terms here. Two instructions take them: column j of acc
//             adds a twice, column j + 8 b and c (sums of 16 and 24 bits, so products with
//             one weight are exact); the caller joins the two
// stage: kStage<RT, G, WIDE> chunks of shared memory of the wave's own; the wave needs no barrier.
// SHARE > 1 (WIDE): that many waves, all of the workgroup, call it together with the same columns
// and k. Each loads and cuts up its part of them, 4 columns at a time in turn (load `wave` + i SHARE
// of them in col[i]), into terms (two sets of set_chunks); there is one barrier a step. stage is then for rows alone, RT * 128 chunks.
// (Down product of 7168 x 2048, 8 of 64 experts, each wave for itself and shared: 128 tokens, four
// waves a CU, 635 and 526 us, 465 with four steps in flight; 64 tokens, eight waves, 324 and 312.
// With one group a step the barrier costs more: 2048 x 1408, 32 tokens, 87 and 103.)
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
template <int DT, int RT, int G, bool WIDE, int SHARE = 1>
__device__ __forceinline__ void stream_products(f32x4 (&acc)[RT][G], const rsrc_t (&w)[RT], uint32_t row_bytes,
                                                rsrc_t x, const uint32_t (&col)[kOwnLoads<G, SHARE>], int K, int first,
                                                int stride, u32x4 *stage, u32x4 *terms = nullptr, int set_chunks = 0)
{
    static_assert(WIDE || SHARE == 1, "");
    constexpr int kLoads = kOwnLoads<G, SHARE>;
    struct Buf {
        u32x4 w[RT][2], x[kLoads];
    };
    const int lane = lane_id();
    const int row = lane / 8, chunk = lane % 8;
    const uint32_t row0 = row * row_bytes + chunk * 16, row1 = row0 + 8 * row_bytes;
    const int kw = chunk * 8, kx = WIDE ? lane % 16 * 4 : kw;
    auto fetch = [&](Buf &buf, int k) {
        const bool in = k < K - kw, inx = k < K - kx;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            buf.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(w[i], in ? row0 : kNowhere, k * 2, kLoadAux);
            buf.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(w[i], in ? row1 : kNowhere, k * 2, kLoadAux);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            buf.x[i] = __builtin_amdgcn_raw_buffer_load_b128(x, inx ? col[i] : kNowhere, k * (WIDE ? 4 : 2), 0);
    };
    // chunk c of a row lies at c ^ (row % 8), so that eight lanes that read one chunk of eight
    // rows, or write a row, fall into different banks
    u32x4 *const xs = stage + RT * 128;
    const int put_w = row * 8 + (chunk ^ row);
    const int i16 = lane % 16, q = lane / 16;
    int get[2], get_next[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        get[h] = i16 * 8 + ((4 * h + q) ^ i16 % 8);
        get_next[h] = get[h] + (i16 < 8 ? 0 : 64);  // WIDE: a again, or c
    }
    // WIDE, in half chunks: a term of eight columns takes the place of eight rows
    const int put_x0 = q * 16 + (i16 / 2 ^ q) * 2 + lane % 2, put_x1 = (4 + q) * 16 + (i16 / 2 ^ (4 + q)) * 2 + lane % 2;
    const int wave = SHARE > 1 ? wave_in_block() : 0;
    auto multiply = [&](const Buf &buf, int set) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            stage[i * 128 + put_w] = buf.w[i][0];
            stage[i * 128 + 64 + put_w] = buf.w[i][1];
        }
        if constexpr (SHARE > 1) {
            u32x4 *const now = terms + set * set_chunks;
            u32x2 *const halves = reinterpret_cast<u32x2 *>(now);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int load = wave + i * SHARE;  // of 2 G: four columns each
                if (load >= 2 * G)
                    break;
                u32x2 t[3];
                three_terms(buf.x[i], t);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    halves[load / 2 * (2 * kTerms) + k * 128 + (load % 2 ? put_x1 : put_x0)] = t[k];
            }
            // Everyone's terms of this step are there. Those of the next go into the other set, and
            // into this one again only after the next barrier, which a wave reaches when its reads
            // below have come. Loads from memory go on.
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_sched_barrier(0);
            u32x4 a[RT][2];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    a[i][h] = stage[i * 128 + get[h]];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 b = now[g * kTerms + get[h]], c = now[g * kTerms + get_next[h]];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        acc[i][g] = mfma16<DT>(a[i][h], b, acc[i][g]);
                        acc[i][g] = mfma16<DT>(a[i][h], c, acc[i][g]);
                    }
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            return;
        }
        if constexpr (!WIDE) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                xs[g * 128 + put_w] = buf.x[2 * g];
                xs[g * 128 + 64 + put_w] = buf.x[2 * g + 1];
            }
        }
        // the lanes of a wave run together and its accesses to shared memory stay in order;
        // the fence keeps the compiler from moving them across
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if constexpr (WIDE) {
            u32x4 a[RT][2];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    a[i][h] = stage[i * 128 + get[h]];
            // a group's products are made when the next one's reads are on their way
            u32x2 *const halves = reinterpret_cast<u32x2 *>(xs);
            u32x4 b[2][2][2];
            auto products = [&](int g) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < RT; ++i)
                            acc[i][g] = mfma16<DT>(a[i][h], b[g % 2][h][k], acc[i][g]);
            };
#pragma unroll
            for (int g = 0; g < G; ++g) {
                u32x2 t0[3], t1[3];
                three_terms(buf.x[2 * g], t0);
                three_terms(buf.x[2 * g + 1], t1);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    halves[k * 128 + put_x0] = t0[k];
                    halves[k * 128 + put_x1] = t1[k];
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    b[g % 2][h][0] = xs[get[h]];
                    b[g % 2][h][1] = xs[get_next[h]];
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (g > 0)
                    products(g - 1);
            }
            products(G - 1);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 b[G];
#pragma unroll
                for (int g = 0; g < G; ++g)
                    b[g] = xs[g * 128 + get[h]];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const u32x4 a = stage[i * 128 + get[h]];
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        acc[i][g] = mfma16<DT>(a, b[g], acc[i][g]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    };
    // steps of loads in flight: four where four waves have the CU to themselves
    constexpr int DEPTH = SHARE == 4 ? 4 : 2;
    Buf buf[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        fetch(buf[d], first + d * stride);
    for (int k = first; k < K;) {  // whole turns of an even depth, so calls use the sets in turn too
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            multiply(buf[d], d % 2);
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
