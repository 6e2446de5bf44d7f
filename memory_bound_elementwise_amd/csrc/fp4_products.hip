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

// A wave's next tiles of RT row blocks, in flight.
template <int RT>
struct Ahead {
    u32x4 codes[RT];
    uint32_t scales[RT];
    __device__ __forceinline__ void load(const Tiles (&w)[RT], int t)
    {
        const int lane = lane_id();
#pragma unroll
        for (int i = 0; i < RT; ++i) {  // a tile past the last reads zeros
            codes[i] = __builtin_amdgcn_raw_buffer_load_b128(w[i].codes, lane * 16, t * kFp4Codes, kLoadAux);
            scales[i] = __builtin_amdgcn_raw_buffer_load_b32(w[i].scales, lane % 16 * 4, t * kFp4Scales, 0);
        }
    }
};

// A barrier that waits for the wave's accesses to shared memory, but not for its loads from memory.
// Nothing is moved across.
__device__ __forceinline__ void sync_shared()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
}

// The same over all k with the columns shared: W waves, each with rows of its own, walk k together. A
// wave loads its part of the columns' next 128 k (load i of wave w takes columns 4 (w + i W) ..+4 of
// them: col[i], the start of column lane / 16 of these plus 16 (lane % 16) bytes), and they meet in
// shared memory: xs, two sets of G * 256 chunks of 16 bytes, used in turn, so that one barrier a step
// is enough. Chunk c of column i lies at c ^ (i % 8), so that lanes that read one chunk of eight
// columns fall into different banks. even, odd: the first two steps' tiles, loaded by the caller.
// groups: those of the G that have columns.
template <int G, int W>
constexpr int kOwnLoads = (4 * G + W - 1) / W;

template <int RT, int G, int W>
__device__ __forceinline__ void walk_products(f32x4 (&acc)[RT][G], const Tiles (&w)[RT], Ahead<RT> &even, Ahead<RT> &odd,
                                              rsrc_t x, const uint32_t (&col)[kOwnLoads<G, W>], int K, int groups, u32x4 *xs)
{
    constexpr int kLoads = kOwnLoads<G, W>;
    struct Columns {
        u32x4 v[kLoads];
    };
    const int lane = lane_id(), wave = wave_in_block(), k_tiles = (K + kFp4K - 1) / kFp4K;
    const int i16 = lane % 16, q = lane / 16;
    auto fetch = [&](Columns &c, int t) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            c.v[i] = __builtin_amdgcn_raw_buffer_load_b128(x, t * kFp4K + i16 * 8 < K ? col[i] : kNowhere, t * kFp4K * 2, 0);
    };
    static_assert(W % 2 == 0, "the columns of a wave's loads have one c % 8");
    const int put = (4 * wave + q) * 16 + (i16 ^ (4 * wave + q) % 8);  // load i: 64 W i further
    const int get = i16 * 16 + (q ^ i16 % 8), get_odd = get ^ 4;       // word j: 8 (j / 2) further
    auto multiply = [&](const Ahead<RT> &tiles, const Columns &c, u32x4 *set) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (wave + i * W < 4 * groups)
                set[put + i * W * 64] = c.v[i];
        // Everyone's columns of this step are there after the barrier. Those of the next go into the
        // other set, and into this one again only after the next barrier, which a wave reaches when
        // its reads below have come.
        sync_shared();
        u32x4 b[2][G];  // the next word's columns are read beside a word's products
        auto read = [&](int j) __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (g == 0 || g < groups)
                    b[j % 2][g] = set[(j % 2 ? get_odd : get) + j / 2 * 8 + g * 256];
        };
        read(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < 3)
                read(j + 1);
            u32x4 a[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                a[i] = fp4_widen(tiles.codes[i][j], fp4_scale(tiles.scales[i], j));
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (g == 0 || g < groups)
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        acc[i][g] = mfma16<DT_BF16>(a[i], b[j % 2][g], acc[i][g]);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    Columns c_even, c_odd;
    fetch(c_even, 0);
    fetch(c_odd, 1);
    for (int t = 0; t < k_tiles; t += 2) {  // whole turns of two, so calls use the sets in turn too
        multiply(even, c_even, xs);
        even.load(w, t + 2);
        fetch(c_even, t + 2);
        multiply(odd, c_odd, xs + G * 256);
        odd.load(w, t + 3);
        fetch(c_odd, t + 3);
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
    __shared__ int counts[kMaxPairs / 64];
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k, e = own_expert(a, pairs);
    if (e < 0)
        return;
    const int n = expert_pairs<kWaves>(a, pairs, e, list, counts);
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

// Up products where experts have many tokens: a workgroup takes one expert and kManyWaves times two
// row tiles, which walk k together (walk_products), so that x is read once for all of them. A
// wave has gate and up of 16 columns of the activation, or 32 columns of one product.
constexpr int kManyWaves = 8;

template <int ACT, int G>
__device__ __forceinline__ void up_many_pass(const ExpertArgs &a, const Tiles (&w)[2], Ahead<2> &even, Ahead<2> &odd,
                                             int c0, const uint16_t *list, int n, u32x4 *xs)
{
    constexpr int W = kManyWaves, kLoads = kOwnLoads<G, W>;
    const int lane = lane_id(), wave = wave_in_block();
    const rsrc_t x = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.hidden * 2u);
    uint32_t col[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int s = 4 * (wave + i * W) + lane / 16;
        col[i] = s < n ? (uint32_t)(list[s] / a.top_k) * (uint32_t)a.hidden * 2u + lane % 16 * 16 : kNowhere;
    }
    f32x4 acc[2][G];
    clear(acc);
    walk_products<2, G, W>(acc, w, even, odd, x, col, a.hidden, (n + 15) / 16, xs);
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
    Tiles w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = tiles_of(a.up_codes, a.up_scales,
                        k_tiles == 0 ? 0 : (ACT == ACT_SWIGLU ? ((int64_t)e * 2 + i) * blocks : (int64_t)e * blocks + i) + c0 / 16,
                        k_tiles);
    Ahead<2> even, odd;  // on their way while the pairs are looked for
    even.load(w, 0);
    odd.load(w, 1);
    const int n = expert_pairs<kManyWaves>(a, pairs, e, list, counts);
    for (int p = 0; p < n; p += G * 16) {
        const int m = n - p < G * 16 ? n - p : G * 16;
        if (p > 0) {
            sync_shared();  // the columns lie elsewhere in xs now
            even.load(w, 0);
            odd.load(w, 1);
        }
        up_many_pass<ACT, G>(a, w, even, odd, c0, list + p, m, xs);
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
    __shared__ int counts[kMaxPairs / 64];
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k, e = own_expert(a, pairs);
    if (e < 0)
        return;
    const int n = expert_pairs<kWaves>(a, pairs, e, list, counts);
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

// Down products where experts have many tokens, as up: four waves of four row tiles (64 columns of the
// output) each.
constexpr int kDownWaves = 4, kDownTiles = 4;

template <int G>
__device__ __forceinline__ void down_many_pass(const ExpertArgs &a, const Tiles (&w)[kDownTiles], Ahead<kDownTiles> &even,
                                               Ahead<kDownTiles> &odd, int c0, const uint16_t *list, int n, u32x4 *xs)
{
    constexpr int RT = kDownTiles, W = kDownWaves, kLoads = kOwnLoads<G, W>;
    const int lane = lane_id(), wave = wave_in_block();
    const uint32_t pairs = (uint32_t)(a.tokens * a.top_k), row_bytes = (uint32_t)a.inter * 2u;
    const rsrc_t h = make_rsrc(a.h, 3u * pairs * row_bytes);
    uint32_t col[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = 4 * (wave + i * W) + lane / 16, c = at % 16, s = at / 16 * kPairs + c / 3;
        col[i] = c < 15 && s < n ? ((uint32_t)(c % 3) * pairs + list[s]) * row_bytes + lane % 16 * 16 : kNowhere;
    }
    f32x4 acc[RT][G];
    clear(acc);
    walk_products<RT, G, W>(acc, w, even, odd, h, col, a.inter, (n + kPairs - 1) / kPairs, xs);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int c = lane % 16, s = g * kPairs + c / 3;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            f32x4 z = acc[i][g];
#pragma unroll
            for (int r = 0; r < 4; ++r)  // row_shl: the second and the third term's lane
                z[r] = z[r] + dpp<0x101>(acc[i][g][r]) + dpp<0x102>(acc[i][g][r]);
            if (c < 15 && c % 3 == 0 && s < n && c0 + 16 * i < a.hidden)
                *reinterpret_cast<f32x4 *>(a.z + (int64_t)list[s] * a.hidden + c0 + 16 * i + lane / 16 * 4) = z;
        }
    }
}

template <int G>
__global__ __launch_bounds__(kDownWaves * 64, G == 4 ? 2 : 3) void fp4_down_many_kernel(ExpertArgs a)
{
    __shared__ u32x4 xs[2 * G * 256];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int counts[kMaxPairs / 64];
    const int pairs = live_tokens(a.valid, a.tokens) * a.top_k, e = own_expert(a, pairs);
    if (e < 0)
        return;
    const int blocks = a.hidden / 16, b0 = (blockIdx.x * kDownWaves + wave_in_block()) * kDownTiles;
    Tiles w[kDownTiles];
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i)  // past the last: no rows of W, but its part of h
        w[i] = tiles_of(a.down_codes, a.down_scales, b0 + i < blocks ? (int64_t)e * blocks + b0 + i : 0,
                        b0 + i < blocks ? (a.inter + kFp4K - 1) / kFp4K : 0);
    Ahead<kDownTiles> even, odd;
    even.load(w, 0);
    odd.load(w, 1);
    const int n = expert_pairs<kDownWaves>(a, pairs, e, list, counts);
    for (int p = 0; p < n; p += G * kPairs) {
        const int m = n - p < G * kPairs ? n - p : G * kPairs;
        if (p > 0) {
            sync_shared();
            even.load(w, 0);
            odd.load(w, 1);
        }
        down_many_pass<G>(a, w, even, odd, b0 * 16, list + p, m, xs);
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
    return each <= group ? 1 : (each <= 2 * group ? 2 : (each <= 3 * group ? 3 : 4));
}

// Whether the waves of a workgroup take rows of their own and share the columns: where that
// still leaves a workgroup for every CU.
bool shares_columns(int64_t rows_of_w, unsigned experts)
{
    return ceil_div(rows_of_w, kManyWaves * 32) * experts >= 256;
}

template <int ACT>
block_status_t launch_up(const ExpertArgs &a, int groups, unsigned each, hipStream_t st)
{
    constexpr int kCols = ACT == ACT_SWIGLU ? 16 : 32;
    if (shares_columns((int64_t)a.inter * 32 / kCols, each) && a.tokens > 1) {
        const dim3 grid((unsigned)ceil_div(a.inter, kManyWaves * kCols), each), threads(kManyWaves * 64);
        if (groups == 1)
            return launch(fp4_up_many_kernel<ACT, 1>, grid, threads, 0, st, a);
        if (groups == 2)
            return launch(fp4_up_many_kernel<ACT, 2>, grid, threads, 0, st, a);
        return launch(fp4_up_many_kernel<ACT, 4>, grid, threads, 0, st, a);
    }
    const dim3 grid((unsigned)(a.inter / 16), each), threads(kWaves * 64);
    if (groups == 1)
        return launch(fp4_up_kernel<ACT, 1>, grid, threads, 0, st, a);
    if (groups == 2)
        return launch(fp4_up_kernel<ACT, 2>, grid, threads, 0, st, a);
    return launch(fp4_up_kernel<ACT, 4>, grid, threads, 0, st, a);
}

block_status_t launch_down(const ExpertArgs &a, int groups, unsigned each, hipStream_t st)
{
    if (shares_columns(a.hidden, each) && a.tokens > 1) {
        const dim3 grid((unsigned)ceil_div(a.hidden, kDownWaves * kDownTiles * 16), each), threads(kDownWaves * 64);
        if (groups == 1)
            return launch(fp4_down_many_kernel<1>, grid, threads, 0, st, a);
        if (groups == 2)
            return launch(fp4_down_many_kernel<2>, grid, threads, 0, st, a);
        if (groups == 3)
            return launch(fp4_down_many_kernel<3>, grid, threads, 0, st, a);
        return launch(fp4_down_many_kernel<4>, grid, threads, 0, st, a);
    }
    const dim3 grid((unsigned)(a.hidden / 16), each), threads(kWaves * 64);
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
    const int groups = pair_groups(s, 16);
    if (const block_status_t r = act == BLOCK_ACT_SWIGLU ? launch_up<ACT_SWIGLU>(a, groups, each, stream)
                                                         : launch_up<ACT_SQUARED_RELU>(a, groups, each, stream))
        return r;
    if (const block_status_t r = launch_down(a, pair_groups(s, kPairs), each, stream))
        return r;
    const dim3 all((unsigned)ceil_div(n, 1024));
    return y_dtype == BLOCK_FP32 ? launch(fp4_combine_kernel<DT_F32>, all, dim3(256), 0, stream, a)
                                 : launch(fp4_combine_kernel<DT_BF16>, all, dim3(256), 0, stream, a);
}

}  // extern "C"
