// The inner loops of products with weights in 4 bits (layout in fp4.h) and a few columns: a wave reads
// tiles of 16 rows x 128 k in whole, straight into the registers from which the matrix
// instructions take them; the columns of x go through shared memory.
#ifndef MBE_FP4_STREAM_H
#define MBE_FP4_STREAM_H

#include <type_traits>

#include "fp4.h"

namespace block {

// Offset of a lane that reads nothing: past the end of every resource, so the load returns zeros
// (tensors of these products stay below 2^31 bytes a resource).
constexpr uint32_t kNowhere = 0x80000000u;

// One block of rows of a matrix for a wave: W's tiles, their scales and how many there are. A load's
// scalar offset is a tile's place, the lane's offset one in it. The range check is on the lane's offset
// against the resource's bytes less the scalar offset, so a tile past the last is read at the
// resource's very end: nothing is left there for any lane, and the load returns zeros.
struct Tiles {
    rsrc_t codes, scales;
    int own;
};

// there: whether the matrix has such a block (its tiles read zeros otherwise).
__device__ __forceinline__ Tiles tiles_of(const uint8_t *codes, const uint8_t *scales, int64_t block, int k_tiles,
                                          bool there = true)
{
    return {make_rsrc(codes + block * k_tiles * kFp4Codes, there ? (uint32_t)k_tiles * kFp4Codes : 0u),
            make_rsrc(scales + block * k_tiles * kFp4Scales, there ? (uint32_t)k_tiles * kFp4Scales : 0u), there ? k_tiles : 0};
}

// Neighbouring row blocks of one matrix over a range of its k tiles: all of their tiles from the first
// one's first to the last one's last, the distance of the blocks in tiles, the range's length and the
// number of blocks. (A resource a block would take four times the scalar registers.)
struct TileRun {
    Tiles all;
    int k_tiles, own, blocks;
};

// there: the blocks that are there, of those that are asked for; own: k tiles from `from` on.
__device__ __forceinline__ TileRun run_of(const uint8_t *codes, const uint8_t *scales, int64_t block, int k_tiles, int there,
                                          int from, int own)
{
    const int64_t tile = block * k_tiles + from;
    const int tiles = there ? (there - 1) * k_tiles + own : 0;
    return {{make_rsrc(codes + tile * kFp4Codes, (uint32_t)tiles * kFp4Codes),
             make_rsrc(scales + tile * kFp4Scales, (uint32_t)tiles * kFp4Scales), tiles},
            k_tiles, own, there};
}

// A wave's next tiles of RT row blocks, in flight. A tile past the last reads zeros.
template <int RT>
struct Ahead {
    u32x4 codes[RT];
    uint32_t scales[RT];
    template <int kAux>
    __device__ __forceinline__ void load(int i, const Tiles &w, int tile)
    {
        const int lane = lane_id();
        codes[i] = __builtin_amdgcn_raw_buffer_load_b128(w.codes, lane * 16, tile * kFp4Codes, kAux);
        scales[i] = __builtin_amdgcn_raw_buffer_load_b32(w.scales, lane % 16 * 4, tile * kFp4Scales, 0);
    }
    // kCached: of weights that other workgroups read too; past the caches otherwise.
    template <bool kCached = false>
    __device__ __forceinline__ void load(const Tiles (&w)[RT], int t)
    {
#pragma unroll
        for (int i = 0; i < RT; ++i)
            load<kCached ? 0 : kLoadAux>(i, w[i], t < w[i].own ? t : w[i].own);
    }
    __device__ __forceinline__ void load(const TileRun &w, int t)
    {
#pragma unroll
        for (int i = 0; i < RT; ++i)
            load<kLoadAux>(i, w.all, t < w.own && i < w.blocks ? i * w.k_tiles + t : w.all.own);
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

// The columns' chunks in shared memory: chunk c (16 bytes) of a column's 128 k lies at c ^ (column %
// 8), so that lanes that read one chunk of eight columns fall into different banks. A lane that
// loads chunk lane % 16 of column `of` puts it at put_at.
__device__ __forceinline__ int put_at(int of) { return of * 16 + (lane_id() % 16 ^ of % 8); }

// acc[i] += 16 rows of W (w[i]) times up to 4 NX columns, over the k tiles first, first + stride, ...,
// by one wave for itself. D steps of tiles and columns are in flight; start() sends the first
// tiles on their way, before the columns need be known. x: resource of the columns; col[i]:
// where column 4 i + lane / 16 starts in it, plus 16 (lane % 16) bytes, or kNowhere. stage: NX
// * 64 chunks of shared memory of the wave's own. (Each lane loading its own operand of x instead
// takes four loads a step, each to 16 lines.)
template <int RT, int NX, int D>
struct Stream {
    Ahead<RT> tiles[D];

    __device__ __forceinline__ void start(const Tiles (&w)[RT], int first, int stride)
    {
#pragma unroll
        for (int d = 0; d < D; ++d)
            tiles[d].load(w, first + d * stride);
    }

    __device__ __forceinline__ void run(f32x4 (&acc)[RT], const Tiles (&w)[RT], rsrc_t x, const uint32_t (&col)[NX],
                                        int K, int first, int stride, u32x4 *stage)
    {
        const int lane = lane_id(), i16 = lane % 16, q = lane / 16, k_tiles = (K + kFp4K - 1) / kFp4K;
        u32x4 buf[D][NX];
        auto fetch = [&](u32x4 (&to)[NX], int t) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                to[i] = __builtin_amdgcn_raw_buffer_load_b128(x, t * kFp4K + i16 * 8 < K ? col[i] : kNowhere, t * kFp4K * 2, 0);
        };
        const int c = i16 % (4 * NX);  // further columns repeat these and are not read
        const int get = c * 16 + (q ^ c % 8), get_odd = get ^ 4;  // word j: 8 (j / 2) further
        auto multiply = [&](const Ahead<RT> &now, const u32x4 (&from)[NX]) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                stage[put_at(4 * i + q)] = from[i];
            // the lanes of a wave run together and its accesses to shared memory stay in order;
            // the fence keeps the compiler from moving them across
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            u32x4 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = stage[(j % 2 ? get_odd : get) + j / 2 * 8];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    acc[i] = mfma16<DT_BF16>(fp4_widen(now.codes[i][j], fp4_scale(now.scales[i], j)), b[j], acc[i]);
        };
#pragma unroll
        for (int d = 0; d < D; ++d)
            fetch(buf[d], first + d * stride);
        for (int t = first; t < k_tiles;) {
#pragma unroll
            for (int d = 0; d < D; ++d) {  // past the last tile: zeros
                multiply(tiles[d], buf[d]);
                tiles[d].load(w, t + D * stride);
                fetch(buf[d], t + D * stride);
                t += stride;
            }
        }
    }
};

// acc[i][g] += 16 rows of W (w[i]) times 16 columns (group g) over K, with the columns shared: W
// waves, each with rows of its own, walk k together. A wave loads its part of the columns' next 128
// k (load i of wave w takes columns 4 (w + i W) ..+4 of them: col[i], the start of column lane / 16
// of these plus 16 (lane % 16) bytes), and they meet in shared memory: xs, two sets of G * 256
// chunks of 16 bytes, used in turn, so that one barrier a step is enough. D steps of tiles and two of
// columns, which come from cache, are in flight. W's blocks are a TileRun where CHAIN, and the walk
// ends by sending for the first steps of the next one.
template <int RT>
struct TileSet {
    Tiles block[RT];
};

template <int RT>
__device__ __forceinline__ void load_tiles(Ahead<RT> &to, const TileSet<RT> &w, int t) { to.load(w.block, t); }
template <int RT>
__device__ __forceinline__ void load_tiles(Ahead<RT> &to, const TileRun &w, int t) { to.load(w, t); }

template <int RT, int G, int W, int D, bool CHAIN>
struct Walk {
    static_assert(D % 2 == 0, "the sets of columns go on in turn");
    static constexpr int kLoads = (4 * G + W - 1) / W;  // a wave's loads of columns a step
    struct Ends {
        typename std::conditional<CHAIN, TileRun, TileSet<RT>>::type w;
        uint32_t col[kLoads];
        int K;
    };
    Ahead<RT> tiles[D];
    u32x4 columns[2][kLoads];

    __device__ __forceinline__ void start_tiles(const Ends &of)
    {
#pragma unroll
        for (int d = 0; d < D; ++d)
            load_tiles(tiles[d], of.w, d);
    }

    __device__ __forceinline__ void fetch(u32x4 (&to)[kLoads], rsrc_t x, const Ends &of, int t)
    {
        const int k = t * kFp4K + lane_id() % 16 * 8;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            to[i] = __builtin_amdgcn_raw_buffer_load_b128(x, k < of.K ? of.col[i] : kNowhere, t * kFp4K * 2, 0);
    }

    __device__ __forceinline__ void start_columns(rsrc_t x, const Ends &of)
    {
        fetch(columns[0], x, of, 0);
        fetch(columns[1], x, of, 1);
    }

    // groups: those of the G that have columns.
    __device__ __forceinline__ void run(f32x4 (&acc)[RT][G], rsrc_t x, const Ends &of, const Ends &next, int groups, u32x4 *xs)
    {
        static_assert(W % 2 == 0, "the columns of a wave's loads have one c % 8");
        const int lane = lane_id(), wave = wave_in_block(), k_tiles = (of.K + kFp4K - 1) / kFp4K;
        const int i16 = lane % 16, q = lane / 16;
        const int put = put_at(4 * wave + q);                         // load i: 64 W i further
        const int get = i16 * 16 + (q ^ i16 % 8), get_odd = get ^ 4;  // word j: 8 (j / 2) further
        auto multiply = [&](const Ahead<RT> &now, const u32x4 (&from)[kLoads], u32x4 *set) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (wave + i * W < 4 * groups)
                    set[put + i * W * 64] = from[i];
            // Everyone's columns of this step are there after the barrier. Those of the next go into the
            // other set, and into this one again only after the next barrier, which a wave reaches when
            // its reads below have come.
            sync_shared();
            // the next word's columns are read beside a word's products, where there are registers
            constexpr int kAhead = G < 3 ? 1 : 0;
            u32x4 b[kAhead + 1][G];
            auto read = [&](int j) __attribute__((always_inline)) {
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (g == 0 || g < groups)
                        b[j % (kAhead + 1)][g] = set[(j % 2 ? get_odd : get) + j / 2 * 8 + g * 256];
            };
            if (kAhead)
                read(0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j + kAhead < 4)
                    read(j + kAhead);
                u32x4 a[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    a[i] = fp4_widen(now.codes[i][j], fp4_scale(now.scales[i], j));
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (g == 0 || g < groups)
#pragma unroll
                        for (int i = 0; i < RT; ++i)
                            acc[i][g] = mfma16<DT_BF16>(a[i], b[j % (kAhead + 1)][g], acc[i][g]);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        };
        const auto once = [&](int d, const Ends &tile_of, int tile, const Ends &column_of, int column)
            __attribute__((always_inline)) {
            multiply(tiles[d], columns[d % 2], xs + d % 2 * G * 256);
            // loads come back in order: columns that are sent for behind later tiles would wait for those
            fetch(columns[d % 2], x, column_of, column);
            load_tiles(tiles[d], tile_of.w, tile);
        };
        int t = 0;
        for (; t + (CHAIN ? D : 0) < k_tiles; t += D) {  // whole turns of D; past the last tile: zeros
#pragma unroll
            for (int d = 0; d < D; ++d)
                once(d, of, t + d + D, of, t + d + 2);
        }
        if constexpr (CHAIN) {
#pragma unroll
            for (int d = 0; d < D; ++d)
                once(d, next, d, d < D - 2 ? of : next, d < D - 2 ? t + d + 2 : d + 2 - D);
        }
    }
};

}  // namespace block

#endif  // MBE_FP4_STREAM_H
