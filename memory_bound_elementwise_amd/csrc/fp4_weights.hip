// Weights to 4 bits with group scales and back, for AMD Instinct MI355X (gfx950). C ABI declared
// in block/moe_block.h, layout in fp4.h. One wave a tile of 16 rows x 128 k. Bound by memory: 8 x
// 4096 x 7168 fp32 to 4 bits 180 us (1.06 GB, 5.9 TB/s), from 4 bits to bf16 97 (0.6 GB, 6.1). Packing
// the same, 250 MB, takes 114 (2.2 TB/s).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp4.h"
#include "fp4_host.h"

namespace {

using namespace block;

constexpr int kTilesHere = 4;  // waves of a workgroup

struct Args {
    const char *from;            // quantize: weights; pack: elements; dequantize: codes
    const uint8_t *from_scales;  // pack: exponents; dequantize: scales
    char *to;
    uint8_t *to_scales;
    int n, k, row_tiles, k_tiles, tiles;
};

// The wave's tile: rows row0 .. row0 + rows - 1 of all matrices together (the tile's further rows lie
// past its matrix's end) from k0 on.
struct Place {
    int64_t tile, row0;
    int rows, k0;
};

__device__ __forceinline__ bool place(const Args &a, Place &p)
{
    const uint32_t tile = blockIdx.x * kTilesHere + wave_in_block();
    if (tile >= (uint32_t)a.tiles)
        return false;
    const uint32_t block = tile / (uint32_t)a.k_tiles, matrix = block / (uint32_t)a.row_tiles;
    const int row = (int)(block - matrix * a.row_tiles) * kFp4Rows;
    p.tile = tile;
    p.k0 = (int)(tile - block * a.k_tiles) * kFp4K;
    p.rows = a.n - row < kFp4Rows ? a.n - row : kFp4Rows;
    p.row0 = (int64_t)matrix * a.n + row;
    return true;
}

// The byte of a group's power of two from the bits of its largest magnitude: the smallest power with
// magnitude < 7 2^power, so that 6, the largest element, is the nearest one to all of the group. (The
// format's own recipe takes the largest power up to the magnitude over 4, and cuts what is then past 6
// off at 6; groups whose largest is from 7 to 8 of those powers get twice the power here.) A group of
// zeros gets 127; one with an infinity or a NaN 255, which makes it all NaN. 252 at most, so that no
// value passes bf16's range (the largest weights become 6 2^125 then).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const int power = (int)((top + 0x200000u) >> 23) - 2;  // carries where the mantissa reaches 1.75
    const uint32_t byte = power < 0 ? 0 : (power > 252 ? 252 : power);
    return top >= 0x7f800000u ? 255u : (top == 0 ? 127u : byte);
}

template <int kCtrl>
__device__ __forceinline__ uint32_t larger_dpp(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
    return o > v ? o : v;
}

// Rows are read as they lie, 16 bytes a lane, a row's 128 k by 16 or (fp32) 32 neighbouring lanes, so
// that a group's largest magnitude is found among four or eight of them; the codes get into
// their tile's order on the way through shared memory. (With the tile's order in the loads, 16 rows
// an instruction: 8 x 4096 x 7168 fp32 242 us.)
template <int DT>
__global__ __launch_bounds__(kTilesHere * 64) void fp4_quantize_kernel(Args a)
{
    constexpr int kEach = 16 / kSize<DT>, kLanes = kFp4K / kEach, kTogether = 64 / kLanes, kLoads = kFp4Rows / kTogether;
    __shared__ u32x4 codes[kTilesHere][64];
    __shared__ uint32_t scales[kTilesHere][kFp4Rows];
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), wave = wave_in_block(), row = lane / kLanes, k = lane % kLanes * kEach;
    // the tile's rows to the last one's end: a load past it, or past a row's end, reads zeros
    const uint32_t row_bytes = (uint32_t)a.k * kSize<DT>;
    const rsrc_t from = make_rsrc(a.from + (p.row0 * a.k + p.k0) * kSize<DT>,
                                  (uint32_t)p.rows * row_bytes - (uint32_t)p.k0 * kSize<DT>);
    u32x4 raw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        raw[i] = __builtin_amdgcn_raw_buffer_load_b128(
            from, p.k0 + k < a.k ? (uint32_t)(i * kTogether + row) * row_bytes + k * kSize<DT> : 0x80000000u, 0, kLoadAux);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        float f[kEach];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (DT == DT_F32) {
                f[q] = __uint_as_float(raw[i][q]);
            } else if constexpr (DT == DT_BF16) {
                f[2 * q] = bf16_lo(raw[i][q]);
                f[2 * q + 1] = bf16_hi(raw[i][q]);
            } else {
                const f32x2 t = unpack_f16x2(raw[i][q]);
                f[2 * q] = t.x;
                f[2 * q + 1] = t.y;
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const uint32_t m = __float_as_uint(f[e]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        top = larger_dpp<0xB1>(top);
        top = larger_dpp<0x4E>(top);
        if constexpr (DT == DT_F32)
            top = larger_dpp<0x141>(top);
        const uint32_t byte = scale_byte(top);
        const float scale = __uint_as_float(byte << 23);
        const int r = i * kTogether + row;
        // word j of lane 16 q + r holds k = 32 j + 8 q ..+8
        char *to = reinterpret_cast<char *>(&codes[wave][k % 32 / 8 * 16 + r]) + k / 32 * 4;
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
        if constexpr (DT == DT_F32) {
            reinterpret_cast<uint16_t *>(to)[k % 8 / 4] = (uint16_t)c;
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
            *reinterpret_cast<uint32_t *>(to) = c;
        }
        if (k % 32 == 0)
            reinterpret_cast<uint8_t *>(&scales[wave][r])[k / 32] = (uint8_t)byte;
        __builtin_amdgcn_sched_barrier(0);
    }
    // the wave's accesses to shared memory stay in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_nontemporal_store(codes[wave][lane], reinterpret_cast<u32x4 *>(a.to + p.tile * kFp4Codes) + lane);
    if (lane < kFp4Rows)
        reinterpret_cast<uint32_t *>(a.to_scales + p.tile * kFp4Scales)[lane] = scales[wave][lane];
}

// In the tile's order, 16 bytes of each of 16 rows an instruction, and the exponents byte by byte: a layer's
// weights are packed once.
__global__ __launch_bounds__(kTilesHere * 64) void fp4_pack_kernel(Args a)
{
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), q = lane / 16, r = lane % 16;
    const bool there = r < p.rows;
    const char *row = a.from + (p.row0 + (there ? r : 0)) * (a.k / 2);
    const uint8_t *exponents = a.from_scales + (p.row0 + (there ? r : 0)) * (a.k / kFp4Group);
    u32x4 codes;
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = p.k0 + 32 * j;
        const bool in = there && k < a.k;
        codes[j] = in ? *reinterpret_cast<const uint32_t *>(row + (k + 8 * q) / 2) : 0;
        bytes |= (uint32_t)(in ? exponents[k / kFp4Group] : 127) << (8 * j);
    }
    reinterpret_cast<u32x4 *>(a.to + p.tile * kFp4Codes)[lane] = codes;
    if (q == 0)
        reinterpret_cast<uint32_t *>(a.to_scales + p.tile * kFp4Scales)[lane] = bytes;
}

// The values go through shared memory too, so that 16 neighbouring lanes write a row's 256 bytes. Chunk
// c of row r lies at c ^ (r % 8): eight lanes that write one chunk of eight rows, or read a
// row, fall into different banks. (Straight from the tile's order, 64 bytes a row: 113 us for 8 x
// 4096 x 7168.)
__global__ __launch_bounds__(kTilesHere * 64) void fp4_dequantize_kernel(Args a)
{
    __shared__ u32x4 shared[kTilesHere][256];
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    u32x4 *values = shared[wave_in_block()];
    const u32x4 codes = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.from + p.tile * kFp4Codes) + lane);
    const uint32_t bytes = reinterpret_cast<const uint32_t *>(a.from_scales + p.tile * kFp4Scales)[i16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        values[i16 * 16 + ((4 * j + q) ^ i16 % 8)] = fp4_widen(codes[j], fp4_scale(bytes, j));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int k = p.k0 + i16 * 8;
    char *to = a.to + ((p.row0 + q) * a.k + k) * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + q;
        if (r < p.rows && k < a.k)
            __builtin_nontemporal_store(values[r * 16 + (i16 ^ r % 8)], reinterpret_cast<u32x4 *>(to + (int64_t)i * 8 * a.k));
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
block_status_t run(void (*kernel)(Args), const void *from, const void *from_scales, void *to, void *to_scales,
                   const Fp4Shape &s, hipStream_t st)
{
    const Args a = {static_cast<const char *>(from), static_cast<const uint8_t *>(from_scales), static_cast<char *>(to),
                    static_cast<uint8_t *>(to_scales), (int)s.n, (int)s.k, (int)s.row_tiles(), (int)s.k_tiles(),
                    (int)s.tiles()};
    return launch(kernel, dim3((unsigned)ceil_div(s.tiles(), kTilesHere)), dim3(kTilesHere * 64), 0, st, a);
}

// The checks that all three share; `plain` is the row-major side, of so many bytes. Null spans
// are refused, so every tensor is there.
template <int W, int R>
block_status_t check(const Fp4Shape &s, const Span (&written)[W], const Span (&read)[R])
{
    for (const Span &t : written)
        if (!t.p)
            return BLOCK_ERR_INVALID_ARG;
    for (const Span &t : read)
        if (!t.p)
            return BLOCK_ERR_INVALID_ARG;
    for (const Span &t : written)
        if (misaligned(t.p, 16))
            return BLOCK_ERR_ALIGNMENT;
    for (const Span &t : read)
        if (misaligned(t.p, 16))
            return BLOCK_ERR_ALIGNMENT;
    return any_overlap<W, R>(written, read) ? BLOCK_ERR_INVALID_ARG : BLOCK_OK;
}

}  // namespace

extern "C" {

int64_t block_fp4_codes_bytes(int64_t n, int64_t k)
{
    const Fp4Shape s = {1, n, k};
    return s.good() && k % 32 == 0 ? s.codes() : 0;
}

int64_t block_fp4_scales_bytes(int64_t n, int64_t k)
{
    const Fp4Shape s = {1, n, k};
    return s.good() && k % 32 == 0 ? s.scales() : 0;
}

block_status_t block_fp4_quantize(const void *weight, block_dtype_t dtype, uint8_t *codes, uint8_t *scales,
                                  int64_t matrices, int64_t n, int64_t k, hipStream_t stream)
{
    const Fp4Shape s = {matrices, n, k};
    if (!s.good() || (dtype != BLOCK_BF16 && dtype != BLOCK_FP16 && dtype != BLOCK_FP32))
        return BLOCK_ERR_INVALID_ARG;
    if (k % 32)
        return BLOCK_ERR_ALIGNMENT;
    if (matrices == 0)
        return BLOCK_OK;
    if (const block_status_t r = check<2, 1>(s, {{codes, s.codes()}, {scales, s.scales()}},
                                             {{weight, matrices * n * k * (dtype == BLOCK_FP32 ? 4 : 2)}}))
        return r;
    auto *kernel = dtype == BLOCK_FP32 ? fp4_quantize_kernel<DT_F32>
                                       : (dtype == BLOCK_BF16 ? fp4_quantize_kernel<DT_BF16> : fp4_quantize_kernel<DT_F16>);
    return run(kernel, weight, nullptr, codes, scales, s, stream);
}

block_status_t block_fp4_pack(const uint8_t *elements, const uint8_t *exponents, uint8_t *codes, uint8_t *scales,
                              int64_t matrices, int64_t n, int64_t k, hipStream_t stream)
{
    const Fp4Shape s = {matrices, n, k};
    if (!s.good())
        return BLOCK_ERR_INVALID_ARG;
    if (k % 32)
        return BLOCK_ERR_ALIGNMENT;
    if (matrices == 0)
        return BLOCK_OK;
    if (const block_status_t r = check<2, 2>(s, {{codes, s.codes()}, {scales, s.scales()}},
                                             {{elements, matrices * n * k / 2}, {exponents, matrices * n * k / 32}}))
        return r;
    return run(fp4_pack_kernel, elements, exponents, codes, scales, s, stream);
}

block_status_t block_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, uint16_t *weight, int64_t matrices,
                                    int64_t n, int64_t k, hipStream_t stream)
{
    const Fp4Shape s = {matrices, n, k};
    if (!s.good())
        return BLOCK_ERR_INVALID_ARG;
    if (k % 32)
        return BLOCK_ERR_ALIGNMENT;
    if (matrices == 0)
        return BLOCK_OK;
    if (const block_status_t r = check<1, 2>(s, {{weight, matrices * n * k * 2}}, {{codes, s.codes()}, {scales, s.scales()}}))
        return r;
    return run(fp4_dequantize_kernel, codes, scales, weight, nullptr, s, stream);
}

}  // extern "C"
