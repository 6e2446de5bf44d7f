// Weights to 4 bits with group scales and back, for AMD Instinct MI355X (gfx950). C ABI declared
// in block/moe_block.h, layout in fp4.h. One wave a tile of 16 rows x 128 k.
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
    int n, k, row_tiles, k_tiles;
    int64_t tiles;
};

struct Place {
    int64_t tile, row;  // row of all matrices together
    int k;              // of the tile
    bool there;         // whether the lane's row exists
};

__device__ __forceinline__ bool place(const Args &a, Place &p)
{
    p.tile = (int64_t)blockIdx.x * kTilesHere + wave_in_block();
    if (p.tile >= a.tiles)
        return false;
    const int64_t block = p.tile / a.k_tiles, matrix = block / a.row_tiles;
    p.k = (int)(p.tile % a.k_tiles) * kFp4K;
    const int row = (int)(block % a.row_tiles) * kFp4Rows + lane_id() % 16;
    p.there = row < a.n;
    p.row = matrix * a.n + (p.there ? row : 0);
    return true;
}

// The byte of a group's power of two from the bits of its largest magnitude: the smallest power
// with magnitude < 7 2^power, so that 6, the largest element, is the nearest one to all of the
// group. A group of zeros gets 127; one with an infinity or a NaN 255, which makes it all NaN.
// 252 at most, so that no value passes bf16's range (the largest weights become 6 2^125 then).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    if (top >= 0x7f800000u)
        return 255;
    if (top == 0)
        return 127;
    const int power = (int)((top + 0x200000u) >> 23) - 2;  // carries where the mantissa reaches 1.75
    return power < 0 ? 0 : (power > 252 ? 252 : power);
}

template <int DT>
__global__ __launch_bounds__(kTilesHere * 64) void fp4_quantize_kernel(Args a)
{
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), q = lane / 16;
    const char *row = a.from + p.row * a.k * kSize<DT>;
    float f[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = p.k + 32 * j;
        widen8<DT>(load8<DT>(row, k + 8 * q, p.there && k < a.k ? a.k : 0), f[j]);
    }
    u32x4 codes;
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = __float_as_uint(f[j][i]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        uint32_t other = __shfl_xor(top, 16);
        top = other > top ? other : top;
        other = __shfl_xor(top, 32);
        top = other > top ? other : top;
        const uint32_t byte = scale_byte(top);
        const float scale = __uint_as_float(byte << 23);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[j][0], f[j][1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[j][2], f[j][3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[j][4], f[j][5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[j][6], f[j][7], scale, 3);
        codes[j] = c;
        bytes |= byte << (8 * j);
    }
    reinterpret_cast<u32x4 *>(a.to + p.tile * kFp4Codes)[lane] = codes;
    if (q == 0)
        reinterpret_cast<uint32_t *>(a.to_scales + p.tile * kFp4Scales)[lane] = bytes;
}

__global__ __launch_bounds__(kTilesHere * 64) void fp4_pack_kernel(Args a)
{
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), q = lane / 16;
    const char *row = a.from + p.row * (a.k / 2);
    const uint8_t *exponents = a.from_scales + p.row * (a.k / kFp4Group);
    u32x4 codes;
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = p.k + 32 * j;
        const bool in = p.there && k < a.k;
        codes[j] = in ? *reinterpret_cast<const uint32_t *>(row + (k + 8 * q) / 2) : 0;
        bytes |= (uint32_t)(in ? exponents[k / kFp4Group] : 127) << (8 * j);
    }
    reinterpret_cast<u32x4 *>(a.to + p.tile * kFp4Codes)[lane] = codes;
    if (q == 0)
        reinterpret_cast<uint32_t *>(a.to_scales + p.tile * kFp4Scales)[lane] = bytes;
}

__global__ __launch_bounds__(kTilesHere * 64) void fp4_dequantize_kernel(Args a)
{
    Place p;
    if (!place(a, p))
        return;
    const int lane = lane_id(), q = lane / 16;
    const u32x4 codes = reinterpret_cast<const u32x4 *>(a.from + p.tile * kFp4Codes)[lane];
    const uint32_t bytes = reinterpret_cast<const uint32_t *>(a.from_scales + p.tile * kFp4Scales)[lane % 16];
    char *row = a.to + p.row * a.k * 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = p.k + 32 * j;
        if (p.there && k < a.k)
            *reinterpret_cast<u32x4 *>(row + (k + 8 * q) * 2) = fp4_widen(codes[j], fp4_scale(bytes, j));
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
block_status_t run(void (*kernel)(Args), const void *from, const void *from_scales, void *to, void *to_scales,
                   const Fp4Shape &s, hipStream_t st)
{
    const Args a = {static_cast<const char *>(from), static_cast<const uint8_t *>(from_scales), static_cast<char *>(to),
                    static_cast<uint8_t *>(to_scales), (int)s.n, (int)s.k, (int)s.row_tiles(), (int)s.k_tiles(), s.tiles()};
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
