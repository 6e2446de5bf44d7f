// The layout of weights in 4 bits with group scales, and what the kernels that read and write it
// share (gfx950).
//
// Elements are of the open microscaling format: a sign, two bits of exponent, one of mantissa (0,
// 0.5, 1, 1.5, 2, 3, 4, 6); 32 neighbours of a row share a power of two 2^(byte - 127). A matrix
// [n, k] lies in tiles of 16 rows x 128 k, tiles of one block of rows one after the other along k:
//   codes   1024 bytes a tile: lane 16 q + r of a wave holds 16 of them, of row r; its 32-bit word
//           j the elements k = 32 j + 8 q + 0 .. 7 of the tile, the first in the lowest bits
//   scales  64 bytes a tile: byte 4 r + j is that of row r's elements k = 32 j .. 32 j + 31
// so that a word is a matrix instruction's operand of 32 k, converted in four instructions, and a
// wave reads a tile as 1024 neighbouring bytes. Rows and k past the matrix's end are zeros.
#ifndef MBE_FP4_H
#define MBE_FP4_H

#include "block_math.h"

namespace block {

constexpr int kFp4Rows = 16, kFp4K = 128, kFp4Group = 32;
constexpr int kFp4Codes = kFp4Rows * kFp4K / 2, kFp4Scales = kFp4Rows * kFp4K / kFp4Group;  // bytes a tile

// The scale of bits 0 .. 255 as the conversions take it: a float's bits, of which they read the
// exponent. (0 stands for 2^-127 there, 255 for NaN, as in the format.)
__device__ __forceinline__ float fp4_scale(uint32_t bytes, int j)
{
    return __uint_as_float(j == 0 ? bytes << 23 : (j == 3 ? bytes >> 1 : bytes << (23 - 8 * j)) & 0x7f800000u);
}

// Eight elements times their scale as bf16, exactly (beyond bf16's range: infinities).
__device__ __forceinline__ u32x4 fp4_widen(uint32_t codes, float scale)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3))};
}

}  // namespace block

#endif  // MBE_FP4_H
