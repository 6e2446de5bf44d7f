// Activations and matrix-core types shared by the products of libmoe_block.so.
#ifndef MBE_BLOCK_MATH_H
#define MBE_BLOCK_MATH_H

#include "block_device.h"

namespace block {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Activation codes of the C ABI (block_act_t).
enum : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_SQUARED_RELU = 3, ACT_SWIGLU = 4 };

// D += A B^T over 32 k for a 16 x 16 tile. Lane l holds A[l % 16][8 (l / 16) ..+8] and
// B[l % 16][8 (l / 16) ..+8]; D[4 (l / 16) + r][l % 16] is element r of its result, A's row
// first. A column of D depends on its own row of B only. Products of two 16-bit values are
// exact in fp32 and the sums are fp32.
template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// z / (1 + e^-w): SiLU for w = z, the tanh form of GELU for w = 2 sqrt(2/pi) (z + 0.044715 z^3)
// (since (1 + tanh u) / 2 = 1 / (1 + e^-2u)). v_exp_f32 and v_rcp_f32 are good to about 1 ulp;
// far out e^-w is inf or 0 and the quotient 0 or z.
__device__ __forceinline__ float logistic_times(float z, float w)
{
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w * -1.4426950408889634f));
}

__device__ __forceinline__ float silu(float z) { return logistic_times(z, z); }

__device__ __forceinline__ float squared_relu(float z)
{
    const float a = __builtin_elementwise_maximum(z, 0.0f);  // keeps NaN
    return a * a;
}

__device__ __forceinline__ float activate(int act, float z)
{
    if (act == ACT_SILU)
        return silu(z);
    if (act == ACT_GELU)
        return logistic_times(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
    if (act == ACT_SQUARED_RELU)
        return squared_relu(z);
    return z;
}

// The same on eight values, decided once.
__device__ __forceinline__ void activate8(int act, float (&z)[8])
{
    if (act == ACT_SQUARED_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = squared_relu(z[i]);
    } else if (act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = silu(z[i]);
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = activate(ACT_GELU, z[i]);
    }
}

// silu(min(gate, L)) * clamp(up, -L, L); minimum and maximum keep NaN.
__device__ __forceinline__ float swiglu(float gate, float up, float limit)
{
    gate = __builtin_elementwise_minimum(gate, limit);
    up = __builtin_elementwise_maximum(__builtin_elementwise_minimum(up, limit), -limit);
    return silu(gate) * up;
}

}  // namespace block

#endif  // MBE_BLOCK_MATH_H
