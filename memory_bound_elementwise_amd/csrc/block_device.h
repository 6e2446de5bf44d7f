// Device helpers shared by the kernels of libmoe_block.so.
#ifndef MBE_BLOCK_DEVICE_H
#define MBE_BLOCK_DEVICE_H

#include "cdna4_stream.h"

namespace block {

using namespace cdna4;

enum : int { DT_BF16 = 0, DT_F16 = 1, DT_F32 = 2 };

template <int DT>
constexpr int kSize = DT == DT_F32 ? 4 : 2;

// 16 bytes at an address aligned to one element: rows of odd width start anywhere. The
// global memory path takes any alignment; only a row's last few elements go one by one.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

template <int DT>
__device__ __forceinline__ float load1(const void *base, int64_t i)
{
    if constexpr (DT == DT_F32)
        return static_cast<const float *>(base)[i];
    const uint16_t w = static_cast<const uint16_t *>(base)[i];
    if constexpr (DT == DT_BF16)
        return __uint_as_float((unsigned)w << 16);
    return (float)__builtin_bit_cast(_Float16, w);
}

template <int DT>
__device__ __forceinline__ void store1(void *base, int64_t i, float v)
{
    if constexpr (DT == DT_F32)
        static_cast<float *>(base)[i] = v;
    else if constexpr (DT == DT_BF16)
        static_cast<uint16_t *>(base)[i] = (uint16_t)pack_bf16x2(v, v);
    else
        static_cast<uint16_t *>(base)[i] = __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Eight elements as they lie in memory (one 16-byte vector for 16-bit types, two for fp32).
template <int DT>
struct Raw8 {
    u32x4 v[kSize<DT> / 2];
};

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT> &o, float (&f)[8])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (DT == DT_BF16) {
            f[2 * q] = bf16_lo(o.v[0][q]);
            f[2 * q + 1] = bf16_hi(o.v[0][q]);
        } else if constexpr (DT == DT_F16) {
            const f32x2 t = unpack_f16x2(o.v[0][q]);
            f[2 * q] = t.x;
            f[2 * q + 1] = t.y;
        } else {
            f[q] = __uint_as_float(o.v[0][q]);
            f[4 + q] = __uint_as_float(o.v[1][q]);
        }
    }
}

template <int DT>
__device__ __forceinline__ Raw8<DT> narrow8(const float (&f)[8])
{
    Raw8<DT> o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (DT == DT_BF16) {
            o.v[0][q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
        } else if constexpr (DT == DT_F16) {
            o.v[0][q] = pack_f16x2(f[2 * q], f[2 * q + 1]);
        } else {
            o.v[0][q] = __float_as_uint(f[q]);
            o.v[1][q] = __float_as_uint(f[4 + q]);
        }
    }
    return o;
}

// Elements j .. j+7 of a row of n (j a multiple of 8), zeros past its end.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const char *row, int j, int n)
{
    Raw8<DT> o;
    const char *p = row + (int64_t)j * kSize<DT>;
    if (j + 8 <= n) {
#pragma unroll
        for (int i = 0; i < kSize<DT> / 2; ++i)
            o.v[i] = reinterpret_cast<const u32x4_any *>(p)[i];
        return o;
    }
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = j + i < n ? load1<DT>(p, i) : 0.0f;
    return narrow8<DT>(f);  // a value of DT, so exact
}

template <int DT>
__device__ __forceinline__ void store8(char *row, int j, int n, const float (&f)[8])
{
    char *p = row + (int64_t)j * kSize<DT>;
    if (j + 8 <= n) {
        const Raw8<DT> o = narrow8<DT>(f);
#pragma unroll
        for (int i = 0; i < kSize<DT> / 2; ++i)
            reinterpret_cast<u32x4_any *>(p)[i] = o.v[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (j + i < n)
            store1<DT>(p, i, f[i]);
}

// The row accesses of a kernel: EVEN (rows of a multiple of eight elements, so 16-byte
// aligned) through a buffer resource of the row, whose range check masks its end and rows
// that are not there without a branch; otherwise one element at a time where a group of eight
// is cut off. Loads stay cached (what was just written is read: 31 us against 34 for the
// forward pass over 6720 x 7168 bf16), stores go past the caches.
template <int DT, bool EVEN>
struct Row {
    rsrc_t rsrc;
    char *p;
    int n;
    __device__ __forceinline__ Row(const void *base, int64_t row, int cols, bool live)
        : p(const_cast<char *>(static_cast<const char *>(base)) + (live ? row * cols * kSize<DT> : 0)), n(live ? cols : 0)
    {
        if constexpr (EVEN)
            rsrc = make_rsrc(p, (uint32_t)n * kSize<DT>);
    }
    __device__ __forceinline__ Raw8<DT> load(int j) const
    {
        if constexpr (EVEN) {
            Raw8<DT> o;
#pragma unroll
            for (int i = 0; i < kSize<DT> / 2; ++i)
                o.v[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (uint32_t)j * kSize<DT> + 16u * i, 0, 0);
            return o;
        }
        return load8<DT>(p, j, n);
    }
    // One fp32 value (rows of DT_F32).
    __device__ __forceinline__ float load1(int j) const
    {
        static_assert(DT == DT_F32 && EVEN, "");
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, (uint32_t)j * 4u, 0, 0));
    }
    __device__ __forceinline__ void store(int j, const float (&f)[8]) const
    {
        if constexpr (EVEN) {
            const Raw8<DT> o = narrow8<DT>(f);
#pragma unroll
            for (int i = 0; i < kSize<DT> / 2; ++i)
                store_vec(rsrc, o.v[i], (uint32_t)j * kSize<DT> + 16u * i);
            return;
        }
        store8<DT>(p, j, n, f);
    }
};

}  // namespace block

#endif  // MBE_BLOCK_DEVICE_H
