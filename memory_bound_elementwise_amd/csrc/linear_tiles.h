// What the products with an epilogue share: their arguments, the epilogue, the kernel that adds the
// parts of a split sum, and the wait of the kernels that load straight into shared memory.
#ifndef MBE_LINEAR_TILES_H
#define MBE_LINEAR_TILES_H

#include "block_math.h"

namespace block {

struct LinearArgs {
    const uint16_t *x, *w, *bias, *residual;
    uint16_t *y;
    int m, n, k, act;
};

template <int DT>
__device__ __forceinline__ void finish(const LinearArgs &a, int row, int col, float z)
{
    if (a.bias)
        z += load1<DT>(a.bias, col);
    z = activate(a.act, z);
    const int64_t at = (int64_t)row * a.n + col;
    if (a.residual)
        z += load1<DT>(a.residual, at);
    store1<DT>(a.y, at, z);
}

// Eight neighbouring columns at once (col and n multiples of 8), with the bias and the residual
// there.
template <int DT>
__device__ __forceinline__ void finish8(const LinearArgs &a, int row, int col, float (&z)[8], const Raw8<DT> &bias,
                                        const Raw8<DT> &residual)
{
    float f[8];
    if (a.bias) {
        widen8<DT>(bias, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += f[i];
    }
    activate8(a.act, z);
    if (a.residual) {
        widen8<DT>(residual, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += f[i];
    }
    // past the caches, which the operands need (6720 x 7168 x 4096: 357 us against 377)
    __builtin_nontemporal_store(narrow8<DT>(z).v[0], reinterpret_cast<u32x4 *>(a.y + (int64_t)row * a.n + col));
}

typedef __attribute__((address_space(3))) void shared_void;

// Waits for the wave's loads into shared memory and its reads of it, then for the workgroup.
// (Loads into shared memory count as loads from memory: a fence need not wait for them.)
// Nothing is moved across.
__device__ __forceinline__ void wait_and_sync()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
}

// The parts' sums in order, then the epilogue. A lane takes eight neighbouring columns.
template <int DT>
static __global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a, int parts, const float *partial)
{
    const int64_t all = (int64_t)a.m * a.n;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < all; i += (int64_t)gridDim.x * 2048) {
        float z[8] = {};
        for (int p = 0; p < parts; p += 2) {  // a power of two, at least 2; two loads at a time
            float f0[8], f1[8];
            widen8<DT_F32>(load8<DT_F32>(reinterpret_cast<const char *>(partial + p * all + i), 0, 8), f0);
            widen8<DT_F32>(load8<DT_F32>(reinterpret_cast<const char *>(partial + (p + 1) * all + i), 0, 8), f1);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = z[e] + f0[e] + f1[e];
        }
        const int row = (int)(i / a.n), col = (int)(i % a.n);
        Raw8<DT> bias, residual;
        if (a.bias)
            bias = load8<DT>(reinterpret_cast<const char *>(a.bias), col, a.n);
        if (a.residual)
            residual = load8<DT>(reinterpret_cast<const char *>(a.residual + i), 0, 8);
        finish8<DT>(a, row, col, z, bias, residual);
    }
}

}  // namespace block

#endif  // MBE_LINEAR_TILES_H
