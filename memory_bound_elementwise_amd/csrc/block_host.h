// Host side shared by the entry points of libmoe_block.so: status reporting, argument
// checks and kernel launches. Nothing here throws or allocates.
#ifndef MBE_BLOCK_HOST_H
#define MBE_BLOCK_HOST_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block/moe_block.h"

namespace block {

// Records the HIP error for moe_block_last_hip_error (defined in block_common.hip).
block_status_t fail_hip(hipError_t e);

inline bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// One tensor of a call: its address and byte count (0 bytes, or a null pointer: absent).
struct Span {
    const void *p;
    int64_t bytes;
};

inline bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Whether any of the written spans overlaps another written one or a read one.
template <int W, int R>
bool any_overlap(const Span (&written)[W], const Span (&read)[R])
{
    for (int i = 0; i < W; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j]))
                return true;
        for (int j = 0; j < R; ++j)
            if (overlap(written[i], read[j]))
                return true;
    }
    return false;
}

// hipLaunchKernel reports its own error; the sticky last error, which may be an earlier
// call's, is neither read nor cleared.
template <typename... P, typename... A>
block_status_t launch(void (*kernel)(P...), dim3 grid, dim3 threads, uint32_t lds, hipStream_t stream, A... args)
{
    static_assert(sizeof...(P) == sizeof...(A), "argument count");
    return [&](P... exact) {
        void *ptrs[] = {static_cast<void *>(&exact)...};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, threads, ptrs, lds, stream);
        return e == hipSuccess ? BLOCK_OK : fail_hip(e);
    }(static_cast<P>(args)...);
}

// The most workgroups of so many threads: a dispatch counts its work-items in 32 bits.
constexpr int64_t max_groups(int threads) { return 0xffffffffu / (unsigned)threads; }

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace block

#endif  // MBE_BLOCK_HOST_H
