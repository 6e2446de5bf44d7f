// Host side of the 4-bit weights: sizes of their layout (fp4.h).
#ifndef MBE_FP4_HOST_H
#define MBE_FP4_HOST_H

#include "block_host.h"

namespace block {

struct Fp4Shape {
    int64_t matrices, n, k;
    int64_t row_tiles() const { return ceil_div(n, 16); }
    int64_t k_tiles() const { return ceil_div(k, 128); }
    int64_t tiles() const { return matrices * row_tiles() * k_tiles(); }
    int64_t codes() const { return tiles() * 1024; }   // bytes
    int64_t scales() const { return tiles() * 64; }
    bool good() const
    {
        return matrices >= 0 && matrices <= (1 << 16) && n >= 1 && k >= 32 && n <= (1 << 20) && k <= (1 << 20) &&
               tiles() <= (1 << 25);
    }
};

}  // namespace block

#endif  // MBE_FP4_HOST_H
