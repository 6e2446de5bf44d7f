// The gate's exponential: plain arithmetic, which a host compiler takes as well.
#ifndef MBE_GATE_MATH_H
#define MBE_GATE_MATH_H

namespace block {

// e^v for v <= 0, within a step of fp64: v = n ln 2 + r with |r| <= ln 2 / 2, and the series of
// e^r to its 13th power (what follows is below 2^-57). ln 2 is taken off in two parts, the first of
// so few bits that n times it is exact, as in fdlibm's exp, whose two parts these are. Half of the
// library function's instructions, which has to deal with larger v.
__device__ __forceinline__ double exp_below(double v)
{
    v = v < -800.0 ? -800.0 : v;  // 0 from there on; keeps NaN
    const double n = __builtin_rint(__builtin_fmax(v, -800.0) * 1.4426950408889634);  // a number for NaN too
    const double r = __builtin_fma(n, -1.9082149292705877e-10, __builtin_fma(n, -0.6931471803691238, v));
    constexpr double c[] = {1.0 / 6227020800, 1.0 / 479001600, 1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320,
                            1.0 / 5040, 1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
    double e = c[0];
#pragma unroll
    for (int i = 1; i < 14; ++i)
        e = __builtin_fma(e, r, c[i]);
    return __builtin_ldexp(e, (int)n);
}

}  // namespace block

#endif  // MBE_GATE_MATH_H
