// angle.cuh -- the angle of a rotation in half turns, for the kernels and (compiled as plain C++) for the host.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define CSA2_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CSA2_HOST_DEVICE inline
#endif

namespace csa2 {

// pos * f radians in half turns, reduced to [-1, 1], off by 2^-52 at most for any 0 <= pos * f < 2^32.
// A product in 64 bits alone is off by 2^-53 of the whole angle, 2^-22 radians at a position near 2^31, so the
// rounding errors of both products and the part of 1/pi below 64 bits are carried along:
//   pos f = a + b,  a / pi = h + (its error) + a (1/pi's rest),  and h - 2 rint(h / 2) is exact.
CSA2_HOST_DEVICE double half_turns(int64_t pos, double f) {
    constexpr double kInvPi = 0.31830988618379067154, kInvPiRest = -1.9678676675182486e-17;
    const double p = (double)pos, a = p * f, b = fma(p, f, -a);
    const double h = a * kInvPi, rest = fma(a, kInvPi, -h) + fma(a, kInvPiRest, b * kInvPi);
    return (h - 2.0 * rint(0.5 * h)) + rest;
}

}  // namespace csa2
