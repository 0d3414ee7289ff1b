// Rotary positions, shared by the kernel that rotates tokens and the one that
// appends rotated keys.  A pair (a, b) of a head's dimensions at position p turns
// by the angle 2 pi t, t = p * turns[i]:
//   a' = f (a cos - b sin),  b' = f (b cos + a sin),
// pair i being the dimensions (i, i + dims / 2), or (2 i, 2 i + 1) where
// interleaved; dimensions from dims on stay as they are.
//
// t is taken in fp64 and only its fraction goes on: at position 10^6 and one
// radian a step, fp32 angles are off by 0.03.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dq {

struct Rope {
    const double* turns;  // [dims / 2] turns per position
    int32_t dims;
    int32_t interleaved;
    double factor;
};

__device__ __forceinline__ double turn_fraction(int32_t pos, double turn)
{
    const double t = (double)pos * turn;
    return t - rint(t);
}

// Sine and cosine of 2 pi t, |t| <= 1/2, within some 2^-52: the nearest quarter turn taken off, their
// Taylor series at |x| <= pi / 4 (the first term left out is below 2^-54 of 1).
__device__ __forceinline__ void sincos_turn(double t, double& s, double& c)
{
    const double q = rint(4.0 * t);
    const double x = fma(-0.25, q, t) * 6.283185307179586476925, z = x * x;
    double u = -1.0 / 1307674368000.0;  // 15!
    u = fma(u, z, 1.0 / 6227020800.0);
    u = fma(u, z, -1.0 / 39916800.0);
    u = fma(u, z, 1.0 / 362880.0);
    u = fma(u, z, -1.0 / 5040.0);
    u = fma(u, z, 1.0 / 120.0);
    u = fma(u, z, -1.0 / 6.0);
    u = fma(u * z, x, x);
    double v = 1.0 / 20922789888000.0;  // 16!
    v = fma(v, z, -1.0 / 87178291200.0);
    v = fma(v, z, 1.0 / 479001600.0);
    v = fma(v, z, -1.0 / 3628800.0);
    v = fma(v, z, 1.0 / 40320.0);
    v = fma(v, z, -1.0 / 720.0);
    v = fma(v, z, 1.0 / 24.0);
    v = fma(v, z, -0.5);
    v = fma(v, z, 1.0);
    const int k = (int)q;  // quarters, -2 .. 2
    s = k & 1 ? v : u;
    c = k & 1 ? u : v;
    if (k & 2) s = -s;
    if ((k + 1) & 2) c = -c;
}

}  // namespace dq
