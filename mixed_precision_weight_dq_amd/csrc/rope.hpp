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

__device__ __forceinline__ double rope_fraction(const Rope& r, int32_t pos, int i)
{
    const double t = (double)pos * r.turns[i];
    return t - rint(t);
}

}  // namespace dq
