// Rotary positions: what the rotation of rows and the rotated cache append share, the pair's arithmetic and the read of a
// table's entries.
//
// A pair (a, b) of channels turns by an angle given as (cos, sin):
//   a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))   in float32.
// Products and sums are rounded one by one, not fused: the result is then the same in whatever order a program
// computes it, and with it the 4-bit codes that the cache append makes of it.
#pragma once

#include "common.cuh"

namespace bsa {

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Eight table entries at 16-byte aligned p.
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

}  // namespace bsa
