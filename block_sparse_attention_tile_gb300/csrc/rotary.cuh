// Rotary positions: what the rotation of rows and the rotated cache append share.
//
// A pair (a, b) of channels turns by an angle given as (cos, sin):
//   a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))   in float32.
// Products and sums are rounded one by one, not fused: the result is then the same in whatever order a program
// computes it, and with it the 4-bit codes that the cache append makes of it.
//
// A row of D channels is cut into units of 16: two runs of 8 channels that a lane reads with wide loads and
// whose pairs lie inside the unit.  Half layout: pair i is (i, i + P), unit u < P / 8 holds channels 8u .. and
// P + 8u ..; the rest of the row, 16 at a time, is copied.  Interleaved layout: pair i is (2i, 2i + 1), unit u
// holds channels 16u .. 16u + 15.  In both, unit u turns by the table's entries 8u .. 8u + 7.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace bsa {

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Eight channels at 16-byte aligned p.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                                              ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// First channels of a unit's two runs.
__device__ __forceinline__ void unit_runs(int u, int P, bool interleaved, int& c0, int& c1) {
    if (!interleaved && 8 * u < P) c0 = 8 * u, c1 = P + 8 * u;
    else c0 = interleaved ? 16 * u : 2 * P + 16 * (u - P / 8), c1 = c0 + 8;
}

// Turns a unit's 16 channels (x[0..7] the first run, x[8..15] the second).
__device__ __forceinline__ void rotate_unit(float* x, const float* c, const float* s, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(x[i], x[8 + i], c[i], s[i]);
    }
}

// Rows of `heads` heads to rotate, x into y (which may be x).
struct RowSet {
    const void* x;
    void* y;
    const float* weight;
    long long xb, xt, xh, yb, yt, yh;  // strides in elements: batch, token, head
    int heads;
};

// A warp takes one token (or a share of its heads): the lane's table entries stay in registers over the heads.
template <typename T, int kLanes>
__device__ __forceinline__ void rotate_heads(const RowSet& r, const T* x0, T* y0, int h0, int h1, int lane, int D,
                                             bool live, bool turn, int c0, int c1, const float* c, const float* s,
                                             bool interleaved, float eps) {
    constexpr int kRows = 32 / kLanes;
    float w[16];
    if (r.weight && live) {
        load8(r.weight + c0, w);
        load8(r.weight + c1, w + 8);
    }
#pragma unroll 2
    for (int h = h0 + lane / kLanes; h < h1 + lane / kLanes; h += kRows) {  // whole warps: shuffles below
        const bool on = live && h < h1;
        float x[16];
        if (on) {
            load8(x0 + h * r.xh + c0, x);
            load8(x0 + h * r.xh + c1, x + 8);
        }
        if (r.weight) {
            float ss = 0.f;
            if (on) {
#pragma unroll
                for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float n = rsqrtf(ss / D + eps);
            if (on) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] *= n * w[i];
            }
        }
        if (on) {
            if (turn) rotate_unit(x, c, s, interleaved);
            store8(y0 + h * r.yh + c0, x);
            store8(y0 + h * r.yh + c1, x + 8);
        }
    }
}

}  // namespace bsa
