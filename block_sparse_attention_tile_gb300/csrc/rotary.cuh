// Rotary positions: what the rotation of rows and the rotated cache append share.
//
// A pair (a, b) of channels turns by an angle given as (cos, sin):
//   a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))   in float32.
// Products and sums are rounded one by one, not fused: the result is then the same in whatever order a program
// computes it, and with it the 4-bit codes that the cache append makes of it.
//
// A row of D channels is cut into units of 8: two runs of 4 channels that a lane reads at once and whose pairs lie
// inside the unit.  Half layout: pair i is (i, i + P), unit u < P / 4 holds channels 4u .. and P + 4u ..; the rest of
// the row, 8 at a time, is copied.  Interleaved layout: pair i is (2i, 2i + 1), unit u holds channels 8u .. 8u + 7.
// In both, unit u turns by the table's entries 4u .. 4u + 3.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace bsa {

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Four channels as they lie in memory (8- or 16-byte aligned), and as floats.
template <typename T> struct Run4;
template <> struct Run4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void floats(float* x) const {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <> struct Run4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void floats(float* x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
// Eight table entries at 16-byte aligned p.
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Lanes that share a row of D channels: a power of two, 8 channels each.
__host__ __device__ constexpr int row_lanes(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Rows of `heads` heads to rotate, x into y (which may be x).
struct RowSet {
    const void* x;
    void* y;
    const float* weight;
    long long xb, xt, xh, yb, yt, yh;  // strides in elements: batch, token, head
    int heads;
};

// One token's heads [h0, h1) by a warp, 32 / kLanes rows a step; the lane's table entries stay in registers over them.
// The rows of kBatch steps are read before the first of them is written (y may be x: the compiler cannot move a read
// over a write).  What bounds it is the read and the write of every row once, so it is made for many bytes on their
// way at 64 registers: units of 8 channels, weights from L1.  (115200 tokens of 24 + 24 heads of 128 channels with a
// norm: units of 16 channels took 561 to 1000 us, by registers or spills; rows copied ahead into shared memory with
// 8 warps an SM 982; this one 489, 87% of the copy rate.)
template <typename T, int kLanes, bool kNorm, bool kInterleaved>
__device__ __forceinline__ void rotate_heads(const float* weight, const T* x, T* y, long long xh, long long yh, int h0,
                                             int h1, int D, int P, const float* c, const float* s, float eps) {
    constexpr int kRows = 32 / kLanes, kBatch = sizeof(T) == 2 ? 3 : 2;
    const int lane = threadIdx.x & 31, u = lane % kLanes, own = lane / kLanes;
    const bool live = 8 * u < D, turn = 4 * u < P;
    const int c0 = kInterleaved ? 8 * u : turn ? 4 * u : 2 * P + 8 * (u - P / 4), c1 = !kInterleaved && turn ? P + 4 * u : c0 + 4;
    x += (h0 + own) * xh + c0;
    y += (h0 + own) * yh + c0;
    const int d = c1 - c0;
    for (int h = h0; h < h1; h += kRows * kBatch) {
        Run4<T> a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (live && h + i * kRows + own < h1) {
                a[i].load(x);
                b[i].load(x + d);
            }
            x += kRows * xh;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (h + i * kRows >= h1) break;  // whole warps: shuffles below
            const bool on = live && h + i * kRows + own < h1;
            float z[8];
            a[i].floats(z);
            b[i].floats(z + 4);
            if (kNorm) {
                float ss = 0.f;
                if (on) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(z[e], z[e], ss);
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float n = rsqrtf(__fdividef(ss, (float)D) + eps);
                if (on) {
                    const float4 w0 = *reinterpret_cast<const float4*>(weight + c0), w1 = *reinterpret_cast<const float4*>(weight + c1);
                    z[0] *= n * w0.x, z[1] *= n * w0.y, z[2] *= n * w0.z, z[3] *= n * w0.w;
                    z[4] *= n * w1.x, z[5] *= n * w1.y, z[6] *= n * w1.z, z[7] *= n * w1.w;
                }
            }
            if (on) {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kInterleaved) rotate_pair(z[2 * e], z[2 * e + 1], c[e], s[e]);
                        else rotate_pair(z[e], z[4 + e], c[e], s[e]);
                    }
                }
                store4(y, z);
                store4(y + d, z + 4);
            }
            y += kRows * yh;
        }
    }
}

}  // namespace bsa
