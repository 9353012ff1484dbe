// The 4-bit paged cache: its layout and the numbers in it.
//
// A page holds page_size tokens (a power of two, 16 .. 1024), cut into strips of
// 16 tokens per KV head: the cache is [n_pages][H][page_size / 16][18 * D] bytes
// and a strip is
//   K codes   [16 tokens][D / 2]
//   V codes   [D / 16 groups][16 tokens][8]
//   K scales  [16 tokens][D / 16]
//   V scales  [D / 16 groups][16 tokens]
// Codes are E2M1 (two to a byte, the even channel in the low nibble), scales E4M3,
// one per token and 16 channels.  A strip is one contiguous run, so one bulk copy
// brings everything that 16 keys of a head need.  K is token-major because a key's
// channels are summed over; V is group-major because there the tokens are, and a
// tensor-core fragment then reads its tokens' channels from adjacent bytes.
//
// E2M1 has 2 and E4M3 4 significant bits, so code * scale has at most 6, and lies
// between 2^-10 and 2688: it is exact in float16 and in bfloat16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace bsa {

constexpr int kStrip = 16;        // tokens of a strip
constexpr float kE2M1Max = 6.f;
constexpr float kE4M3Max = 448.f;

__host__ __device__ constexpr int strip_bytes(int D) { return 18 * D; }

inline bool page_size_ok(int P) { return P >= 16 && P <= 1024 && (P & (P - 1)) == 0; }
inline int log2i(int x) { int s = 0; while ((1 << s) < x) ++s; return s; }

// Two E2M1 codes (one byte, low nibble first) as float16.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tmov.b32 {b, _, _, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
    return r;
}
// Two E4M3 values (16 bits, low byte first) as float16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tmov.b32 {h, _}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// E2M1 codes of two floats (round to nearest even, saturating), the first in the low nibble.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, 0, 0, 0};\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// E4M3 of a float >= 0 (round to nearest even, saturating).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, 0f00000000, %1;\n\tmov.b32 %0, {h, 0};\n\t}"
        : "=r"(r) : "f"(x));
    return r & 0xffu;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) {
    return __half22float2(*reinterpret_cast<__half2*>(&x));
}

}  // namespace bsa
