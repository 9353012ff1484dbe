// a18 cross attention in float32 on the tensor cores: any head dim up to 128, any strides.
//
// "VSA 实现详解：三维分块、均值路由与块稀疏 Attention" §6.5 for the online softmax in the log2 domain.
//
// An operand x is split into x = hi + lo, both rounded to tf32, and a product is lo hi + hi lo + hi hi (what is left out,
// lo lo and lo's own roundings, is 3 x 2^-22 of it at most).  Where hi is infinite (an infinity, or a value within 2^-12 of
// the largest float) that is NaN: a block with NaN in its results takes its keys once more, with hi stopped at the largest
// value (kSat; the conversion that does so costs 10% where all blocks use it), and an infinity is then one in lo alone.
// A block holds 64 rows, 16 to a warp, against tiles of 32 keys that are copied two ahead of each other.  The weights of
// keys 2c and 2c + 1, which a lane of quad c holds after the product with K, are its operands at k = c and c + 4 of the
// product with V, whose rows are read in that order; a tile's weighted values are summed from zero and added to O
// rounded, because the tensor cores' own additions are not.
// Three products an element pair cost a third of the tf32 rate; the kernel is bound by the instructions around them (per
// three products two reads of shared memory and four to split them): 46 TFLOP/s at 4096 x 4096 x 8 heads, D = 128.
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "cross.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace cross {

constexpr int kFRows = 64, kFKeys = 32;  // the products take four column tiles of 8 at a time
// Key tiles whose sums are added up in registers: equal terms, and so equal roundings, would take 2^19 keys 2e-4 off.  After
// as many the sums are put aside, in the output's place, and those are added up (kLong, for calls whose states could be
// that long: the code for it costs 2 to 5%).
constexpr int kFAside = 128;

struct Split { uint32_t hi, lo; };
template <bool kSat = false>
__device__ __forceinline__ Split split(float x) {
    Split s;
    if constexpr (kSat) asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(s.hi) : "f"(x));
    else asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(s.hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(s.lo) : "f"(x - __uint_as_float(s.hi)));
    return s;
}
__device__ __forceinline__ void mma1688(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d[j] += a b[j] for four column tiles, the small products first; a tile's products depend on one another, so the
// tiles take turns.
__device__ __forceinline__ void mma3x4(float (*d)[4], const Split* a, const Split (*b)[2]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) mma1688(d[j], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[j][0].hi, b[j][1].hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) mma1688(d[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].lo, b[j][1].lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) mma1688(d[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].hi, b[j][1].hi);
}
// 16 or 4 bytes to shared memory, zeros where `on` is false.
template <int kBytes>
__device__ __forceinline__ void copy_in(float* dst, const float* src, bool on) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// HD: channels padded to 64 or 128; kBytes: 16 where rows can be copied by 16 bytes, else 4.
template <int HD, int kBytes, bool kLong>
__global__ void __launch_bounds__(128, HD == 64 ? 3 : 2) cross_f32_kernel(const Cross a) {
    constexpr int ld = HD + 4, kN = kBytes / 4, kTile = kFKeys * ld;
    extern __shared__ __align__(16) float f32_smem[];
    float *Qs = f32_smem, *KV = Qs + kFRows * ld;  // then K and V of two tiles
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, part = blockIdx.z;
    int b, row0, q0, n, k0, m;
    tile_of<kFRows>(a, blockIdx.x, b, row0);
    if (b < 0) return;
    queries_of(a, b, q0, n);
    keys_of(a, b, k0, m);
    const int rows = (int)min((long long)kFRows, (long long)n * a.G - row0);
    const long long qbat = a.query_start ? 0 : b, kbat = a.key_start ? 0 : b;
    const float* q = (const float*)a.q + qbat * a.qb + (long long)h * a.G * a.qh;
    const float* k = (const float*)a.k + kbat * a.kb + (long long)h * a.kh + k0 * a.kt;
    const float* v = (const float*)a.v + kbat * a.vb + (long long)h * a.vh + k0 * a.vt;
    for (int i = threadIdx.x; i < kFRows * (HD / kN); i += 128) {
        const int r = i / (HD / kN), d = i % (HD / kN) * kN, t = (row0 + r) / a.G;
        const bool on = r < rows && d < a.D;
        copy_in<kBytes>(Qs + r * ld + d, on ? q + (q0 + t) * a.qt + (row0 + r - t * a.G) * a.qh + d : q, on);
    }
    const int nt = (m + kFKeys - 1) / kFKeys, t1 = (int)((long long)nt * (part + 1) / a.parts);
    auto fetch = [&](int tile) {
        if (tile < t1) {
            float *K = KV + (tile & 1) * 2 * kTile, *V = K + kTile;
            for (int i = threadIdx.x; i < kFKeys * (HD / kN); i += 128) {
                const int r = i / (HD / kN), d = i % (HD / kN) * kN, key = tile * kFKeys + r;
                const bool on = key < m && d < a.D;
                copy_in<kBytes>(K + r * ld + d, on ? k + key * a.kt + d : k, on);
                copy_in<kBytes>(V + r * ld + d, on ? v + key * a.vt + d : v, on);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto pass = [&](auto sat) {  // whether there is a NaN among the thread's results
        constexpr bool kSat = decltype(sat)::value;
        int t = (int)((long long)nt * part / a.parts);
        fetch(t);
        const float scale = fmaxf(a.scale * kLog2e, 1.2e-38f);  // 0 would turn a masked -inf into NaN
        float mx[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f}, o[HD / 8][4] = {};
        float m_aside[2] = {-CUDART_INF_F, -CUDART_INF_F}, l_aside[2] = {0.f, 0.f};
        bool first = true, bad = false;  // first: nothing put aside
        for (int stop = kLong ? min(t1, t + kFAside) : t1;; stop = min(t1, stop + kFAside)) {
            for (; t < stop; ++t) {
                fetch(t + 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncthreads();
                const float *K = KV + (t & 1) * 2 * kTile, *V = K + kTile, *Q = Qs + (16 * warp) * ld;
                float s[kFKeys / 8][4] = {};
#pragma unroll 4
                for (int d = 0; d < HD; d += 8) {
                    const Split x[4] = {split<kSat>(Q[g * ld + d + c]), split<kSat>(Q[(g + 8) * ld + d + c]), split<kSat>(Q[g * ld + d + c + 4]),
                                        split<kSat>(Q[(g + 8) * ld + d + c + 4])};
                    Split y[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) y[j][e] = split<kSat>(K[(8 * j + g) * ld + d + c + 4 * e]);
                    mma3x4(s, x, y);
                }
                const int left = m - t * kFKeys;
                Split p[kFKeys / 8][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = -CUDART_INF_F;
#pragma unroll
                    for (int j = 0; j < kFKeys / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& x = s[j][2 * r + e];
                            x = 8 * j + 2 * c + e < left ? x * scale : -CUDART_INF_F;
                            top = fmaxf(top, x);
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float now = fmaxf(mx[r], top), ref = now == -CUDART_INF_F ? 0.f : now, alpha = exp2f(mx[r] - ref);
                    mx[r] = now;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < kFKeys / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float w = exp2f(s[j][2 * r + e] - ref);
                            if (kSat) w *= 0.5f;  // the largest float's two halves may add up to 2^128
                            sum += w;
                            p[j][2 * e + r] = split(w);
                        }
                    l[r] = l[r] * alpha + sum;
#pragma unroll
                    for (int j = 0; j < HD / 8; ++j) {
                        o[j][2 * r] *= alpha;
                        o[j][2 * r + 1] *= alpha;
                    }
                }
#pragma unroll
                for (int j0 = 0; j0 < HD / 8; j0 += 4) {
                    float y[4][4] = {};
#pragma unroll
                    for (int i = 0; i < kFKeys / 8; ++i) {
                        Split w[4][2];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) w[j][e] = split<kSat>(V[(8 * i + 2 * c + e) * ld + 8 * (j0 + j) + g]);
                        mma3x4(y, p[i], w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[j0 + j][e] += y[j][e];
                }
                __syncthreads();
            }
            const bool last = !kLong || t >= t1;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                const int at = 16 * warp + g + 8 * r;
                if (at >= rows) continue;
                const int rr = row0 + at, tok = q0 + rr / a.G, hq = h * a.G + rr % a.G;
                const float f = m_aside[r] == -CUDART_INF_F ? 0.f : exp2f(m_aside[r] - mx[r]);
                l_aside[r] = fmaf(l_aside[r], f, l[r]);
                m_aside[r] = mx[r];
                float* to = (float*)a.out + qbat * a.ob + tok * a.ot + hq * a.oh;
                float* to_lse = a.lse ? a.lse + qbat * a.lb + tok * a.lt + hq * a.lh : nullptr;
                if (a.parts > 1) {
                    const long long row = ((long long)part * (a.query_start ? a.N : (long long)a.B * a.N) + qbat * a.N + tok) * a.HQ + hq;
                    to = a.part_out + row * a.D;
                    to_lse = a.part_lse + row;
                }
                const float inv = !last ? 1.f : l_aside[r] == 0.f ? 0.f : 1.f / l_aside[r];
                if (last && c == 0 && to_lse) *to_lse = l_aside[r] == 0.f ? -CUDART_INF_F : (mx[r] + log2f(kSat ? 2.f * l_aside[r] : l_aside[r])) * kLn2;
                bad = bad || l_aside[r] != l_aside[r];
#pragma unroll
                for (int j = 0; j < HD / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* x = to + 8 * j + 2 * c + e;
                        if (8 * j + 2 * c + e >= a.D) continue;
                        const float y = !kLong || first ? o[j][2 * r + e] : fmaf(*x, f, o[j][2 * r + e]);
                        bad = bad || y != y;
                        *x = y * inv;
                    }
            }
            if (last) break;
            first = false;
            l[0] = l[1] = 0.f;
#pragma unroll
            for (int j = 0; j < HD / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        return bad;
    };
    if (__syncthreads_or(pass(std::false_type{}))) pass(std::true_type{});
}

template <int HD, int kBytes, bool kLong>
static bsa_status launch_f32(const Cross& a, cudaStream_t st) {
    constexpr int kSmem = sizeof(float) * (HD + 4) * (kFRows + 4 * kFKeys);
    cudaError_t e = cudaFuncSetAttribute(cross_f32_kernel<HD, kBytes, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return fail(BSA_ERR_CUDA, "cross attention attribute: %s", cudaGetErrorString(e));
    cross_f32_kernel<HD, kBytes, kLong><<<dim3((unsigned)a.tiles, a.H, a.parts), 128, kSmem, st>>>(a);
    return check_launch("cross_f32_kernel");
}
template <int HD, int kBytes>
static bsa_status launch_f32(const Cross& a, cudaStream_t st) {
    const int tiles = ((a.M + kFKeys - 1) / kFKeys + a.parts - 1) / a.parts;  // that an item may have
    return tiles > kFAside ? launch_f32<HD, kBytes, true>(a, st) : launch_f32<HD, kBytes, false>(a, st);
}

}  // namespace cross

// a.tiles: row tiles of 64 rows.
bsa_status cross_f32(const Cross& a, cudaStream_t st) {
    uintptr_t any = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v;
    for (long long s : {a.qb, a.qt, a.qh, a.kb, a.kt, a.kh, a.vb, a.vt, a.vh}) any |= (uintptr_t)(4 * s);
    if (a.D % 4 == 0 && (any & 15) == 0)
        return a.D <= 64 ? cross::launch_f32<64, 16>(a, st) : cross::launch_f32<128, 16>(a, st);
    return a.D <= 64 ? cross::launch_f32<64, 4>(a, st) : cross::launch_f32<128, 4>(a, st);
}

}  // namespace bsa
