// Attention over the 4-bit paged cache (a14) on the tensor cores, D = 64 or 128.
//
// A row is one token's up to 16 query heads of one KV head.  Its strips (16 keys each,
// one contiguous run of 18 D bytes) are dealt out in tiles of four: to the row's CTAs in
// equal runs, within a CTA to its four warps in turn.  Every warp works alone until its
// keys are done: it copies its tiles into a ring of its own (one bulk copy per strip),
// keeps its own running maximum, sum and output, and meets the others only in the merge
//   m = max m_w,   l = sum l_w 2^(m_w - m),   U = sum U_w 2^(m_w - m),   O = U / l
// over the warps (shared memory), the CTAs of a cluster (distributed shared memory) and,
// where a row is cut finer than a cluster, over the clusters (workspace, second kernel).
//
// Numbers.  code * scale is exact in float16, so K and V enter the products exactly.  A
// row of q is scaled by the power of two that brings its largest magnitude to 2^14..2^15
// and is then exact in float16 when it is bf16 (8 bits, over 28 binades); a float32 q is
// split into two float16 parts.  Weights are 2^15 times their value (so that float16 keeps
// full precision over 29 binades below the largest) and rounded to float16 for bf16
// outputs, u = 2^-11 against the output's own 2^-8, or split in two for float32 ones.
// Maxima, sums and both accumulators are float32.
//
// Fragments.  mma.m16n8k16 lets the summed index be permuted freely as long as both
// operands agree, so a lane takes what lies together: of K the D / 4 consecutive channels
// of one key (one 16-byte load at D = 128), of V the D / 8 consecutive channels of four keys.
// Codes become float16 with cvt (two per byte) and one multiplication by their scales;
// V's codes are first paired along the keys, four logic instructions per 16 codes.
// No converted value is ever written back to shared memory.
#include <algorithm>

#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 4;     // strips of a tile
constexpr int kStages = 2;   // tiles of a warp's ring
constexpr uint64_t kWaitNs = 500ull * 1000 * 1000;
constexpr float kWeightLog2 = 15.f;

struct Split {
    int head_tiles;  // tiles of 16 query heads per KV head
    int splits;      // CTAs of a row: clusters of a row times cluster size
    int clusters;
    float* part;     // [rows][clusters][16][D] when clusters > 1
    float2* ml;      // [rows][clusters][16]
};

// ---------------------------------------------------------------- pieces

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Eight codes -> four float16 pairs, in byte order.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t* out) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// (a's low nibbles | b's low nibbles << 4) and the same of the high ones: codes paired along the keys.
__device__ __forceinline__ void pair_nibbles(uint32_t a, uint32_t b, uint32_t& even, uint32_t& odd) {
    constexpr uint32_t m = 0x0f0f0f0fu;
    even = (a & m) | ((b << 4) & ~m);
    odd = ((a >> 4) & m) | (b & ~m);
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
template <typename V> __device__ __forceinline__ V lds(uint32_t addr);
template <> __device__ __forceinline__ uint4 lds<uint4>(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint2 lds<uint2>(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint32_t lds<uint32_t>(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint16_t lds<uint16_t>(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint8_t lds<uint8_t>(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return (uint8_t)v;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// 2^(m_w - m) of a part (m_w, l_w); a part without keys weighs nothing, one whose logits
// are all NaN stays NaN.
__device__ __forceinline__ float weight_of(float2 part, float m) {
    return part.x == -INFINITY && part.y == 0.f ? 0.f : ptx::ex2(part.x - m);
}

// Waits for a tile; after kWaitNs latches BSA_ERR_TIMEOUT and gives up.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, int* status) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > kWaitNs) {
            raise_status(status, BSA_ERR_TIMEOUT);
            return false;
        }
    return true;
}

// ---------------------------------------------------------------- shared memory

template <int D>
struct Layout {
    static constexpr int kStripB = strip_bytes(D);
    static constexpr int kTileB = kTile * kStripB;
    static constexpr int kRing = kWarps * kStages * kTileB;
    // merge: four warps' U, rows padded so that a quarter warp's 16-byte stores meet no bank twice
    static constexpr int kRow = D + 16;
    static constexpr int kMerge = kWarps * 16 * kRow * 4;
    static constexpr int kBuf = kRing > kMerge ? kRing : kMerge;
    static constexpr int kBars = kBuf;                                // kWarps * kStages mbarriers
    static constexpr int kFirst = kBars + kWarps * kStages * 8;       // first key of each strip of the ring
    static constexpr int kML = kFirst + kWarps * kStages * kTile * 4; // (m, l) of each warp and row; then the CTA's
    static constexpr int kBytes = kML + kWarps * 16 * 8;
    static __device__ __forceinline__ int at(int row, int ch) { return row * kRow + ch + ch / (D / 4) * 4; }
};

// ---------------------------------------------------------------- the kernel

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 3 : 2) cache_attn_mma_kernel(CacheAttn a, Split sp) {
    using L = Layout<D>;
    constexpr int kTerms = sizeof(T) == 2 ? 1 : 2;  // float16 parts of q and of the weights
    constexpr int kSteps = D / 16;                  // k-steps of q K^T
    constexpr int kCh = D / 8;                      // channels of a lane's V fragment, and n-tiles of U
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int split = blockIdx.x % sp.splits, row_tile = blockIdx.x / sp.splits;
    const int tile_h = row_tile % sp.head_tiles, h = row_tile / sp.head_tiles % a.H, t = row_tile / sp.head_tiles / a.H;
    const int G = a.HQ / a.H, heads = min(16, G - tile_h * 16), hq0 = h * G + tile_h * 16;

    const Row row = row_of(a, t, h, tid == 0);
    if (row.req < 0) return;  // the whole cluster shares the row

    const int tiles = (row.strips + kTile - 1) / kTile;
    const int lo = (int)((long long)tiles * split / sp.splits), hi = (int)((long long)tiles * (split + 1) / sp.splits);
    const int mine = max(0, (hi - lo - warp + kWarps - 1) / kWarps);

    const uint32_t ring = sbase + warp * kStages * L::kTileB;
    const uint32_t bars = sbase + L::kBars + warp * kStages * 8;
    int* firsts = reinterpret_cast<int*>(smem + L::kFirst) + warp * kStages * kTile;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(bars + s * 8, 1);
        ptx::fence_mbar_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();

    // Lane i holds strip i % 4 of the warp's tile 8 b + i / 4: its first key (-1: none to see) and its place.
    auto resolve = [&](int b, int& first, int& place) {
        const int tile = lo + warp + (8 * b + (lane >> 2)) * kWarps, n = tile * kTile + (lane & 3);
        first = -1, place = 0;
        if (tile >= hi || n >= row.strips) return;
        first = first_key(a, row, n, true);
        if (first < 0) return;
        place = strip_index(a, row, h, first, true);
        if (place < 0) first = -1;
    };
    int first, place, next_first = -1, next_place = 0;
    resolve(0, first, place);
    auto issue = [&](int j) {
        const int src = (j & 7) * 4 + c, stage = j % kStages;
        const int f = __shfl_sync(0xffffffffu, first, src), p = __shfl_sync(0xffffffffu, place, src);
        const uint32_t live = __ballot_sync(0xffffffffu, f >= 0) & 15u;
        if (lane < 4) firsts[stage * kTile + lane] = f;
        if (lane == 0) ptx::mbar_arrive_expect_tx(bars + stage * 8, __popc(live) * L::kStripB);
        __syncwarp();
        if (lane < 4 && f >= 0)
            bulk_copy(ring + stage * L::kTileB + lane * L::kStripB, a.cache + (long long)p * L::kStripB, L::kStripB,
                      bars + stage * 8);
    };
    for (int j = 0; j < kStages && j < mine; ++j) issue(j);

    // q: lane (g, c) holds channels c D/4 .. of rows g and g + 8
    uint32_t qa[kTerms][kSteps][4];
    float rs[2];
    {
        const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (long long)hq0 * D + c * (D / 4);
        const float ks = (a.k_scale ? a.k_scale[h] : 1.f) * a.scale_log2;
        const bool wide = (((uintptr_t)a.q | (uintptr_t)(a.q_stride * (long long)sizeof(T))) & 15) == 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = g + half * 8;
            float x[D / 4];
            if (r < heads) {
                const T* p = q + (long long)r * D;
                if (wide) {
                    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
                    for (int i = 0; i < D / 4 / kPer; ++i) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (sizeof(T) == 2) {
                                x[i * kPer + 2 * e] = __uint_as_float(w[e] << 16);
                                x[i * kPer + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                            } else {
                                x[i * kPer + e] = __uint_as_float(w[e]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) x[i] = to_f32(p[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
            }
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - floor(log2 top)), its exponent kept in range; zero, infinite and NaN rows stay as they are
            const int e = (int)(__float_as_uint(top) >> 23);
            const int up = e == 0 || e == 255 ? 0 : min(126, 14 + 127 - e);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
            rs[half] = ks * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const float x0 = x[4 * s + 2 * e2] * f, x1 = x[4 * s + 2 * e2 + 1] * f;
                    const uint32_t hi2 = pack_f16x2(x0, x1);
                    qa[0][s][half + 2 * e2] = hi2;
                    if constexpr (kTerms == 2) {
                        const float2 b = f16x2_to_f32(hi2);
                        qa[1][s][half + 2 * e2] = pack_f16x2(x0 - b.x, x1 - b.y);
                    }
                }
        }
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, u[kCh][4];
#pragma unroll
    for (int j = 0; j < kCh; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[j][i] = 0.f;

    bool alive = true;
    for (int j = 0; j < mine; ++j) {
        const int stage = j % kStages;
        const uint32_t bar = bars + stage * 8, parity = (j / kStages) & 1, tile = ring + stage * L::kTileB;
        if (!ptx::mbar_try_wait(bar, parity)) alive = wait_slow(bar, parity, a.status);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;  // nothing is issued any more; the copies in flight are waited for below
        int fk[kTile];
#pragma unroll
        for (int i = 0; i < kTile; ++i) fk[i] = firsts[stage * kTile + i];

        // ---- S = q K^T
        float s[kTile][2][4];
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
            if (fk[i] < 0) continue;
            const uint32_t strip = tile + i * L::kStripB;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int key = g + 8 * n;
                uint32_t w[D / 32], sc[2];
                if constexpr (D == 128) {
                    const uint4 v = lds<uint4>(strip + key * 64 + c * 16);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                    const uint32_t two = e4m3x2_to_f16x2(lds<uint16_t>(strip + 16 * D + key * 8 + c * 2));
                    sc[0] = __byte_perm(two, two, 0x1010);
                    sc[1] = __byte_perm(two, two, 0x3232);
                } else {
                    const uint2 v = lds<uint2>(strip + key * 32 + c * 8);
                    w[0] = v.x, w[1] = v.y;
                    const uint32_t one = e4m3x2_to_f16x2(lds<uint8_t>(strip + 16 * D + key * 4 + c));
                    sc[0] = sc[1] = __byte_perm(one, one, 0x1010);
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t b[4];
                    unpack8(w[x], b);
                    const uint32_t scale = sc[x * 2 / (D / 32)];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = hmul2(b[e], scale);
#pragma unroll
                    for (int term = 0; term < kTerms; ++term) {
                        mma(s[i][n], qa[term][2 * x], b[0], b[1]);
                        mma(s[i][n], qa[term][2 * x + 1], b[2], b[3]);
                    }
                }
            }
        }

        // ---- logits in base 2, masked; running maximum
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            const int seen = fk[i] < 0 ? -1 : row.pos - fk[i];  // the strip's last visible key
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = n * 8 + c * 2 + (e & 1);
                    s[i][n][e] = key <= seen ? s[i][n][e] * rs[e >> 1] : -INFINITY;
                    top[e >> 1] = fmaxf(top[e >> 1], s[i][n][e]);
                }
        }
        bool moved = false;
        float base[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            top[r] = fmaxf(top[r], m[r]);
            moved = moved || top[r] != m[r];
            base[r] = top[r] == -INFINITY ? 0.f : top[r] - kWeightLog2;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float f = top[r] == -INFINITY ? 1.f : ptx::ex2(m[r] - top[r]);
                l[r] *= f;
                m[r] = top[r];
#pragma unroll
                for (int j2 = 0; j2 < kCh; ++j2) u[j2][2 * r] *= f, u[j2][2 * r + 1] *= f;
            }
        }

        // ---- weights and U += P V
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            if (fk[i] < 0) continue;
            uint32_t pa[kTerms][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = ptx::ex2(s[i][n][2 * r] - base[r]), p1 = ptx::ex2(s[i][n][2 * r + 1] - base[r]);
                    l[r] += p0 + p1;
                    const uint32_t two = pack_f16x2(p0, p1);
                    pa[0][2 * n + r] = two;
                    if constexpr (kTerms == 2) {
                        const float2 b = f16x2_to_f32(two);
                        pa[1][2 * n + r] = pack_f16x2(p0 - b.x, p1 - b.y);
                    }
                }
            const uint32_t strip = tile + i * L::kStripB;
            const int grp = D == 128 ? g : g >> 1;
            uint32_t s0 = e4m3x2_to_f16x2(lds<uint16_t>(strip + 17 * D + grp * 16 + c * 2));
            uint32_t s1 = e4m3x2_to_f16x2(lds<uint16_t>(strip + 17 * D + grp * 16 + c * 2 + 8));
            const int seen = row.pos - fk[i];
            if (seen < kStrip - 1) {  // keys behind the position may hold anything
                const int k0 = c * 2;
                s0 &= (k0 <= seen ? 0xffffu : 0u) | (k0 + 1 <= seen ? 0xffff0000u : 0u);
                s1 &= (k0 + 8 <= seen ? 0xffffu : 0u) | (k0 + 9 <= seen ? 0xffff0000u : 0u);
            }
            // the codes of keys (2c, 2c + 1) and (2c + 8, 2c + 9): kCh / 8 words of each
            uint32_t va[2][2][kCh / 8];
            if constexpr (D == 128) {
                // odd groups read their halves in the other order: a quarter warp then meets no bank twice
                const uint32_t at = strip + 8 * D + g * 128 + c * 16, flip = (g & 1) * 64;
                const uint4 x = lds<uint4>(at + flip), y = lds<uint4>(at + 64 - flip);
                const uint4 v0 = flip ? y : x, v1 = flip ? x : y;
                va[0][0][0] = v0.x, va[0][0][1] = v0.y, va[0][1][0] = v0.z, va[0][1][1] = v0.w;
                va[1][0][0] = v1.x, va[1][0][1] = v1.y, va[1][1][0] = v1.z, va[1][1][1] = v1.w;
            } else {
                const uint32_t at = strip + 8 * D + ((g >> 1) * 16 + c * 2) * 8 + (g & 1) * 4;
                va[0][0][0] = lds<uint32_t>(at), va[0][1][0] = lds<uint32_t>(at + 8);
                va[1][0][0] = lds<uint32_t>(at + 64), va[1][1][0] = lds<uint32_t>(at + 72);
            }
#pragma unroll
            for (int w = 0; w < kCh / 8; ++w) {
                uint32_t b0[2][4], b1[2][4], even, odd;  // [channel parity][channel / 2]
                pair_nibbles(va[0][0][w], va[0][1][w], even, odd);
                unpack8(even, b0[0]);
                unpack8(odd, b0[1]);
                pair_nibbles(va[1][0][w], va[1][1][w], even, odd);
                unpack8(even, b1[0]);
                unpack8(odd, b1[1]);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t v0 = hmul2(b0[x & 1][x >> 1], s0), v1 = hmul2(b1[x & 1][x >> 1], s1);
#pragma unroll
                    for (int term = 0; term < kTerms; ++term) mma(u[w * 8 + x], pa[term], v0, v1);
                }
            }
        }
        __syncwarp();
        const int jn = j + kStages;
        if (jn < mine) {
            if ((jn & 7) == 0) first = next_first, place = next_place;
            issue(jn);
            if ((jn & 7) == 4) resolve((jn >> 3) + 1, next_first, next_place);
        }
    }
    if (!alive)  // bounded too: let the copies of the ring land before the memory is given up
        for (int s = 0; s < kStages; ++s) wait_slow(bars + s * 8, 0, a.status), wait_slow(bars + s * 8, 1, a.status);

    // ---- merge the warps
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    float2* ml = reinterpret_cast<float2*>(smem + L::kML);
    float* U = reinterpret_cast<float*>(smem);
    if (c == 0) {
        ml[warp * 16 + g] = make_float2(m[0], l[0]);
        ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();  // every warp is done with its ring
    float cm[2], cl[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float2 w[kWarps];
        cm[r] = -INFINITY, cl[r] = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            w[k] = ml[k * 16 + g + 8 * r];
            cm[r] = fmaxf(cm[r], w[k].x);
        }
#pragma unroll
        for (int k = 0; k < kWarps; ++k) cl[r] += w[k].y * weight_of(w[k], cm[r]);
        const float f = weight_of(make_float2(m[r], l[r]), cm[r]);
        float* dst = U + warp * 16 * L::kRow;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < kCh / 4; ++i) {
                float4 v;
                v.x = u[4 * i][2 * r + e] * f, v.y = u[4 * i + 1][2 * r + e] * f;
                v.z = u[4 * i + 2][2 * r + e] * f, v.w = u[4 * i + 3][2 * r + e] * f;
                *reinterpret_cast<float4*>(dst + L::at(g + 8 * r, (2 * c + e) * kCh + 4 * i)) = v;
            }
    }
    __syncthreads();
    if (warp == 0 && c == 0) {
        ml[g] = make_float2(cm[0], cl[0]);
        ml[g + 8] = make_float2(cm[1], cl[1]);
    }
    const int csize = sp.splits / sp.clusters;
    const uint32_t rank = csize > 1 ? cluster_rank() : 0;
    constexpr int kVecs = 16 * D / 4;  // float4s of U
    if (csize > 1) {
        // the CTA's sum into the first warp's rows, where the others of the cluster read it
#pragma unroll
        for (int v = tid; v < kVecs; v += kWarps * 32) {
            float4* p = reinterpret_cast<float4*>(U + L::at(v / (D / 4), v % (D / 4) * 4));
            float4 x = p[0];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) {
                const float4 y = p[k * 4 * L::kRow];
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            p[0] = x;
        }
        cluster_sync();
    } else {
        __syncthreads();
    }
    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
    const int cl_id = split / csize;
    for (int v = rank * (kVecs / csize) + tid; v < (int)(rank + 1) * (kVecs / csize); v += kWarps * 32) {
        const int r = v / (D / 4), ch = v % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float mm = -INFINITY, ll = 0.f;
        if (csize > 1) {
            const uint32_t mine_ml = sbase + L::kML + r * 8, mine_u = sbase + L::at(r, ch) * 4;
            for (int k = 0; k < csize; ++k) mm = fmaxf(mm, ld_cluster2(at_rank(mine_ml, k)).x);
            for (int k = 0; k < csize; ++k) {
                const float2 w = ld_cluster2(at_rank(mine_ml, k));
                const float f = weight_of(w, mm);
                const float4 y = ld_cluster4(at_rank(mine_u, k));
                ll += w.y * f;
                x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
            }
        } else {
            mm = ml[r].x, ll = ml[r].y;
            const float4* p = reinterpret_cast<const float4*>(U + L::at(r, ch));
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 y = p[k * 4 * L::kRow];
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
        }
        if (sp.clusters > 1) {
            const long long at = ((long long)row_tile * sp.clusters + cl_id) * 16 + r;
            *reinterpret_cast<float4*>(sp.part + at * D + ch) = x;
            if (ch == 0) sp.ml[at] = make_float2(mm, ll);
        } else if (r < heads) {
            const long long at = (long long)t * a.HQ + hq0 + r;
            const float f = ll == 0.f ? 0.f : vs / ll;
            T* o = static_cast<T*>(a.out) + at * D + ch;
            o[0] = from_f32<T>(x.x * f), o[1] = from_f32<T>(x.y * f);
            o[2] = from_f32<T>(x.z * f), o[3] = from_f32<T>(x.w * f);
            if (a.lse && ch == 0) a.lse[at] = ll == 0.f ? -INFINITY : (mm - kWeightLog2 + log2f(ll)) * kLn2;
        }
    }
    if (csize > 1) cluster_sync();  // nobody leaves while others read its shared memory
}

// The rows' clusters joined: a warp per query head.
template <int D, typename T>
__global__ void __launch_bounds__(128) cache_attn_join_kernel(CacheAttn a, Split sp) {
    const int lane = threadIdx.x & 31, G = a.HQ / a.H;
    const long long head = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (head >= (long long)a.T * a.HQ) return;
    const int t = (int)(head / a.HQ), hq = (int)(head % a.HQ), h = hq / G, in = hq % G;
    if (a.req[t] < 0 || a.req[t] >= a.R) return;
    const long long at = (((long long)t * a.H + h) * sp.head_tiles + in / 16) * sp.clusters * 16 + in % 16;
    constexpr int kPer = D / 32;
    float mm = -INFINITY, ll = 0.f, x[kPer] = {};
    for (int k = 0; k < sp.clusters; ++k) mm = fmaxf(mm, sp.ml[at + k * 16].x);
    for (int k = 0; k < sp.clusters; ++k) {
        const float2 w = sp.ml[at + k * 16];
        const float f = weight_of(w, mm);
        ll += w.y * f;
        const float* p = sp.part + (at + k * 16) * D + lane * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] += p[i] * f;
    }
    const float f = ll == 0.f ? 0.f : (a.v_scale ? a.v_scale[h] : 1.f) / ll;
    T* o = static_cast<T*>(a.out) + head * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = from_f32<T>(x[i] * f);
    if (a.lse && lane == 0) a.lse[head] = ll == 0.f ? -INFINITY : (mm - kWeightLog2 + log2f(ll)) * kLn2;
}

constexpr int kSlots = 152 * 3;  // CTAs resident at once

// How a row is cut, from the sizes that the host knows.
void plan(int T, int HQ, int H, long long max_keys, int* head_tiles, int* cluster, int* clusters) {
    *head_tiles = (HQ / H + 15) / 16;
    const long long rows = (long long)T * H * *head_tiles;
    const long long tiles = (max_keys + kTile * kStrip - 1) / (kTile * kStrip);
    const long long most = std::max<long long>(1, (tiles + kWarps - 1) / kWarps);  // a tile for every warp at least
    const long long want = std::min(most, std::max<long long>(1, kSlots / std::max<long long>(rows, 1)));
    int c = 1;
    while (c < 8 && 2 * c <= want) c *= 2;
    *cluster = c;
    *clusters = (int)(want / c);
}

template <int D, typename T>
bsa_status launch(const CacheAttn& a, Split sp, int cluster, cudaStream_t st) {
    using L = Layout<D>;
    auto kern = cache_attn_mma_kernel<D, T>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != cudaSuccess) return fail(BSA_ERR_CUDA, "cache_attn_mma_kernel: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.T * a.H * sp.head_tiles * sp.splits));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cudaLaunchKernelEx(&cfg, kern, a, sp);
    bsa_status rc = check_launch("cache_attn_mma_kernel");
    if (rc != BSA_OK || sp.clusters == 1) return rc;
    const long long heads = (long long)a.T * a.HQ;
    cache_attn_join_kernel<D, T><<<(unsigned)((heads + 3) / 4), 128, 0, st>>>(a, sp);
    return check_launch("cache_attn_join_kernel");
}

}  // namespace

size_t mma_cache_attention_workspace(int T, int HQ, int H, int D, long long max_keys) {
    int head_tiles, cluster, clusters;
    plan(T, HQ, H, max_keys, &head_tiles, &cluster, &clusters);
    return clusters == 1 ? 0 : (size_t)T * H * head_tiles * clusters * 16 * (D + 2) * sizeof(float);
}

bsa_status mma_cache_attention(const CacheAttn& a, bsa_dtype dtype, long long max_keys, void* workspace,
                               cudaStream_t st) {
    Split sp;
    int cluster;
    plan(a.T, a.HQ, a.H, max_keys, &sp.head_tiles, &cluster, &sp.clusters);
    sp.splits = cluster * sp.clusters;
    const long long rows = (long long)a.T * a.H * sp.head_tiles;
    if (rows * sp.splits > 0x7fffffffLL) return fail(BSA_ERR_UNSUPPORTED, "cache attention: too many (token, head) rows");
    sp.part = static_cast<float*>(workspace);
    sp.ml = reinterpret_cast<float2*>(sp.part + (sp.clusters > 1 ? rows * sp.clusters * 16 * a.D : 0));
    if (dtype == BSA_F32) return a.D == 128 ? launch<128, float>(a, sp, cluster, st) : launch<64, float>(a, sp, cluster, st);
    return a.D == 128 ? launch<128, __nv_bfloat16>(a, sp, cluster, st) : launch<64, __nv_bfloat16>(a, sp, cluster, st);
}

}  // namespace bsa
