// a18 cross attention of few rows (single tokens, drafts): bf16, head dims up to 128 that are multiples of 8.
//
// "VSA 实现详解：三维分块、均值路由与块稀疏 Attention" §6.5 for the online softmax in the log2 domain.
//
// A row tile is the 16 rows of one warp-level product (tokens x the heads of a KV head); what bounds it is the read of
// K and V.  A warp takes 16 keys at a time straight from global memory into the fragments of its products, no shared
// memory between: the sum over channels may run in any order, so lane (g, c) = (lane / 4, lane % 4) reads 16 bytes of
// key g at channels 8 (c + 4 i), which are its four registers of two products' K, and the queries are laid out the same
// way; of V it reads 16 bytes at channels 8 g of the four keys 2c, 2c + 1, 2c + 8, 2c + 9 whose weights it holds, so
// that channel 8 g + j is column g of product j.  The next 16 keys' reads go out as soon as a register is consumed:
// 8 KB a warp are on their way, 64 KB an SM.
// The four warps of a block, and the blocks of a cluster (up to 8, by shared memory of each other), join their parts
// of the keys; with more parts than that the second kernel does.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>

#include "cross.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace cross {

namespace cg = cooperative_groups;

constexpr int kRowTile = 16, kStep = 16, kWarps = 4;
constexpr float kGrow = 8.f;  // log2 units: the running maximum is raised, and O rescaled, only when it grows by more

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 read16(const __nv_bfloat16* p, bool on) {
    return on ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

template <int HD>  // 64 or 128: channels, padded with zeros
__global__ void __launch_bounds__(32 * kWarps, 2) cross_rows_kernel(const Cross a) {
    constexpr int kC = HD / 32, kV = HD / 64;  // 16-byte runs of K and of V a lane reads of a key
    extern __shared__ __align__(16) float rows_smem[];
    float* so = rows_smem;                                    // [kWarps][16][HD]
    float* sm = so + kWarps * kRowTile * HD;                  // [kWarps][16] maxima, then sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, part = blockIdx.z;
    int b, row0, q0, n, k0, m;
    tile_of<kRowTile>(a, blockIdx.x, b, row0);
    if (b < 0) return;  // the whole cluster
    queries_of(a, b, q0, n);
    keys_of(a, b, k0, m);
    const int rows = (int)min((long long)kRowTile, (long long)n * a.G - row0);
    const long long qbat = a.query_start ? 0 : b, kbat = a.key_start ? 0 : b;
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + qbat * a.qb + (long long)h * a.G * a.qh;
    const __nv_bfloat16* k = (const __nv_bfloat16*)a.k + kbat * a.kb + (long long)h * a.kh + k0 * a.kt;
    const __nv_bfloat16* v = (const __nv_bfloat16*)a.v + kbat * a.vb + (long long)h * a.vh + k0 * a.vt;

    uint32_t qa[2 * kC][4];  // A operands of the products over channels
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = row0 + g + 8 * s;
            const int t = r / a.G;
            const uint4 x = read16(q + (q0 + t) * a.qt + (r - t * a.G) * a.qh + 8 * (c + 4 * i), g + 8 * s < rows && 8 * (c + 4 * i) < a.D);
            qa[2 * i][s] = x.x, qa[2 * i][2 + s] = x.y, qa[2 * i + 1][s] = x.z, qa[2 * i + 1][2 + s] = x.w;
        }

    const int nt = (m + kStep - 1) / kStep;
    const int t1 = (int)((long long)nt * (part + 1) / a.parts);
    int t = (int)((long long)nt * part / a.parts) + warp;
    uint4 kx[2][kC], vx[4][kV];
    auto read_k = [&](int step) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int key = step * kStep + 8 * s + g;
            const __nv_bfloat16* p = k + (long long)key * a.kt;
#pragma unroll
            for (int i = 0; i < kC; ++i) kx[s][i] = read16(p + 8 * (c + 4 * i), step < t1 && key < m && 8 * (c + 4 * i) < a.D);
        }
    };
    auto read_v = [&](int step) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int key = step * kStep + 8 * (s >> 1) + 2 * c + (s & 1);
            const __nv_bfloat16* p = v + (long long)key * a.vt;
#pragma unroll
            for (int i = 0; i < kV; ++i) vx[s][i] = read16(p + 8 * (g + 8 * i), step < t1 && key < m && 8 * (g + 8 * i) < a.D);
        }
    };
    const float scale = fmaxf(a.scale * kLog2e, 1.2e-38f);  // 0 would turn a masked -inf into NaN
    float ref[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f}, o[8 * kV][4];
#pragma unroll
    for (int j = 0; j < 8 * kV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    read_k(t);
    read_v(t);
    for (; t < t1; t += kWarps) {
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mma16816(s[u], qa[2 * i], kx[u][i].x, kx[u][i].y);
                mma16816(s[u], qa[2 * i + 1], kx[u][i].z, kx[u][i].w);
            }
        read_k(t + kWarps);
        if (t * kStep + kStep > m) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t * kStep + 8 * u + 2 * c + (e & 1) >= m) s[u][e] = -CUDART_INF_F;
        }
        float now[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            now[r] = fmaxf(ref[r], x * scale);
        }
        if (__any_sync(0xffffffffu, now[0] > ref[0] + kGrow || now[1] > ref[1] + kGrow)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool up = now[r] > ref[r] + kGrow;  // the same in a row's four lanes
                const float alpha = up ? ptx::ex2(ref[r] - now[r]) : 1.f;
                if (up) ref[r] = now[r];
                l[r] *= alpha;
#pragma unroll
                for (int j = 0; j < 8 * kV; ++j) {
                    o[j][2 * r] *= alpha;
                    o[j][2 * r + 1] *= alpha;
                }
            }
        }
        uint32_t p[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float base = ref[r] == -CUDART_INF_F ? 0.f : ref[r];
            float w[4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) w[2 * u + e] = ptx::ex2(fmaf(s[u][2 * r + e], scale, -base));
            l[r] += (w[0] + w[1]) + (w[2] + w[3]);
            p[r] = ptx::pack_bf16x2(w[0], w[1]);
            p[2 + r] = ptx::pack_bf16x2(w[2], w[3]);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t* x[4] = {&vx[0][i].x, &vx[1][i].x, &vx[2][i].x, &vx[3][i].x};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int sel = j & 1 ? 0x7632 : 0x5410;
                mma16816(o[8 * i + j], p, __byte_perm(x[0][j >> 1], x[1][j >> 1], sel), __byte_perm(x[2][j >> 1], x[3][j >> 1], sel));
            }
        }
        read_v(t + kWarps);
    }

    // the warps' parts: product j's columns 2c, 2c + 1 are channels 8 (2c) + j and 8 (2c + 1) + j of a run of 64
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        float* to = so + (warp * kRowTile + g + 8 * r) * HD;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4*>(to + 64 * i + 8 * (2 * c + e) + j) =
                        make_float4(o[8 * i + j][2 * r + e], o[8 * i + j + 1][2 * r + e], o[8 * i + j + 2][2 * r + e], o[8 * i + j + 3][2 * r + e]);
        if (c == 0) {
            sm[warp * kRowTile + g + 8 * r] = ref[r];
            sm[(kWarps + warp) * kRowTile + g + 8 * r] = l[r];
        }
    }
    auto cluster = cg::this_cluster();
    const int peers = cluster.num_blocks(), rank = cluster.block_rank();
    if (peers > 1) cluster.sync();
    else __syncthreads();
    // every block of the cluster finishes its share of the rows, four channels a thread
    const int per = (kRowTile + peers - 1) / peers;
    constexpr int kQuads = HD / 4;
    for (int i = threadIdx.x; i < per * kQuads; i += 32 * kWarps) {
        const int r = rank * per + i / kQuads, ch = i % kQuads * 4;
        if (r >= rows) break;
        float top = -CUDART_INF_F;
        for (int x = 0; x < peers; ++x) {
            const float* ps = peers > 1 ? cluster.map_shared_rank(sm, x) : sm;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ps[w * kRowTile + r]);
        }
        const float base = top == -CUDART_INF_F ? 0.f : top;
        float sum = 0.f, y[4] = {};
        for (int x = 0; x < peers; ++x) {
            const float* ps = peers > 1 ? cluster.map_shared_rank(sm, x) : sm;
            const float* po = peers > 1 ? cluster.map_shared_rank(so, x) : so;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ptx::ex2(ps[w * kRowTile + r] - base);
                sum = fmaf(ps[(kWarps + w) * kRowTile + r], f, sum);
                const float4 z = *reinterpret_cast<const float4*>(po + (w * kRowTile + r) * HD + ch);
                y[0] = fmaf(z.x, f, y[0]), y[1] = fmaf(z.y, f, y[1]), y[2] = fmaf(z.z, f, y[2]), y[3] = fmaf(z.w, f, y[3]);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum, lse = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= inv;
        const int rr = row0 + r, tok = q0 + rr / a.G, hq = h * a.G + rr % a.G;
        if (peers < a.parts) {
            const long long total = a.query_start ? a.N : (long long)a.B * a.N;
            const long long at = ((long long)(part / peers) * total + qbat * a.N + tok) * a.HQ + hq;
            if (ch < a.D) *reinterpret_cast<float4*>(a.part_out + at * a.D + ch) = make_float4(y[0], y[1], y[2], y[3]);
            if (ch == 0) a.part_lse[at] = lse;
        } else {
            if (ch < a.D)
                *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + qbat * a.ob + tok * a.ot + hq * a.oh + ch) =
                    make_uint2(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]));
            if (ch == 0 && a.lse) a.lse[qbat * a.lb + tok * a.lt + hq * a.lh] = lse;
        }
    }
    if (peers > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

template <int HD>
static bsa_status launch_rows(const Cross& a, int tiles, int cluster, cudaStream_t st) {
    constexpr int kSmem = sizeof(float) * (kWarps * kRowTile * HD + 2 * kWarps * kRowTile);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, a.H, a.parts);
    cfg.blockDim = 32 * kWarps;
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, cross_rows_kernel<HD>, a);
    return check_launch("cross_rows_kernel");
}

}  // namespace cross

// parts: of the keys, a multiple of `cluster`; the join then has parts / cluster of them.
bsa_status cross_rows(Cross a, int cluster, cudaStream_t st, bool* handled) {
    *handled = false;
    const long long tiles = row_tiles(a.B, a.N, a.G, a.query_start != nullptr, cross::kRowTile);
    uintptr_t any = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.out;
    for (long long s : {a.qb, a.qt, a.qh, a.kb, a.kt, a.kh, a.vb, a.vt, a.vh, a.ob, a.ot, a.oh}) any |= (uintptr_t)(2 * s);
    if ((any & 15) || a.M == 0 || a.H > 65535 || tiles > 0x7fffffffLL) return BSA_OK;
    *handled = true;
    return a.D <= 64 ? cross::launch_rows<64>(a, (int)tiles, cluster, st) : cross::launch_rows<128>(a, (int)tiles, cluster, st);
}

}  // namespace bsa
