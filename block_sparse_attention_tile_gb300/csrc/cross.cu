// a18 cross attention on the CUDA cores (sizes, strides and addresses that the tensor-core kernels do not take), the join
// of the keys' parts, and the entry points.
//
// "VSA 实现详解：三维分块、均值路由与块稀疏 Attention" §6.5: the log2-domain recurrence of the online softmax; a row with
// no key outputs zero.
#include <algorithm>
#include <climits>
#include <math_constants.h>

#include "cross.cuh"

namespace bsa {

// ---------------------------------------------------------------- CUDA cores
//
// A block holds 64 rows against 64 keys at a time: 16 x 16 threads, 4 rows x 4 keys of the logits and 4 rows x D / 16
// channels of the output each, both products from shared memory in float32.  A tile's weighted values are summed from zero
// and then added to the output: of 2^18 equal terms one after the other, equally rounded, an output was 4e-3 off.
constexpr int kSimtRows = 64, kSimtKeys = 64;

static size_t simt_smem(int D4) { return sizeof(float) * ((size_t)kSimtRows * (D4 + 4) + 2 * kSimtKeys * (D4 + 4) + kSimtRows * (kSimtKeys + 4)); }

template <typename T, int kC>  // kC: groups of 64 channels
__global__ void __launch_bounds__(256) cross_simt_kernel(const Cross a) {
    extern __shared__ __align__(16) float smem[];
    const int Dp = (a.D + 3) & ~3, ld = Dp + 4;
    float *Qs = smem, *Ks = Qs + kSimtRows * ld, *Vs = Ks + kSimtKeys * ld, *Ps = Vs + kSimtKeys * ld;
    constexpr int kPd = kSimtKeys + 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int h = blockIdx.y, part = blockIdx.z;
    int b, row0, q0, n, k0, m;
    tile_of<kSimtRows>(a, blockIdx.x, b, row0);
    if (b < 0) return;
    queries_of(a, b, q0, n);
    keys_of(a, b, k0, m);
    const long long rows = (long long)n * a.G;
    const int nr = (int)min((long long)kSimtRows, rows - row0);
    const long long qbat = a.query_start ? 0 : b, kbat = a.key_start ? 0 : b;
    const T* q = (const T*)a.q + qbat * a.qb + (long long)h * a.G * a.qh;
    const T* k = (const T*)a.k + kbat * a.kb + (long long)h * a.kh + k0 * a.kt;
    const T* v = (const T*)a.v + kbat * a.vb + (long long)h * a.vh + k0 * a.vt;
    const float scale = a.scale * kLog2e;
    for (int i = threadIdx.x; i < kSimtRows * Dp; i += 256) {
        const int r = i / Dp, d = i - r * Dp;
        float x = 0.f;
        if (r < nr && d < a.D) x = to_f32(q[(long long)(q0 + (row0 + r) / a.G) * a.qt + (row0 + r) % a.G * a.qh + d]);
        Qs[r * ld + d] = x * scale;
    }
    float mx[4], l[4], acc[4][kC][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        mx[r] = -CUDART_INF_F;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][c][e] = 0.f;
    }
    const int nt = (m + kSimtKeys - 1) / kSimtKeys;
    const int t1 = (int)((long long)nt * (part + 1) / a.parts);
    for (int t = (int)((long long)nt * part / a.parts); t < t1; ++t) {
        const int first = t * kSimtKeys, nk = min(kSimtKeys, m - first);
        __syncthreads();
        for (int i = threadIdx.x; i < kSimtKeys * Dp; i += 256) {
            const int r = i / Dp, d = i - r * Dp;
            const bool on = r < nk && d < a.D;
            Ks[r * ld + d] = on ? to_f32(k[(first + r) * a.kt + d]) : 0.f;
            Vs[r * ld + d] = on ? to_f32(v[(first + r) * a.vt + d]) : 0.f;
        }
        __syncthreads();
        float s[4][4] = {}, alpha[4];
        for (int d = 0; d < Dp; d += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) qv[r] = *reinterpret_cast<const float4*>(Qs + (4 * ty + r) * ld + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * ld + d);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[r][j] = fmaf(qv[r].x, kv[j].x, fmaf(qv[r].y, kv[j].y, fmaf(qv[r].z, kv[j].z, fmaf(qv[r].w, kv[j].w, s[r][j]))));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (tx + 16 * j >= nk) s[r][j] = -CUDART_INF_F;
                top = fmaxf(top, s[r][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float now = fmaxf(mx[r], top), ref = now == -CUDART_INF_F ? 0.f : now;
            alpha[r] = exp2f(mx[r] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[r][j] - ref);
                Ps[(4 * ty + r) * kPd + tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mx[r] = now;
            l[r] = l[r] * alpha[r] + sum;
        }
        __syncwarp();  // a row's weights are written and read by one warp
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            if (4 * tx + 64 * c >= Dp) continue;
            float y[4][4] = {};
            for (int j = 0; j < nk; j += 4) {  // keys behind the last: weights and values of 0
                float4 p[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(Ps + (4 * ty + r) * kPd + j);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 x = *reinterpret_cast<const float4*>(Vs + (j + u) * ld + 4 * tx + 64 * c);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = u == 0 ? p[r].x : u == 1 ? p[r].y : u == 2 ? p[r].z : p[r].w;
                        y[r][0] = fmaf(w, x.x, y[r][0]);
                        y[r][1] = fmaf(w, x.y, y[r][1]);
                        y[r][2] = fmaf(w, x.z, y[r][2]);
                        y[r][3] = fmaf(w, x.w, y[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][c][e] = fmaf(acc[r][c][e], alpha[r], y[r][e]);
        }
        __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (4 * ty + r >= nr) break;
        const int tok = q0 + (row0 + 4 * ty + r) / a.G, hq = h * a.G + (row0 + 4 * ty + r) % a.G;
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r], lse = l[r] == 0.f ? -CUDART_INF_F : (mx[r] + log2f(l[r])) * kLn2;
        if (a.parts > 1) {
            const long long total = a.query_start ? a.N : (long long)a.B * a.N;
            const long long at = (part * total + (a.query_start ? 0 : (long long)b * a.N) + tok) * a.HQ + hq;
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * tx + 64 * c + e < a.D) a.part_out[at * a.D + 4 * tx + 64 * c + e] = acc[r][c][e] * inv;
            if (tx == 0) a.part_lse[at] = lse;
        } else {
            T* o = (T*)a.out + qbat * a.ob + tok * a.ot + hq * a.oh;
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * tx + 64 * c + e < a.D) o[4 * tx + 64 * c + e] = from_f32<T>(acc[r][c][e] * inv);
            if (tx == 0 && a.lse) a.lse[qbat * a.lb + tok * a.lt + hq * a.lh] = lse;
        }
    }
}

// ---------------------------------------------------------------- join
//
// A warp a row, four channels a lane: out = sum_p exp(lse_p - L) out_p, L = log sum_p exp(lse_p), in the order of the
// parts.  (With eight rows a warp one after the other it took longer than what it joins.)
constexpr int kJoinRows = 8;  // a block

template <typename T>
__global__ void __launch_bounds__(32 * kJoinRows) cross_join_kernel(const Cross a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    int b, row0, q0, n;
    tile_of<kJoinRows>(a, blockIdx.x, b, row0);
    if (b < 0) return;
    queries_of(a, b, q0, n);
    const long long r = row0 + (threadIdx.x >> 5);
    if (r >= (long long)n * a.G) return;
    const int tok = q0 + (int)(r / a.G), hq = h * a.G + (int)(r % a.G), ch = 4 * lane;
    const long long total = a.query_start ? a.N : (long long)a.B * a.N, step = total * a.HQ, qbat = a.query_start ? 0 : b;
    const long long i = (qbat * a.N + tok) * a.HQ + hq;
    const bool wide = a.D % 4 == 0;
    float top = -CUDART_INF_F;
#pragma unroll 8
    for (int p = 0; p < a.parts; ++p) top = fmaxf(top, a.part_lse[p * step + i]);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f, y[4] = {};
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p) {
        const float* x = a.part_out + (p * step + i) * a.D + ch;
        float z[4] = {};
        if (wide) {
            if (ch < a.D) {
                const float4 v = *reinterpret_cast<const float4*>(x);
                z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ch + e < a.D) z[e] = x[e];
        }
        const float w = exp2f((a.part_lse[p * step + i] - ref) * kLog2e);
        sum += w;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fmaf(w, z[e], y[e]);
    }
    T* o = (T*)a.out + qbat * a.ob + tok * a.ot + hq * a.oh + ch;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (ch + e < a.D) o[e] = from_f32<T>(y[e] * inv);
    if (lane == 0 && a.lse) a.lse[qbat * a.lb + tok * a.lt + hq * a.lh] = sum == 0.f ? -CUDART_INF_F : top + log2f(sum) * kLn2;
}

// ---------------------------------------------------------------- host side

struct CrossPlan {
    int way;      // 0 CUDA cores, 1 tensor cores, 2 tensor cores with 16 rows a tile, 3 tensor cores, float32
    int parts;    // of the keys, in the workspace
    int cluster;  // way 2: blocks that join their keys in a cluster
    int runs;     // way 2, long rows: equal runs of all keys instead
};

constexpr int kAtOnce = 2 * 152;  // blocks of the 16-row kernels that run at once
constexpr int kLongRow = 1024;    // keys

// Parts of the keys for the kernels of 64 rows an item: several blocks an SM, of 128 keys or more (float32, 4096 x 4096 x 8
// heads: 1495 us in 2 parts, 1685 whole, 1488 in 4).
static int key_parts(int B, int N, int M, int G, int H, bool packed_q, bool packed_k) {
    const long long keys = packed_k ? (M + B - 1) / B : M, items = row_tiles(B, N, G, packed_q, kSimtRows) * H;
    return (int)std::max<long long>(1, std::min<long long>({8 * 152 / std::max(items, 1LL), (keys + 127) / 128, 64}));
}

// Which kernel, and how the keys are cut.  Only sizes that the host knows: a batch's average stands for its sequences.  The
// CUDA cores take the plan's cut where they stand in for its kernel (by BSA_FORCE_SIMT, or for strides and addresses), so
// that the workspace does not depend on that.
static CrossPlan cross_plan(bsa_dtype dtype, int B, int N, int M, int HQ, int H, int D, bool packed_q, bool packed_k) {
    CrossPlan p{};
    const int G = HQ / H, Gt = cross_tc_heads(G);
    const long long rows = (packed_q ? (N + B - 1) / B : (long long)N) * G;  // of a sequence and KV head, on average
    const long long keys = packed_k ? (M + B - 1) / B : M;
    const long long few = row_tiles(B, N, G, packed_q, 16) * H;              // items of 16 rows
    p.parts = p.cluster = 1;
    // Up to 16 rows the 16-row kernels.  Short rows, inputs in L2: 64 requests of 4 rows over 700 states 16 us against the
    // 256-row kernel's 23, 30 of 10 over 400 (D = 64) 7 against 15.  Long ones, L2 overwritten: 8 ragged requests of 1024 to
    // 32768 keys 100 against 185, since equal runs balance what whole items do not.  Where all lengths are the same the
    // 256-row kernel would be the faster (8 of 4096 keys 42 against 48, one of 131072 78 against 88), but the lengths are
    // on the device.  17 to 31 rows are two tiles, which read the keys twice: only for short rows whose blocks all run at
    // once (8 requests of 24 rows over 300 states 9 against 12; but 64 over 700 33 against 23, 8 over 4096 52 against 32).
    if (cross_tc_sizes(dtype, D) && (rows <= 16 || (rows < 32 && keys <= kLongRow && few <= kAtOnce))) {
        p.way = 2;
        // Clusters of blocks of 128 keys or more, no more blocks than run at once: 8 requests of 8 heads and 600 keys
        // take 16.5 us in clusters of 4 (L2 overwritten), 17.5 in 2, 19.6 alone, 23.7 in 8
        while (p.cluster < 8 && p.cluster * 128 < keys && 2 * p.cluster * few <= kAtOnce) p.cluster *= 2;
        // Long rows: equal runs of four 64-key chunks or more (the 8 ragged requests: 100 us, in clusters of 8 124, whole
        // 491); with rows enough to fill the card twice they are left whole (256 of 1500 keys x 16 heads, D = 64: 278 us
        // against 323)
        if (keys > kLongRow && few < 2 * kAtOnce)
            p.runs = (int)std::min<long long>((D <= 64 ? 3 : 2) * 152, std::max<long long>(1, few * keys / 256));
    } else if (cross_tc_sizes(dtype, D)) {
        p.way = 1;
        // as many parts as leave every SM an item, of two key tiles or more: more of them cost more to start and to join than
        // they balance (8 requests of 64 rows over 4096 states: 44 us with 2 parts, 47 with 4, 50 with 8, 54 whole)
        const long long items = row_tiles(B, N, Gt, packed_q, 256) * (HQ / Gt);
        p.parts = (int)std::max<long long>(1, std::min<long long>({152 / std::max(items, 1LL), (keys + 255) / 256, 64}));
    } else {
        p.way = dtype == BSA_F32 ? 3 : 0;
        p.parts = key_parts(B, N, M, G, H, packed_q, packed_k);
    }
    return p;
}

static bool cross_sizes_ok(int B, int N, int M, int HQ, int H, int D, bool packed_q) {
    if (B < 0 || N < 0 || M < 0 || HQ < 1 || H < 1 || HQ > 65535 || HQ % H || D < 1 || D > 128) return false;
    if (M > INT_MAX / 2) return false;  // a tile may end past the last state
    const long long rows = (packed_q ? 1LL : std::max(B, 1)) * (long long)N;  // and with the heads of a KV head
    return rows <= INT_MAX && rows * (HQ / H) <= INT_MAX / 2 && B <= INT_MAX / 2;
}

static size_t part_bytes(const CrossPlan& p, int B, int N, int HQ, int D, bool packed_q) {
    if (p.runs) return cross_runs_bytes(p.runs, D);
    return p.parts <= 1 ? 0 : sizeof(float) * (size_t)p.parts * (packed_q ? N : (size_t)B * N) * HQ * (D + 1);
}

template <typename T>
static bsa_status launch_cross_simt(const Cross& a, cudaStream_t st) {
    const size_t smem = simt_smem((a.D + 3) & ~3);
    const dim3 grid((unsigned)a.tiles, a.H, a.parts);
    auto fn = a.D <= 64 ? cross_simt_kernel<T, 1> : cross_simt_kernel<T, 2>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(BSA_ERR_CUDA, "cross attention attribute: %s", cudaGetErrorString(e));
    fn<<<grid, 256, smem, st>>>(a);
    return check_launch("cross_simt_kernel");
}

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsa_cross_workspace(bsa_dtype dtype, int B, int N, int M, int HQ, int H, int D, int packed_queries,
                           int packed_keys) {
    if ((dtype != BSA_F32 && dtype != BSA_BF16) || !cross_sizes_ok(B, N, M, HQ, H, D, packed_queries != 0) || B == 0 || N == 0) return 0;
    return part_bytes(cross_plan(dtype, B, N, M, HQ, H, D, packed_queries != 0, packed_keys != 0), B, N, HQ, D,
                      packed_queries != 0);
}

int bsa_cross_way(bsa_dtype dtype, int B, int N, int M, int HQ, int H, int D, int packed_queries, int packed_keys) {
    if ((dtype != BSA_F32 && dtype != BSA_BF16) || !cross_sizes_ok(B, N, M, HQ, H, D, packed_queries != 0) || B == 0 || N == 0) return -1;
    return force_simt() ? 0 : cross_plan(dtype, B, N, M, HQ, H, D, packed_queries != 0, packed_keys != 0).way;
}

bsa_status bsa_fwd_cross(const void* q, const void* k, const void* v, bsa_dtype dtype, int B, int N, int M, int HQ,
                         int H, int D, const int64_t* strides, const int32_t* query_start, const int32_t* key_start,
                         const int32_t* key_lens, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    BSA_REQUIRE(dtype == BSA_F32 || dtype == BSA_BF16, "cross attention: dtype");
    BSA_REQUIRE(cross_sizes_ok(B, N, M, HQ, H, D, query_start != nullptr), "cross attention: sizes out of range (B=%d N=%d M=%d HQ=%d H=%d D=%d)",
                B, N, M, HQ, H, D);
    BSA_REQUIRE(strides, "cross attention: null strides");
    BSA_REQUIRE(!(key_start && key_lens), "cross attention: key_start and key_lens exclude each other");
    BSA_REQUIRE(scale >= 0.f && scale <= 3.0e38f, "cross attention: the scale must be finite and not negative");
    if (B == 0 || N == 0) return BSA_OK;
    BSA_REQUIRE(q && out && (M == 0 || (k && v)), "cross attention: null pointer");
    const CrossPlan p = cross_plan(dtype, B, N, M, HQ, H, D, query_start != nullptr, key_start != nullptr);
    const size_t need = part_bytes(p, B, N, HQ, D, query_start != nullptr);
    BSA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && ((uintptr_t)workspace & 31) == 0),
                "cross attention: a 32-byte aligned workspace of %zu bytes is needed", need);
    Cross a{};
    a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse;
    long long* to[15] = {&a.qb, &a.qt, &a.qh, &a.kb, &a.kt, &a.kh, &a.vb, &a.vt, &a.vh, &a.ob, &a.ot, &a.oh, &a.lb, &a.lt, &a.lh};
    for (int i = 0; i < 15; ++i) *to[i] = strides[i];
    a.query_start = query_start, a.key_start = key_start, a.key_lens = key_lens;
    a.B = B, a.N = N, a.M = M, a.HQ = HQ, a.H = H, a.D = D, a.G = HQ / H;
    a.scale = scale;
    a.parts = p.parts;
    a.tiles = (int)row_tiles(B, N, a.G, query_start != nullptr, kSimtRows);
    a.status = status_word();
    const long long rows = (query_start ? (long long)N : (long long)B * N) * HQ;
    a.part_out = need ? static_cast<float*>(workspace) : nullptr;
    a.part_lse = need ? a.part_out + (p.runs ? (size_t)2 * p.runs * 16 : (size_t)p.parts * rows) * D : nullptr;
    cudaStream_t st = as_stream(stream);
    bsa_status rc = BSA_OK;
    bool handled = false;
    const int way = force_simt() ? 0 : p.way;
    if (way == 1) rc = cross_tc(a, st, &handled);
    if (way == 2) {
        Cross r = a;
        r.parts = p.cluster;
        rc = cross_rows(r, p.runs, st, &handled);
    }
    if (way == 3) rc = cross_f32(a, st), handled = true;
    if (!handled && p.runs) {
        // in place of the 16-row kernels: as many parts as the runs' workspace holds (at an odd address, one token
        // over 131072 states, 8 heads, D = 64: 0.8 ms in 64 parts, 18.6 whole)
        a.parts = (int)std::max<size_t>(1, std::min<size_t>(key_parts(B, N, M, a.G, H, query_start != nullptr, key_start != nullptr),
                                                            need / (sizeof(float) * (D + 1) * rows)));
        a.part_lse = a.part_out + (size_t)a.parts * rows * D;
    }
    if (!handled && rc == BSA_OK)
        rc = dtype == BSA_F32 ? launch_cross_simt<float>(a, st) : launch_cross_simt<__nv_bfloat16>(a, st);
    if (rc != BSA_OK || a.parts == 1) return rc;  // runs join by themselves
    const dim3 grid((unsigned)row_tiles(B, N, a.G, query_start != nullptr, kJoinRows), H);
    if (dtype == BSA_F32) cross_join_kernel<float><<<grid, 32 * kJoinRows, 0, st>>>(a);
    else cross_join_kernel<__nv_bfloat16><<<grid, 32 * kJoinRows, 0, st>>>(a);
    return check_launch("cross_join_kernel");
}

}  // extern "C"
