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
// 8 ragged requests of 1024 to 32768 keys, 32 heads over 8, D = 128: 554 MB in 105 to 108 us, 76 to 78% of the copy rate; a warp waits for
// its reads most of the time, and 254 registers leave two blocks an SM.
// The four warps of a block join their parts of the keys in shared memory.  Short rows: a cluster of up to 8 blocks an
// item, which read each other's shared memory (one launch).  Long ones: equal runs and a join.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>

#include "cross.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace cross {

namespace cg = cooperative_groups;

constexpr int kRowTile = 16, kStep = 16, kWarps = 4;
constexpr int kChunk = kStep * kWarps;
// The tensor cores cut off what they add to a sum, which over values of one sign does not average out (outputs between 1 and 2
// over 2^21 keys, 2^19 a warp, were 6e-3 off, 4e-3 of it the output's rounding): every so many steps a warp puts its sums
// aside, into the shared memory that they are joined in, and those are added up rounded.
constexpr int kAside = 1024;
constexpr float kGrow = 8.f;  // log2 units: the running maximum is raised, and O rescaled, only when it grows by more

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 read16(const __nv_bfloat16* p, bool on) {
    return on ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// Key tiles [t0, t1) of 16 keys of sequence b and KV head h against the rows from row0: every warp's part of the
// output, the maxima and the sums into shared memory (so: [kWarps][16][HD], sm: [kWarps][16] maxima, then sums).
template <int HD>  // 64 or 128: channels, padded with zeros
__device__ __forceinline__ void walk_keys(const Cross& a, int b, int h, int row0, int rows, int q0, int k0, int m, int t0, int t1,
                                          float* so, float* sm) {
    constexpr int kC = HD / 32, kV = HD / 64;  // 16-byte runs of K and of V a lane reads of a key
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
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

    int t = t0 + warp;
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
    bool first = true;  // nothing put aside
    for (int stop = min(t1, t0 + kAside * kWarps);; stop = min(t1, stop + kAside * kWarps)) {
        for (; t < stop; t += kWarps) {
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
            const int row = warp * kRowTile + g + 8 * r;
            const float was = first ? -CUDART_INF_F : sm[row], f = was == -CUDART_INF_F ? 0.f : ptx::ex2(was - ref[r]);
            __syncwarp();  // all have read what c = 0 writes
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            float* to = so + row * HD;
#pragma unroll
            for (int i = 0; i < kV; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        float4& at = *reinterpret_cast<float4*>(to + 64 * i + 8 * (2 * c + e) + j);
                        const float4 x = first ? make_float4(0.f, 0.f, 0.f, 0.f) : at;
                        at = make_float4(fmaf(x.x, f, o[8 * i + j][2 * r + e]), fmaf(x.y, f, o[8 * i + j + 1][2 * r + e]),
                                         fmaf(x.z, f, o[8 * i + j + 2][2 * r + e]), fmaf(x.w, f, o[8 * i + j + 3][2 * r + e]));
                    }
            if (c == 0) {
                sm[row] = ref[r];
                sm[kWarps * kRowTile + row] = first ? l[r] : fmaf(sm[kWarps * kRowTile + row], f, l[r]);
            }
            l[r] = 0.f;
        }
        if (t >= t1) break;
        first = false;
#pragma unroll
        for (int j = 0; j < 8 * kV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        __syncwarp();
    }
}

// Where row r of an item goes: the output, or (to a part's results) float32 and its log-sum-exp.  Four channels a thread.
__device__ __forceinline__ void write_row(const Cross& a, int b, int h, int rr, int q0, int ch, const float* y, float lse,
                                          long long part_row) {
    const long long qbat = a.query_start ? 0 : b;
    const int tok = q0 + rr / a.G, hq = h * a.G + rr % a.G;
    if (part_row >= 0) {
        if (ch < a.D) *reinterpret_cast<float4*>(a.part_out + part_row * a.D + ch) = make_float4(y[0], y[1], y[2], y[3]);
        if (ch == 0) a.part_lse[part_row] = lse;
    } else {
        if (ch < a.D)
            *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + qbat * a.ob + tok * a.ot + hq * a.oh + ch) =
                make_uint2(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]));
        if (ch == 0 && a.lse) a.lse[qbat * a.lb + tok * a.lt + hq * a.lh] = lse;
    }
}

// One row of one block's warps, added to (top's scale) sum and y.
template <int HD>
__device__ __forceinline__ void add_warps(const float* so, const float* sm, int r, int ch, float base, float& sum, float* y) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = ptx::ex2(sm[w * kRowTile + r] - base);
        sum = fmaf(sm[(kWarps + w) * kRowTile + r], f, sum);
        const float4 z = *reinterpret_cast<const float4*>(so + (w * kRowTile + r) * HD + ch);
        y[0] = fmaf(z.x, f, y[0]), y[1] = fmaf(z.y, f, y[1]), y[2] = fmaf(z.z, f, y[2]), y[3] = fmaf(z.w, f, y[3]);
    }
}
__device__ __forceinline__ void normalise(float top, float sum, float* y, float& lse) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    lse = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
}

// One item a cluster: its blocks take parts of the keys and finish a share of the rows each.
template <int HD>
__global__ void __launch_bounds__(32 * kWarps, 2) cross_rows_kernel(const Cross a) {
    extern __shared__ __align__(16) float rows_smem[];
    float *so = rows_smem, *sm = so + kWarps * kRowTile * HD;
    const int h = blockIdx.y, part = blockIdx.z;
    int b, row0, q0, n, k0, m;
    tile_of<kRowTile>(a, blockIdx.x, b, row0);
    if (b < 0) return;  // the whole cluster
    queries_of(a, b, q0, n);
    keys_of(a, b, k0, m);
    const int rows = (int)min((long long)kRowTile, (long long)n * a.G - row0), nt = (m + kStep - 1) / kStep;
    walk_keys<HD>(a, b, h, row0, rows, q0, k0, m, (int)((long long)nt * part / a.parts),
                  (int)((long long)nt * (part + 1) / a.parts), so, sm);
    auto cluster = cg::this_cluster();
    const int peers = cluster.num_blocks(), rank = cluster.block_rank();
    if (peers > 1) cluster.sync();
    else __syncthreads();
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
        float sum = 0.f, y[4] = {}, lse;
        for (int x = 0; x < peers; ++x)
            add_warps<HD>(peers > 1 ? cluster.map_shared_rank(so, x) : so, peers > 1 ? cluster.map_shared_rank(sm, x) : sm, r,
                          ch, base, sum, y);
        normalise(top, sum, y, lse);
        write_row(a, b, h, row0 + r, q0, ch, y, lse, -1);
    }
    if (peers > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

// ---------------------------------------------------------------- long rows: equal runs
//
// Every block takes an equal run of all items' 64-key chunks, in order of sequence, KV head, row tile and key, so that
// ragged lengths balance themselves.  An item that lies in one run is finished there; of one that is cut every run
// leaves its part in one of its two slots (0: the run's first segment, 1: its last), and the join finds them again from
// the same counts.
__device__ __forceinline__ long long chunks_of(const Cross& a, int b, int& tiles, int& per) {
    int q0, n, k0, m;
    queries_of(a, b, q0, n);
    keys_of(a, b, k0, m);
    tiles = (int)(((long long)n * a.G + kRowTile - 1) / kRowTile);
    per = max(1, (m + kChunk - 1) / kChunk);  // a sequence without keys is written too
    return (long long)tiles * per * a.H;
}
// The sequence that holds chunk `at` and the chunks before that sequence, or the chunks of all for at < 0; by a warp.
__device__ __forceinline__ long long find_chunk(const Cross& a, long long at, int& b) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    b = -1;
    for (int base = 0; base < a.B; base += 32) {
        int tiles, per;
        long long sum = base + lane < a.B ? chunks_of(a, base + lane, tiles, per) : 0;
        const long long own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at >= 0 && before + sum > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = base + l;
            return before + __shfl_sync(0xffffffffu, sum - own, l);
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return before;
}

template <int HD>
__global__ void __launch_bounds__(32 * kWarps, 2) cross_runs_kernel(const Cross a) {
    extern __shared__ __align__(16) float rows_smem[];
    float *so = rows_smem, *sm = so + kWarps * kRowTile * HD;
    int b;
    const long long all = find_chunk(a, -1, b);
    const long long runs = min((long long)gridDim.x, all);  // none is empty
    if (blockIdx.x >= runs) return;
    long long at = all * blockIdx.x / runs;
    const long long end = all * (blockIdx.x + 1) / runs, begin = at;
    long long before = find_chunk(a, at, b);
    while (at < end) {
        int tiles, per, q0, n, k0, m;
        const long long size = chunks_of(a, b, tiles, per);
        if (at >= before + size) {  // the next sequence
            before += size;
            ++b;
            continue;
        }
        queries_of(a, b, q0, n);
        keys_of(a, b, k0, m);
        const long long in = at - before, item = in / per;
        const int chunk = (int)(in - item * per), h = (int)(item / tiles), row0 = (int)(item - (long long)h * tiles) * kRowTile;
        const int take = (int)min((long long)(per - chunk), end - at);
        const int rows = (int)min((long long)kRowTile, (long long)n * a.G - row0), nt = (m + kStep - 1) / kStep;
        walk_keys<HD>(a, b, h, row0, rows, q0, k0, m, chunk * (kChunk / kStep), min(nt, (chunk + take) * (kChunk / kStep)), so, sm);
        __syncthreads();
        const long long slot = take == per ? -1 : 2 * (long long)blockIdx.x + (at != begin);
        constexpr int kQuads = HD / 4;
        for (int i = threadIdx.x; i < kRowTile * kQuads; i += 32 * kWarps) {
            const int r = i / kQuads, ch = i % kQuads * 4;
            if (r >= rows) break;
            float top = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * kRowTile + r]);
            float sum = 0.f, y[4] = {}, lse;
            add_warps<HD>(so, sm, r, ch, top == -CUDART_INF_F ? 0.f : top, sum, y);
            normalise(top, sum, y, lse);
            write_row(a, b, h, row0 + r, q0, ch, y, lse, slot < 0 ? -1 : slot * kRowTile + r);
        }
        __syncthreads();
        at += take;
    }
}

// Four rows of an item a block: the parts that runs left of it, in order.
template <int HD>
__global__ void __launch_bounds__(4 * HD / 4) cross_runs_join_kernel(const Cross a, int blocks) {
    const int h = blockIdx.y, lane = threadIdx.x & 31;
    int b, row0, q0, n, none;
    const long long all = find_chunk(a, -1, none), runs = min((long long)blocks, all);
    tile_of<kRowTile>(a, blockIdx.x, b, row0);
    if (b < 0) return;
    queries_of(a, b, q0, n);
    int tiles, per;
    chunks_of(a, b, tiles, per);
    long long before = 0;  // chunks of the sequences before b
    for (int base = 0; base < b; base += 32) {
        int x, y;
        long long sum = base + lane < b ? chunks_of(a, base + lane, x, y) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        before += sum;
    }
    const long long first = before + ((long long)h * tiles + row0 / kRowTile) * per, last = first + per - 1;
    // run i holds the chunks [all i / runs, all (i + 1) / runs)
    const int i0 = (int)(((first + 1) * runs - 1) / all), i1 = (int)(((last + 1) * runs - 1) / all);
    if (i0 == i1) return;  // finished by its run
    const int r = blockIdx.z * 4 + threadIdx.x / (HD / 4), ch = threadIdx.x % (HD / 4) * 4;
    if (r >= min((long long)kRowTile, (long long)n * a.G - row0)) return;
    // rows of the parts: the first run's last slot unless it begins with this item, the others' first
    const long long lead = (2LL * i0 + (all * i0 / runs != first)) * kRowTile + r, next = (2LL * i0 + 2) * kRowTile + r;
    const int parts = i1 - i0 + 1;
    auto row_of = [&](int x) { return x == 0 ? lead : next + (long long)(x - 1) * 2 * kRowTile; };
    float top = -CUDART_INF_F;
#pragma unroll 8
    for (int x = 0; x < parts; ++x) top = fmaxf(top, a.part_lse[row_of(x)]);
    const float base = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f, y[4] = {};
#pragma unroll 8
    for (int x = 0; x < parts; ++x) {
        const long long row = row_of(x);
        const float w = exp2f((a.part_lse[row] - base) * kLog2e);
        const float4 z = ch < a.D ? *reinterpret_cast<const float4*>(a.part_out + row * a.D + ch) : make_float4(0.f, 0.f, 0.f, 0.f);
        sum += w;
        y[0] = fmaf(w, z.x, y[0]), y[1] = fmaf(w, z.y, y[1]), y[2] = fmaf(w, z.z, y[2]), y[3] = fmaf(w, z.w, y[3]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
    write_row(a, b, h, row0 + r, q0, ch, y, sum == 0.f ? -CUDART_INF_F : top + log2f(sum) * kLn2, -1);
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

template <int HD>
static bsa_status launch_runs(const Cross& a, int tiles, int runs, cudaStream_t st) {
    constexpr int kSmem = sizeof(float) * (kWarps * kRowTile * HD + 2 * kWarps * kRowTile);
    cross_runs_kernel<HD><<<runs, 32 * kWarps, kSmem, st>>>(a);
    bsa_status rc = check_launch("cross_runs_kernel");
    if (rc != BSA_OK) return rc;
    cross_runs_join_kernel<HD><<<dim3(tiles, a.H, kRowTile / 4), HD, 0, st>>>(a, runs);
    return check_launch("cross_runs_join_kernel");
}

}  // namespace cross

size_t cross_runs_bytes(int runs, int D) { return sizeof(float) * (size_t)2 * runs * cross::kRowTile * (D + 1); }

// runs > 0: equal runs of all keys, and a join; otherwise one cluster of a.parts blocks an item.
bsa_status cross_rows(const Cross& a, int runs, cudaStream_t st, bool* handled) {
    *handled = false;
    const long long tiles = row_tiles(a.B, a.N, a.G, a.query_start != nullptr, cross::kRowTile);
    uintptr_t any = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.out;
    for (long long s : {a.qb, a.qt, a.qh, a.kb, a.kt, a.kh, a.vb, a.vt, a.vh, a.ob, a.ot, a.oh}) any |= (uintptr_t)(2 * s);
    if ((any & 15) || a.M == 0 || a.H > 65535 || tiles > 0x7fffffffLL) return BSA_OK;
    *handled = true;
    if (runs) return a.D <= 64 ? cross::launch_runs<64>(a, (int)tiles, runs, st) : cross::launch_runs<128>(a, (int)tiles, runs, st);
    return a.D <= 64 ? cross::launch_rows<64>(a, (int)tiles, a.parts, st) : cross::launch_rows<128>(a, (int)tiles, a.parts, st);
}

}  // namespace bsa
