// Attention over the 4-bit paged cache (a14) on the tensor cores, D = 64 or 128.
//
// A row is one token's up to 16 query heads of one KV head.  Its strips (16 keys each, one
// contiguous run of 18 D bytes) are taken in tiles of up to four.  Every warp works alone: it
// copies its tiles into a ring of its own (one bulk copy per strip), keeps its own running
// maximum, sum and output, and goes on to its next row without waiting for anyone, the first
// tiles of which are in flight by then.  Which tiles a warp takes:
//   stream  two or three CTAs of four warps an SM, every warp an equal run of the rows' tiles laid end to
//           end (so a batch of ragged lengths is balanced to a tile); a row that is cut leaves
//           parts (m, l, U) in the workspace, and a second kernel joins them:
//             m = max m_i,   l = sum l_i 2^(m_i - m),   U = sum U_i 2^(m_i - m),   O = U / l;
//   units   many rows of about the same length, two CTAs an SM: clusters of these two share out the rows,
//           whole, and the warps of a cluster its tiles; a cut row is joined inside its cluster, in one launch;
//   rows    so many rows that whole ones balance: each warp takes the next row when it is done with one (from the
//           stream's work counter; in a captured graph every warps-th row);
//   split   so few tiles that one launch counts: a cluster of up to 8 CTAs per row, joined through
//           shared and distributed shared memory.
//
// Numbers.  code * scale is exact in float16, so K and V enter the products exactly.  A
// row of q is scaled by the power of two that brings its largest magnitude to 2^14..2^15
// and is then exact in float16 when it is bf16 (8 bits, over 28 binades); a float32 q is
// split into two float16 parts.  Weights are held as 2^11 2^(logit - reference), the reference at
// most 2^4 below the running maximum (the sums and the output are rescaled only when the maximum
// grows by more than that): they stay below float16's 2^16 and keep full precision over 25
// binades.  They are rounded to float16 for bf16 outputs, u = 2^-11 against the output's own
// 2^-8 (a second product for the rest would cost what float32 outputs pay: 64 us for 24 requests of 8192
// keys, against 40), or split in two for float32 ones.  The rows' sums take them unrounded, since the LSE is
// float32 from them.  Maxima, sums and both accumulators are float32.
//
// Fragments.  mma.m16n8k16 lets the summed index be permuted freely as long as both
// operands agree, so a lane takes what lies together: of K the D / 4 consecutive channels
// of one key (one 16-byte load at D = 128), of V the D / 8 consecutive channels of four keys.
// Codes become float16 with cvt (two per byte) and one multiplication by their scales;
// V's codes are first paired along the keys, four logic instructions per 16 codes.
// No converted value is ever written back to shared memory.  With more than 8 heads q and the
// weights are the 16-row operand; with up to 8 (kNarrow) K and V are, q and the weights the
// 8-column one (transposed in registers by movmatrix), which halves the products and the output's
// registers.
//
// What bounds it.  mma.sync keeps a scheduler for about 8 cycles, during which
// little else issues (measured: 32 mma with 64 cvt and 64 multiplications take 2 cycles per mma
// plus 1/4 per other instruction on an SM, whether 8 or 16 warps run), so a tile of 64 keys at
// D = 128 costs 256 + 970 / 4 = 498 cycles wide; its bytes take 400 at the measured copy bandwidth.  It
// takes about 620: a scheduler has two warps, and both mostly wait for results of their own (profiled:
// 42 to 47% of the issue slots used, 0.5 to 0.6 warps ready a cycle, 1.2 cycles an instruction waiting for the one
// before it, 0.5 for the tensor pipe, 0.2 to 0.4 for memory).  Narrow it is 128 + 860 / 4, and the bytes bind.
// Measured on the device: 48 ragged requests, 909 MB, 8 heads a KV head: 161 us, 84% of the copy bandwidth; 256
// tokens of 2048 selected keys, 301 MB, 16 heads: 82 us, 54%.  About 7 us of a launch pass before the first tile
// is worked on (start of the run, lookups, first copies), part of them for fetching instructions:
// a kernel for each of the four ways instead of one with branches took 1 to 4 us less (31.2 -> 30.5 us
// for one request of 131072 keys, 9.0 -> 8.5 us for 8 short ones).
//
// Tried and slower: a copying warp for four others (five warps a CTA limit registers to 168);
// three CTAs an SM wide (168 registers, 15% more instructions); codes to float16 by shifts and masks (5.7
// against 3.1 cycles per 8 codes and warp).
#pragma once

#include <algorithm>
#include <atomic>

#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace cmma {

constexpr int kWarps = 4;    // of a CTA
constexpr int kTile = 4;     // strips of a tile, at most
constexpr uint64_t kWaitNs = 500ull * 1000 * 1000;
constexpr float kWeightLog2 = 11.f;  // weights are held 2^11 times, relative to a reference
constexpr float kSlack = 4.f;        // that the running maximum may pass by 2^4 before it is moved
// The tensor cores cut sums off rather than round them, each time by up to a step of the running sum, so a run of n
// keys brings values of one sign out short by about 6e-9 n: 8e-4 of them at 131072 keys, 3e-3 at half a million.  bf16
// outputs therefore put their sums aside every so many tiles, where they are added up rounded to nearest (float32 ones
// add every strip so): 5e-5 short at most, an eightieth of the output's own rounding.  Measured, us, without, with 256,
// 128 and 64 tiles: 300 requests of 32768 keys, 16 heads on each of 4, 1161, 1166, 1171, 1176; 8 on 8, 1708, 1735,
// 1742, 1753.
constexpr int kAside = 128;

enum Mode { kSplit, kStream, kUnits, kRows };

struct Plan {
    int head_tiles;   // tiles of 16 query heads per KV head
    int tile_strips;  // strips of a tile, at most kTile
    int tile_log2;
    int splits;       // kSplit: CTAs of a row (the cluster)
    int G;            // query heads per KV head
    unsigned long long inv_H;  // ceil(2^32 / H): g / H = g * inv_H >> 32 for g * H below 2^32
    int unit;         // kUnits: CTAs of a unit (their cluster)
    int rows;
    int warps;        // of the grid
    unsigned* work;   // kRows: (rows claimed behind the first ones, warps done), zero between launches, or null
    int stall;        // tests only: a tile of each warp that is never copied (-1: none), waits end after 1 ms
    float* part;      // kStream, kUnits: [warps][2][rows of U][D], slot 0 a row carried on, slot 1 a row begun
    float2* ml;       // [warps][2][rows of U]
    int2* begun;      // [rows] the warp that began a cut row and in how many parts it is (0: whole)
    float* aside;     // [warps][rows of U][D] sums of runs longer than kAside tiles, or null: no row has as many
};

// ---------------------------------------------------------------- pieces

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_zero(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// d += a b + a2 b2, the products summed first.
__device__ __forceinline__ void add_products(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const uint32_t* a2,
                                             uint32_t c0, uint32_t c1) {
    float e[4];
    mma_zero(e, a2, c0, c1);
    mma(e, a, b0, b1);
    const float2 lo = ptx::fadd2(make_float2(d[0], d[1]), make_float2(e[0], e[1]));
    const float2 hi = ptx::fadd2(make_float2(d[2], d[3]), make_float2(e[2], e[3]));
    d[0] = lo.x, d[1] = lo.y, d[2] = hi.x, d[3] = hi.y;
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
template <typename V> __device__ __forceinline__ V lds(const unsigned char* p) { return *reinterpret_cast<const V*>(p); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <int N> __device__ __forceinline__ void bar_sync(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
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

// Waits for a phase; after kWaitNs (1 ms in the test of this) latches BSA_ERR_TIMEOUT and gives up.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, int* status, int stall) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > (stall >= 0 ? 1000000ull : kWaitNs)) {
            raise_status(status, BSA_ERR_TIMEOUT);
            return false;
        }
    return true;
}

// ---------------------------------------------------------------- shapes

template <int D, typename T, bool kNarrow>
struct Shape {
    static constexpr int kTerms = sizeof(T) == 2 ? 1 : 2;  // float16 parts of q and of the weights
    static constexpr int kThreads = kWarps * 32;
    // CTAs of an SM and tiles of a warp's ring: what registers and shared memory hold
    static constexpr int kBlocks = kNarrow && kTerms == 1 ? 3 : 2, kStages = kBlocks == 3 ? 2 : 3;
    static constexpr int kRows = kNarrow ? 8 : 16;
    static constexpr int kStripB = strip_bytes(D);
    static constexpr int kTileB = kTile * kStripB;
    // kSplit: U of each warp over the ring, rows padded so that a quarter warp's 16-byte stores meet no bank twice
    static constexpr int kRowF = D + 16;
    static constexpr int kRing = kWarps * kStages * kTileB, kU = kWarps * kRows * kRowF * 4;
    static constexpr int kML = kRing > kU ? kRing : kU;           // (m, l) of each warp and row
    static constexpr int kCML = kML + kWarps * kRows * 8;         // the CTA's
    static constexpr int kMeta = kCML + kRows * 8;                // of each tile of the ring: 8 ints
    static constexpr int kFull = kMeta + kWarps * kStages * 32;
    static constexpr int kBytes = kFull + kWarps * kStages * 8;
    static __device__ __forceinline__ int at(int row, int ch) { return row * kRowF + ch + ch / (D / 4) * 4; }
};

// Row number -> token, KV head, head tile and the walk over its keys.
struct Where {
    int t, h, heads, hq0;
};
__device__ __forceinline__ Where where(const CacheAttn& a, const Plan& p, int r) {
    Where w;
    unsigned tile_h = 0, th = r;
    if (p.head_tiles > 1) th = (unsigned)r / (unsigned)p.head_tiles, tile_h = r - th * p.head_tiles;
    w.t = th / (unsigned)a.H;
    w.h = th - w.t * a.H;
    w.heads = min(16, p.G - (int)tile_h * 16);
    w.hq0 = w.h * p.G + tile_h * 16;
    return w;
}
// A row without keys still has an output to write (one empty tile); a padding row has none.
__device__ __forceinline__ int tiles_of(const Row& r, const Plan& p) {
    return r.req < 0 ? 0 : max(1, (r.strips + p.tile_strips - 1) >> p.tile_log2);
}

// Flags of a tile.
constexpr int kBegin = 1, kEnd = 2, kCarried = 4, kCut = 8;
constexpr int kPut = 16, kHeld = 32;  // the row's sums are put aside behind this tile; they were behind an earlier one

// The tiles of a warp, looked up eight at a time (lane 4 i + j: strip j of the batch's tile i), a
// batch ahead of the first copy that needs it.
struct Ahead {
    bool have = false;
    int next_row = 0, first_tile = 0;  // the row after the current one; where the run begins in its first row
    int left = 0;                      // tiles behind the current row's (kRows: 1)
    unsigned claim = 0;                // kRows, lane 0: the row claimed for later
    // the current row: tiles [lo, hi) of n are the warp's, the batch is [off, off + size), the tile held off + at
    int row = 0, lo = 0, hi = 0, n = 0, off = 0, size = 0, at = 0;
    bool opened = false;               // kStream, kUnits: the row begins here
    Row r;
    int h = 0;
    int first = -1, page = 0;  // the lane's strip: its first key (-1: none to see), its page as the table has it

    template <Mode M>
    __device__ __forceinline__ void next(const CacheAttn& a, const Plan& p, int lane, int elem) {
        have = false;
        if (++at < size) {
            have = true;
            return;
        }
        off += size, size = 0;
        while (off == hi) {
            if (left <= 0 || next_row >= p.rows) return;
            row = next_row++;
            if constexpr (M == kRows) {  // the claim made at the last row becomes the next one
                next_row = p.work ? p.warps + (int)__shfl_sync(0xffffffffu, claim, 0) : row + p.warps;
                if (p.work && lane == 0 && next_row < p.rows) claim = atomicAdd(p.work, 1u);
            }
            const Where w = where(a, p, row);
            h = w.h;
            r = row_of(a, w.t, w.h, lane == 0);
            n = tiles_of(r, p);
            lo = off = min(n, first_tile);
            first_tile = 0;
            // the row's queries are needed a few tiles from now
            const char* q = static_cast<const char*>(a.q) + ((long long)w.t * a.q_stride + (long long)w.hq0 * a.D) * elem;
            for (int i = lane * 128; i < w.heads * a.D * elem; i += 32 * 128)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
            if constexpr (M == kRows) {
                hi = n;
            } else {
                hi = min(n, off + left);
                left -= hi - off;
                opened = opened || (lo == 0 && hi > 0);
            }
        }
        size = min(8, hi - off), at = 0;
        have = true;
        const int tile = off + (lane >> 2), s = tile * p.tile_strips + (lane & 3);
        first = -1;
        if ((lane & 3) < p.tile_strips && tile < hi && s < r.strips) {
            first = first_key(a, r, s, true);
            if (first >= 0) page = a.table[(long long)r.req * a.max_pages + (first >> a.sh)];
        }
    }
    template <bool kPuts>
    __device__ __forceinline__ int flags() const {
        const int t = off + at;
        int f = (t == lo ? kBegin : 0) | (t == hi - 1 ? kEnd : 0) | (lo > 0 ? kCarried : 0) | (lo > 0 || hi < n ? kCut : 0);
        if constexpr (kPuts)
            if (t - lo >= kAside - 1) f |= ((t - lo) % kAside == kAside - 1 && t < hi - 1 ? kPut : 0) | (t - lo >= kAside ? kHeld : 0);
        return f;
    }
};

// kStream, kUnits: where each warp's run begins and how long it is.  The tiles of a group of rows that
// share their keys' number are counted once: a token's without lists, a (token, head)'s with.
constexpr int kScanGroups = 8192;
// The row that holds tile x, the tile of the row it is, and the row's tiles: the warp cuts the groups in 32 until one
// is left.  One copy of it: a launch's first microseconds go into fetching its instructions.
static __device__ __noinline__ int3 find_tile(const int* sums, int groups, int mult, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = groups;  // the first group that ends behind x is in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 31) >> 5, at = lo + lane * step, end = min(at + step, lo + len);
        const uint32_t behind = __ballot_sync(0xffffffffu, at < lo + len && sums[max(end, 1) - 1] * mult > x);
        const int pick = lo + (__ffs(behind) - 1) * step;
        len = min(step, lo + len - pick);
        lo = pick;
    }
    const int before = lo ? sums[lo - 1] : 0, in = x - before * mult, n = sums[lo] - before;
    const int whole = (unsigned)in / (unsigned)n;
    return make_int3(lo * mult + whole, in - whole * n, n);
}
template <Mode M>
__device__ __forceinline__ void find_start(const CacheAttn& a, const Plan& p, int* sums, int warps, int id, Ahead& ahead,
                                           int& base, int& total, int& run_hi) {
    __shared__ int part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mult = a.blocks ? p.head_tiles : a.H * p.head_tiles, groups = p.rows / mult;
    int all = 0;
    for (int g0 = 0; g0 < groups; g0 += 8 * kWarps * 32) {  // eight consecutive groups a thread
        int v[8], req[8], pos[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = min(g0 + tid * 8 + i, groups - 1), t = a.blocks ? (int)(g * p.inv_H >> 32) : g;
            req[i] = a.req[t], pos[i] = a.pos[t];
            v[i] = a.blocks ? a.counts[g] : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = g0 + tid * 8 + i < groups ? tiles_of(row_from(a, req[i], pos[i], v[i], blockIdx.x == 0), p) : 0;
            if (i) v[i] += v[i - 1];
        }
        int inc = v[7];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        if (lane == 31) part[warp] = inc;
        __syncthreads();
        int before = all + inc - v[7];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) before += part[k];
            all += part[k];
        }
        int4* to = reinterpret_cast<int4*>(sums + g0 + tid * 8);
        to[0] = make_int4(before + v[0], before + v[1], before + v[2], before + v[3]);
        to[1] = make_int4(before + v[4], before + v[5], before + v[6], before + v[7]);
        __syncthreads();
    }
    total = all * mult;  // below 2^31: checked by the host
    auto find = [&](int x, int& row, int& tile, int& n) {
        const int3 f = find_tile(sums, groups, mult, x);
        row = f.x, tile = f.y, n = f.z;
    };
    base = 0;
    if constexpr (M == kUnits) {  // the unit's share begins and ends with the row that begins at or behind an equal cut
        const int units = gridDim.x / p.unit, u = blockIdx.x / p.unit;
        int ends[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ends[k] = (int)((long long)total * (u + k) / units);
            int row, tile, n;
            if (ends[k] < total) {
                find(ends[k], row, tile, n);
                if (tile) ends[k] += n - tile;
            }
        }
        base = ends[0], total = ends[1] - ends[0];
    }
    // total id / warps in 32 bits: total = q warps + rest
    const unsigned q = (unsigned)total / (unsigned)warps, rest = (unsigned)total - q * warps;
    const unsigned run_lo = base + q * id + rest * id / warps;
    run_hi = base + q * (id + 1) + rest * (id + 1) / warps;
    ahead.left = run_hi - run_lo;
    int n;
    if (ahead.left > 0) find(run_lo, ahead.next_row, ahead.first_tile, n);
    // the sums lie in the ring: everyone has read them before the first copy lands there
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
}

// ---------------------------------------------------------------- a warp's part of a row

template <int D, typename T, bool kNarrow>
struct Part {
    using S = Shape<D, T, kNarrow>;
    static constexpr int kTerms = S::kTerms;
    static constexpr int kSteps = D / 16;             // k-steps of q K^T
    static constexpr int kCh = D / 8;                 // channels of a lane's V fragment
    static constexpr int kQ = kNarrow ? 2 : 4;        // registers of q per k-step
    static constexpr int kU = kNarrow ? kCh / 2 : kCh;  // accumulator tiles of U

    // Two "rows" (query heads) per lane: wide g and g + 8, narrow 2 c and 2 c + 1.
    uint32_t q[kTerms][kSteps][kQ];
    float rs[2], m[2], u[kU][4];
    float2 l[2];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int r = 0; r < 2; ++r) m[r] = -INFINITY, l[r] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kU; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[j][i] = 0.f;
    }

    // The lane's queries as they lie in memory, channels c D/4 .. of rows g (and g + 8): fetched ahead of their use.
    static constexpr int kHalves = kNarrow ? 1 : 2, kRaw = D / 4 * sizeof(T) / 4;
    struct Raw {
        uint32_t w[kHalves][kRaw];
        float ks;
    };
    static __device__ __forceinline__ void fetch_q(Raw& raw, const CacheAttn& a, const Plan& p, int row, int g, int c) {
        const Where w = where(a, p, row);
        const T* base = static_cast<const T*>(a.q) + w.t * a.q_stride + (long long)w.hq0 * D + c * (D / 4);
        const bool wide = (((uintptr_t)a.q | (uintptr_t)(a.q_stride * (long long)sizeof(T))) & 15) == 0;
        raw.ks = (a.k_scale ? a.k_scale[w.h] : 1.f) * a.scale_log2;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            const int r = min(g + half * 8, w.heads - 1);  // rows behind the last head repeat it and are not written
            const T* src = base + (long long)r * D;
            if (wide) {
#pragma unroll
                for (int i = 0; i < kRaw / 4; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
                    raw.w[half][4 * i] = v.x, raw.w[half][4 * i + 1] = v.y;
                    raw.w[half][4 * i + 2] = v.z, raw.w[half][4 * i + 3] = v.w;
                }
            } else if constexpr (sizeof(T) == 2) {
                const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
                for (int i = 0; i < kRaw; ++i) raw.w[half][i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
            } else {
#pragma unroll
                for (int i = 0; i < kRaw; ++i) raw.w[half][i] = __float_as_uint(to_f32(src[i]));
            }
        }
    }
    // Each row scaled to 2^14 .. 2^15 and rounded to (or split into) float16.
    __device__ __forceinline__ void convert_q(const Raw& raw, int c) {
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            float top = 0.f;
            if constexpr (sizeof(T) == 2) {
                // magnitudes of bf16 order as integers do; NaN is above infinity
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < kRaw; ++i) most = __vmaxu2(most, raw.w[half][i] & 0x7fff7fffu);
                top = __uint_as_float(max(most << 16, most & 0xffff0000u));
            } else {
#pragma unroll
                for (int i = 0; i < kRaw; ++i) top = fmaxf(top, fabsf(__uint_as_float(raw.w[half][i])));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - floor(log2 top)), its exponent kept in range; zero, infinite and NaN rows stay as they
            // are.  The sign of the logits' factor goes into q, so that rs is positive; at least the
            // smallest normal, so that a scale of zero leaves masked logits at -inf.
            const int e = (int)(__float_as_uint(top) >> 23);
            const int up = e == 0 || e == 255 ? 0 : min(126, 14 + 127 - e);
            const float f = copysignf(__uint_as_float((uint32_t)(127 + up) << 23), raw.ks);
            const float size = fabsf(raw.ks) * __uint_as_float((uint32_t)(127 - up) << 23);
            rs[half] = size < 1.17549435e-38f ? 1.17549435e-38f : size;  // a NaN stays one
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int at = kNarrow ? e2 : half + 2 * e2, i = 4 * s + 2 * e2;
                    float x0, x1;
                    if constexpr (sizeof(T) == 2) {
                        const uint32_t w = raw.w[half][i / 2];
                        x0 = __uint_as_float(w << 16) * f, x1 = __uint_as_float(w & 0xffff0000u) * f;
                    } else {
                        x0 = __uint_as_float(raw.w[half][i]) * f, x1 = __uint_as_float(raw.w[half][i + 1]) * f;
                    }
                    q[0][s][at] = pack_f16x2(x0, x1);
                    if constexpr (kTerms == 2) {
                        const float2 b = f16x2_to_f32(q[0][s][at]);
                        q[1][s][at] = pack_f16x2(x0 - b.x, x1 - b.y);
                    }
                }
        }
        if constexpr (kNarrow) {  // the lane's logits are those of heads 2 c and 2 c + 1
            const float mine = rs[0];
            rs[0] = __shfl_sync(0xffffffffu, mine, c * 8);
            rs[1] = __shfl_sync(0xffffffffu, mine, c * 8 + 4);
        }
    }

    // One tile: fk[i] the first key of strip i, -1 if the row sees none of it.  kWhole: the row sees every
    // key of the four strips (all but a row's last tile, and lists' last blocks).
    template <bool kWhole>
    __device__ __forceinline__ void tile(const unsigned char* tile, const int* fk, int pos, int g, int c) {
        // ---- S: [strip][keys g, g + 8 (narrow) or keys 2 c .. and 8 + 2 c .. (wide)]; s[i][n][2 r + e] in the wide
        // form is key 8 n + 2 c + e of row r, s[i][n][r] in the narrow one key 8 n + g of row r
        constexpr int kE = kNarrow ? 2 : 4;
        float s[kTile][2][kE];
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            const unsigned char* strip = tile + i * S::kStripB;
            if (!kWhole && fk[i] < 0) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < kE; ++e) s[i][n][e] = -INFINITY;
                continue;
            }
            uint32_t kf[2][D / 32][4];
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
                    unpack8(w[x], kf[n][x]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) kf[n][x][e] = hmul2(kf[n][x][e], sc[x * 2 / (D / 32)]);
                }
            }
            if constexpr (kNarrow) {
                float d[4];
#pragma unroll
                for (int term = kTerms - 1; term >= 0; --term)  // the small products first: less of them is cut off
#pragma unroll
                    for (int x = 0; x < D / 32; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t ka[4] = {kf[0][x][2 * y], kf[1][x][2 * y], kf[0][x][2 * y + 1], kf[1][x][2 * y + 1]};
                            const uint32_t* b = q[term][2 * x + y];
                            if (x + y == 0 && term == kTerms - 1) mma_zero(d, ka, b[0], b[1]);
                            else mma(d, ka, b[0], b[1]);
                        }
                s[i][0][0] = d[0], s[i][0][1] = d[1], s[i][1][0] = d[2], s[i][1][1] = d[3];
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int term = kTerms - 1; term >= 0; --term)
#pragma unroll
                        for (int x = 0; x < D / 32; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t* b = kf[n][x] + 2 * y;
                                if (x + y == 0 && term == kTerms - 1) mma_zero(s[i][n], q[term][0], b[0], b[1]);
                                else mma(s[i][n], q[term][2 * x + y], b[0], b[1]);
                            }
            }
        }

        if constexpr (!kWhole) {
#pragma unroll
            for (int i = 0; i < kTile; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        if (fk[i] + n * 8 + (kNarrow ? g : c * 2 + (e & 1)) > pos) s[i][n][e] = -INFINITY;
        }

        // ---- the reference moves when a logit passes it by more than kSlack: first a test without any exchange
        float top[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (kNarrow) {
                top[r] = fmaxf(s[0][0][r], s[0][1][r]);
#pragma unroll
                for (int i = 1; i < kTile; ++i) top[r] = ptx::fmax3(top[r], s[i][0][r], s[i][1][r]);
            } else {
                top[r] = fmaxf(s[0][0][2 * r], s[0][0][2 * r + 1]);
#pragma unroll
                for (int i = 0; i < kTile; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        if (i + n > 0) top[r] = ptx::fmax3(top[r], s[i][n][2 * r], s[i][n][2 * r + 1]);
            }
        }
        if (__any_sync(0xffffffffu, top[0] * rs[0] > m[0] + kSlack || top[1] * rs[1] > m[1] + kSlack)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                constexpr int d0 = kNarrow ? 4 : 1, d1 = kNarrow ? 32 : 4;
#pragma unroll
                for (int d = d0; d < d1; d *= 2) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
                const float to = top[r] * rs[r];
                const bool move = to > m[r] + kSlack;
                const float f = move ? ptx::ex2(m[r] - to) : 1.f;
                m[r] = move ? to : m[r];
                if constexpr (kNarrow) (r ? l[0].y : l[0].x) *= f;  // l[0] holds both rows' sums
                else l[r].x *= f, l[r].y *= f;
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    if constexpr (kNarrow) u[j][r] *= f, u[j][2 + r] *= f;
                    else u[j][2 * r] *= f, u[j][2 * r + 1] *= f;
                }
            }
        }
        float base[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) base[r] = m[r] == -INFINITY ? 0.f : kWeightLog2 - m[r];

        // ---- weights and U += P V
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            if (!kWhole && fk[i] < 0) continue;
            uint32_t pf[kTerms][kNarrow ? 2 : 4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if constexpr (kNarrow) {
                    float2 p = ptx::ffma2(make_float2(s[i][n][0], s[i][n][1]), make_float2(rs[0], rs[1]),
                                          make_float2(base[0], base[1]));
                    p.x = ptx::ex2(p.x), p.y = ptx::ex2(p.y);
                    l[0] = ptx::fadd2(l[0], p);  // (row 0, row 1); l[1] is not used
                    const uint32_t two = pack_f16x2(p.x, p.y);
                    pf[0][n] = transpose8x8(two);
                    if constexpr (kTerms == 2) {
                        const float2 b = f16x2_to_f32(two);
                        pf[1][n] = transpose8x8(pack_f16x2(p.x - b.x, p.y - b.y));
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float2 p = ptx::ffma2(make_float2(s[i][n][2 * r], s[i][n][2 * r + 1]),
                                              make_float2(rs[r], rs[r]), make_float2(base[r], base[r]));
                        p.x = ptx::ex2(p.x), p.y = ptx::ex2(p.y);
                        l[r] = ptx::fadd2(l[r], p);
                        const uint32_t two = pack_f16x2(p.x, p.y);
                        pf[0][2 * n + r] = two;
                        if constexpr (kTerms == 2) {
                            const float2 b = f16x2_to_f32(two);
                            pf[1][2 * n + r] = pack_f16x2(p.x - b.x, p.y - b.y);
                        }
                    }
                }
            }
            const unsigned char* strip = tile + i * S::kStripB;
            const int grp = D == 128 ? g : g >> 1;
            uint32_t s0 = e4m3x2_to_f16x2(lds<uint16_t>(strip + 17 * D + grp * 16 + c * 2));
            uint32_t s1 = e4m3x2_to_f16x2(lds<uint16_t>(strip + 17 * D + grp * 16 + c * 2 + 8));
            if constexpr (!kWhole) {  // keys behind the position may hold anything
                const int k0 = c * 2, seen = pos - fk[i];
                s0 &= (k0 <= seen ? 0xffffu : 0u) | (k0 + 1 <= seen ? 0xffff0000u : 0u);
                s1 &= (k0 + 8 <= seen ? 0xffffu : 0u) | (k0 + 9 <= seen ? 0xffff0000u : 0u);
            }
            // the codes of keys (2c, 2c + 1) and (2c + 8, 2c + 9): kCh / 8 words of each.  At D = 128 the groups
            // of a quarter warp meet in the same banks; the second pass costs less than reordering registers.
            uint32_t va[2][2][kCh / 8];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if constexpr (D == 128) {
                    const uint4 v = lds<uint4>(strip + 8 * D + g * 128 + half * 64 + c * 16);
                    va[half][0][0] = v.x, va[half][0][1] = v.y, va[half][1][0] = v.z, va[half][1][1] = v.w;
                } else {
                    const unsigned char* at = strip + 8 * D + ((g >> 1) * 16 + half * 8 + c * 2) * 8 + (g & 1) * 4;
                    va[half][0][0] = lds<uint32_t>(at), va[half][1][0] = lds<uint32_t>(at + 8);
                }
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
                for (int x = 0; x < 4; ++x) {  // channels 2 x and 2 x + 1 of the lane's
                    const uint32_t v[4] = {hmul2(b0[0][x], s0), hmul2(b0[1][x], s0), hmul2(b1[0][x], s1),
                                           hmul2(b1[1][x], s1)};
                    if constexpr (kTerms == 2) {
                        // The tensor cores cut sums off rather than round them, each time by up to a step of the
                        // running sum: over a long row that shrinks float32 outputs by several steps.  So a strip's
                        // products are summed from zero and added here, rounded to nearest.  With the logits' small
                        // products first: 5e-7 off instead of 1.0 to 1.7e-6 (of the outputs' norm, 4000 to 32768
                        // keys), for 63 us instead of 57 (24 requests of 8192 keys, 16 heads on each of 4).
                        if constexpr (kNarrow) {
                            add_products(u[w * 4 + x], v, pf[0][0], pf[0][1], v, pf[1][0], pf[1][1]);
                        } else {
                            add_products(u[w * 8 + 2 * x], pf[0], v[0], v[2], pf[1], v[0], v[2]);
                            add_products(u[w * 8 + 2 * x + 1], pf[0], v[1], v[3], pf[1], v[1], v[3]);
                        }
                    } else if constexpr (kNarrow) {
                        mma(u[w * 4 + x], v, pf[0][0], pf[0][1]);
                    } else {
                        mma(u[w * 8 + 2 * x], pf[0], v[0], v[2]);
                        mma(u[w * 8 + 2 * x + 1], pf[0], v[1], v[3]);
                    }
                }
            }
        }
    }

    // Sums of the lane's rows, complete over the warp.
    __device__ __forceinline__ void totals(float* sum) const {
        if constexpr (kNarrow) sum[0] = l[0].x, sum[1] = l[0].y;
        else sum[0] = l[0].x + l[0].y, sum[1] = l[1].x + l[1].y;
        constexpr int d0 = kNarrow ? 4 : 1, d1 = kNarrow ? 32 : 4;
#pragma unroll
        for (int d = d0; d < d1; d *= 2) {
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
            sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], d);
        }
    }
    // The lane's U as runs of kRun consecutive channels: run i of row r begins at channel ch(i).
    static constexpr int kRun = kNarrow ? kCh : 2 * kCh;
    static __device__ __forceinline__ int row_at(int r, int g, int c) { return kNarrow ? 2 * c + r : g + 8 * r; }
    static __device__ __forceinline__ int ch_at(int g, int c) { return kNarrow ? g * kCh : c * 2 * kCh; }
    __device__ __forceinline__ float at(int r, int i) const {  // i-th channel of the run
        if constexpr (kNarrow) return u[i / 2][(i & 1) * 2 + r];
        else return u[i % kCh][2 * r + i / kCh];
    }
    __device__ __forceinline__ float& ref(int r, int i) {
        if constexpr (kNarrow) return u[i / 2][(i & 1) * 2 + r];
        else return u[i % kCh][2 * r + i / kCh];
    }

    // Sums of a long run beside U: at `at` (the warp's, kept lane by lane in runs of eight 256 floats apart) relative
    // to references `was`, -inf while there are none.  U += those.
    __device__ __forceinline__ void add_aside(const float* at, const float* was, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = was[r] == -INFINITY ? 0.f : ptx::ex2(was[r] - m[r]);
#pragma unroll
            for (int i = 0; i < kRun; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(at + r * (S::kRows * D / 2) + i / 8 * 256 + lane * 8 + i % 8);
                ref(r, i) = fmaf(x.x, f, ref(r, i)), ref(r, i + 1) = fmaf(x.y, f, ref(r, i + 1));
                ref(r, i + 2) = fmaf(x.z, f, ref(r, i + 2)), ref(r, i + 3) = fmaf(x.w, f, ref(r, i + 3));
            }
        }
    }
    __device__ __forceinline__ void put_aside(float* at, float* was, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            was[r] = m[r];
#pragma unroll
            for (int i = 0; i < kRun; i += 8) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = ref(r, i + k), ref(r, i + k) = 0.f;
                ptx::st_global_v8(at + r * (S::kRows * D / 2) + i * 32 + lane * 8, reinterpret_cast<const uint32_t*>(v));
            }
        }
    }
};

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m - kWeightLog2 + log2f(l)) * kLn2;
}
// Four channels of a finished row.
template <int D, typename T>
__device__ __forceinline__ void write_out(const CacheAttn& a, const Where& w, int r, int ch, float4 x, float m, float l) {
    if (r >= w.heads) return;
    const long long at = (long long)w.t * a.HQ + w.hq0 + r;
    const float f = l == 0.f ? 0.f : (a.v_scale ? a.v_scale[w.h] : 1.f) / l;
    T v[4] = {from_f32<T>(x.x * f), from_f32<T>(x.y * f), from_f32<T>(x.z * f), from_f32<T>(x.w * f)};
    T* o = static_cast<T*>(a.out) + at * D + ch;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(v);
    else *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(v);
    if (a.lse && ch == 0) a.lse[at] = lse_of(m, l);
}

// ---------------------------------------------------------------- the kernel

// kPuts: rows may have more tiles than kAside, and bf16 outputs.
template <int D, typename T, bool kNarrow, Mode M, bool kPuts>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, T, kNarrow>::kBlocks) cache_attn_mma_kernel(CacheAttn a, Plan p) {
    using S = Shape<D, T, kNarrow>;
    using P = Part<D, T, kNarrow>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t full = sbase + S::kFull + warp * kStages * 8;
    int* meta = reinterpret_cast<int*>(smem + S::kMeta) + warp * kStages * 8;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(full + i * 8, 1);
        ptx::fence_mbar_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();

    // the warps that share out the tiles: the grid's, or the unit's
    const int id = blockIdx.x * kWarps + warp, warps = (M == kUnits ? p.unit : gridDim.x) * kWarps;
    const int in_unit = M == kUnits ? id % warps : id;
    Ahead ahead;
    int base = 0, total = 0, run_hi = 0;
    int begun = 0;  // parts of the row that the run's end cuts, if the run holds its beginning
    // the next tile; a cut row has a part in every warp up to the one that holds its last tile, tile x being the
    // last warp b's with base + total b / warps < x + 1
    auto advance = [&] {
        ahead.next<M>(a, p, lane, sizeof(T));
        if ((M == kStream || M == kUnits) && ahead.opened) {
            const long long end = (long long)run_hi - ahead.hi + ahead.n - base;
            begun = ahead.hi == ahead.n ? 0 : (int)((end * warps + total - 1) / total) - in_unit;
            if (M == kStream && lane == 0) p.begun[ahead.row] = make_int2(id, begun);
            ahead.opened = false;
        }
    };
    if constexpr (M == kStream || M == kUnits) {
        if (M == kStream) asm volatile("griddepcontrol.launch_dependents;");
        find_start<M>(a, p, reinterpret_cast<int*>(smem), warps, in_unit, ahead, base, total, run_hi);
        if (ahead.left == 0 && lane < S::kRows)  // an empty run inside a row that is cut around it
            p.ml[(long long)id * 2 * S::kRows + lane] = make_float2(-INFINITY, 0.f);
        advance();
    } else if constexpr (M == kRows) {
        ahead.next_row = id;
        ahead.left = 1;
        if (p.work && lane == 0) ahead.claim = atomicAdd(p.work, 1u);
        advance();
    } else {
        ahead.next_row = blockIdx.x / p.splits;
        const Where w = where(a, p, ahead.next_row);
        const Row r = row_of(a, w.t, w.h, tid == 0);
        const int n = tiles_of(r, p), part = blockIdx.x % p.splits * kWarps + warp, parts = p.splits * kWarps;
        if (n == 0) return;  // a padding row: the whole cluster leaves
        ahead.first_tile = (int)((long long)n * part / parts);
        ahead.left = (int)((long long)n * (part + 1) / parts) - ahead.first_tile;
        if (ahead.left > 0) advance();
    }

    int issued = 0, last = -1;
    auto issue = [&](int stage) {
        const bool mine = (lane >> 2) == ahead.at;
        int first = mine ? ahead.first : -1;
        if (first >= 0 && (unsigned)ahead.page >= (unsigned)a.n_pages) {
            raise_status(a.status, BSA_ERR_INDEX);
            first = -1;
        }
        const uint32_t live = __ballot_sync(0xffffffffu, first >= 0);
        int* mt = meta + stage * 8;
        if (mine) mt[lane & 3] = first;
        if (lane == 0) {
            mt[4] = ahead.row, mt[5] = ahead.r.pos, mt[6] = ahead.flags<kPuts>();
            ptx::mbar_arrive_expect_tx(full + stage * 8, __popc(live) * S::kStripB);
        }
        __syncwarp();
        if (first >= 0 && issued != p.stall) {
            const int strip = ((ahead.page * a.H + ahead.h) << (a.sh - 4)) + ((first & ((1 << a.sh) - 1)) >> 4);
            bulk_copy(sbase + (warp * kStages + stage) * S::kTileB + (lane & 3) * S::kStripB,
                      a.cache + (long long)strip * S::kStripB, S::kStripB, full + stage * 8);
        }
    };

    P part;
    part.reset();
    const bool owner = kNarrow ? g == 0 : c == 0;
    float sum[2];
    // O = U / l of a row that is complete in the registers
    auto finish = [&](int number) {
        const Where w = where(a, p, number);
        const float vs = a.v_scale ? a.v_scale[w.h] : 1.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = P::row_at(r, g, c);
            if (row >= w.heads) continue;
            const long long to = (long long)w.t * a.HQ + w.hq0 + row;
            const float f = sum[r] == 0.f ? 0.f : vs / sum[r];
            T* o = static_cast<T*>(a.out) + to * D + P::ch_at(g, c);
#pragma unroll
            for (int i = 0; i < P::kRun; i += 16 / (int)sizeof(T)) {
                T v[16 / sizeof(T)];
#pragma unroll
                for (int k = 0; k < 16 / (int)sizeof(T); ++k) v[k] = from_f32<T>(part.at(r, i + k) * f);
                *reinterpret_cast<uint4*>(o + i) = *reinterpret_cast<const uint4*>(v);
            }
            if (a.lse && owner) a.lse[to] = lse_of(part.m[r], sum[r]);
        }
    };
    // a lane's values of row r of a part, eight channels together, runs of eight 256 floats apart
    auto unit_part = [&](int of, int r, int ln) {
        return p.part + (long long)of * 2 * S::kRows * D + r * (S::kRows * D / 2) + ln * 8;
    };
    float was[2];
    auto aside = [&] { return p.aside + (long long)id * S::kRows * D; };
    bool alive = true;
    {
        typename P::Raw raw;  // the first row's queries while its first tiles are looked up
        if (ahead.have) P::fetch_q(raw, a, p, ahead.row, g, c);
        while (issued < kStages && ahead.have) {
            issue(issued);
            ++issued;
            advance();
        }
        __syncwarp();
        if (issued) part.convert_q(raw, c);
    }
    for (int n = 0, stage = 0, parity = 0; n < issued; ++n) {
        const int4 fk4 = *reinterpret_cast<const int4*>(meta + stage * 8);
        const int4 tag = *reinterpret_cast<const int4*>(meta + stage * 8 + 4);  // row, position, flags
        if ((tag.z & kBegin) && n) {  // the row's queries, while its first tile is on its way
            part.reset();
            typename P::Raw raw;
            P::fetch_q(raw, a, p, tag.x, g, c);
            part.convert_q(raw, c);
        }
        if (!ptx::mbar_try_wait(full + stage * 8, parity)) alive = wait_slow(full + stage * 8, parity, a.status, p.stall);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;  // nothing more is issued; the copies in flight are waited for below
        const int fk[kTile] = {fk4.x, fk4.y, fk4.z, fk4.w};
        const unsigned char* tile = smem + (warp * kStages + stage) * S::kTileB;
        const int least = min(min(fk4.x, fk4.y), min(fk4.z, fk4.w)), most = max(max(fk4.x, fk4.y), max(fk4.z, fk4.w));
        if (least >= 0 && most + kStrip - 1 <= tag.y) part.template tile<true>(tile, fk, tag.y, g, c);
        else if (most >= 0) part.template tile<false>(tile, fk, tag.y, g, c);
        __syncwarp();
        if (ahead.have) {
            issue(stage);
            ++issued;
            advance();
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, parity ^= 1;
        if (M != kSplit && (tag.z & (kEnd | kPut))) {
            if (kPuts && (tag.z & kHeld)) part.add_aside(aside(), was, lane);
            part.totals(sum);
            if (kPuts && (tag.z & kPut)) {
                part.put_aside(aside(), was, lane);
            } else if (M == kRows || !(tag.z & kCut)) {
                finish(tag.x);
            } else if (M == kStream || (tag.z & kCarried)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const long long to = ((long long)id * 2 + (tag.z & kCarried ? 0 : 1)) * S::kRows + P::row_at(r, g, c);
                    if (owner) p.ml[to] = make_float2(part.m[r], sum[r]);
                    // a unit's part is read back lane by lane, the others' row by row
                    float* dst = M == kUnits ? unit_part(id, r, lane) : p.part + to * D + P::ch_at(g, c);
                    constexpr int step = M == kUnits ? 32 : 1;
#pragma unroll
                    for (int i = 0; i < P::kRun; i += 8) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = part.at(r, i + k);
                        ptx::st_global_v8(dst + i * step, reinterpret_cast<const uint32_t*>(v));
                    }
                }
            } else {
                last = tag.x;  // the run's last row, begun here and cut: it stays in the registers
            }
        }
    }
    if (!alive)  // bounded too: let the copies of the ring land before the memory is given up
        for (int i = 0; i < kStages; ++i) wait_slow(full + i * 8, 0, a.status, p.stall), wait_slow(full + i * 8, 1, a.status, p.stall);
    if (M == kRows && p.work && lane == 0) {
        __threadfence();
        if (atomicAdd(p.work + 1, 1u) == (unsigned)p.warps - 1) {  // nobody claims any more: zero for the next launch
            p.work[0] = 0;
            p.work[1] = 0;
        }
    }
    if constexpr (M == kUnits) {
        // ---- the cut rows of the unit: the warp that began one adds the following warps' parts
        cluster_sync();
        if (last < 0) return;
        for (int k = 1; k < begun; ++k) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const long long from = (long long)(id + k) * 2 * S::kRows + P::row_at(r, g, c);
                const float2 w = __ldcg(p.ml + from);
                const float top = fmaxf(part.m[r], w.x), keep = weight_of(make_float2(part.m[r], sum[r]), top),
                            f = weight_of(w, top);
                part.m[r] = top;
                sum[r] = sum[r] * keep + w.y * f;
                const float* src = unit_part(id + k, r, lane);
#pragma unroll
                for (int i = 0; i < P::kRun; i += 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(src + i / 8 * 256 + i % 8));
                    const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // no part, no weight: memory of no meaning
                        part.ref(r, i + j) = f != 0.f ? fmaf(v[j], f, part.at(r, i + j) * keep) : part.at(r, i + j) * keep;
                }
            }
        }
        finish(last);
    }
    if constexpr (M != kSplit) return;

    // ---- kSplit: join the CTA's warps, then the cluster's CTAs
    float* U = reinterpret_cast<float*>(smem);
    float2* ml = reinterpret_cast<float2*>(smem + S::kML);
    float2* cml = reinterpret_cast<float2*>(smem + S::kCML);
    part.totals(sum);
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (owner) ml[warp * S::kRows + P::row_at(r, g, c)] = make_float2(part.m[r], sum[r]);
    __syncthreads();  // also: every warp is done with its ring
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = P::row_at(r, g, c), ch = P::ch_at(g, c);
        float cm = -INFINITY, cl = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) cm = fmaxf(cm, ml[k * S::kRows + row].x);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) cl += ml[k * S::kRows + row].y * weight_of(ml[k * S::kRows + row], cm);
        if (warp == 0 && owner) cml[row] = make_float2(cm, cl);
        const float f = weight_of(make_float2(part.m[r], sum[r]), cm);
        float* dst = U + warp * S::kRows * S::kRowF;
#pragma unroll
        for (int i = 0; i < P::kRun; i += 4)
            *reinterpret_cast<float4*>(dst + S::at(row, ch + i)) =
                make_float4(part.at(r, i) * f, part.at(r, i + 1) * f, part.at(r, i + 2) * f, part.at(r, i + 3) * f);
    }
    __syncthreads();
    const Where w = where(a, p, blockIdx.x / p.splits);
    for (int v = tid; v < S::kRows * D / 4; v += kWarps * 32) {
        const int r = v / (D / 4), ch = v % (D / 4) * 4;
        float4* src = reinterpret_cast<float4*>(U + S::at(r, ch));
        float4 x = src[0];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
            const float4 y = src[k * S::kRows * S::kRowF / 4];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        if (p.splits > 1) src[0] = x;
        else write_out<D, T>(a, w, r, ch, x, cml[r].x, cml[r].y);
    }
    if (p.splits == 1) return;
    cluster_sync();
    const int rank = (int)cluster_rank(), share = S::kRows * D / 4 / p.splits;
    for (int v = rank * share + tid; v < (rank + 1) * share; v += kWarps * 32) {
        const int r = v / (D / 4), ch = v % (D / 4) * 4;
        const uint32_t at_ml = sbase + S::kCML + r * 8, at_u = sbase + S::at(r, ch) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll 8
        for (int k = 0; k < p.splits; ++k) mm = fmaxf(mm, ld_cluster2(at_rank(at_ml, k)).x);
#pragma unroll 4
        for (int k = 0; k < p.splits; ++k) {
            const float2 y = ld_cluster2(at_rank(at_ml, k));
            const float f = weight_of(y, mm);
            const float4 z = ld_cluster4(at_rank(at_u, k));
            ll += y.y * f;
            x.x += z.x * f, x.y += z.y * f, x.z += z.z * f, x.w += z.w * f;
        }
        write_out<D, T>(a, w, r, ch, x, mm, ll);
    }
    cluster_sync();  // nobody leaves while others read its shared memory
}

// Joins the parts of a cut row, those of the warp that began it and of the following ones.  A block
// takes 1 / gridDim.y of the row's heads; blockDim / (D / 4 * heads) threads share the parts of four channels.
template <int D, typename T, bool kNarrow>
__global__ void __launch_bounds__(1024) cache_attn_join_kernel(CacheAttn a, Plan p) {
    constexpr int kRows = Shape<D, T, kNarrow>::kRows, kVec = D / 4;
    __shared__ float4 xs[1024];
    __shared__ float2 mls[1024];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the stream's kernel still runs
    const Where w = where(a, p, blockIdx.x);
    const int req = a.req[w.t];
    const int2 begun = p.begun[blockIdx.x];
    if (req < 0 || req >= a.R) return;  // a padding row is never begun
    // nothing to join of a whole row; after an expired wait a row may not have been begun: then this is any number
    if ((unsigned)begun.x >= (unsigned)p.warps || begun.y <= 0 || begun.y > p.warps - begun.x) return;
    const int heads = kRows / gridDim.y, lanes = blockDim.x / kVec / heads;
    const int v = threadIdx.x % kVec, r = threadIdx.x / kVec % heads, part = threadIdx.x / kVec / heads;
    const int row = blockIdx.y * heads + r;
    auto slot = [&](int k) { return ((long long)(begun.x + k) * 2 + (k == 0)) * kRows + row; };
    float mm = -INFINITY, ll = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = part; k0 < begun.y; k0 += 4 * lanes) {  // four parts' loads at a time
        float2 ml[4];
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i * lanes;
            ml[i] = make_float2(-INFINITY, 0.f);
            y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < begun.y) {
                ml[i] = p.ml[slot(k)];
                y[i] = *reinterpret_cast<const float4*>(p.part + slot(k) * D + v * 4);
            }
        }
        float top = fmaxf(fmaxf(mm, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
        const float keep = weight_of(make_float2(mm, ll), top);
        mm = top, ll *= keep;
        x.x *= keep, x.y *= keep, x.z *= keep, x.w *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = weight_of(ml[i], top);
            ll += ml[i].y * f;
            if (f != 0.f) x.x += y[i].x * f, x.y += y[i].y * f, x.z += y[i].z * f, x.w += y[i].w * f;  // else no part: memory of no meaning
        }
    }
    if (lanes == 1) {
        write_out<D, T>(a, w, row, v * 4, x, mm, ll);
        return;
    }
    xs[threadIdx.x] = x;
    mls[threadIdx.x] = make_float2(mm, ll);
    __syncthreads();
    if (part > 0) return;
    const int step = kVec * heads;
    float top = -INFINITY;
    for (int k = 0; k < lanes; ++k) top = fmaxf(top, mls[threadIdx.x + k * step].x);
    ll = 0.f, x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < lanes; ++k) {
        const float2 part_ml = mls[threadIdx.x + k * step];
        const float4 y = xs[threadIdx.x + k * step];
        const float f = weight_of(part_ml, top);
        ll += part_ml.y * f;
        x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
    }
    write_out<D, T>(a, w, row, v * 4, x, top, ll);
}

// ---------------------------------------------------------------- launches

template <typename F>
static bool once_per_device(F f) {  // f(): whether it succeeded; called until it has, for each device and place of call
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return f();
    if (done.load(std::memory_order_acquire) >> dev & 1) return true;
    if (!f()) return false;
    done.fetch_or(1ull << dev, std::memory_order_acq_rel);
    return true;
}

struct Sizes {
    Mode mode;
    Plan plan;
    int grid;
    size_t part, ml, begun, aside;  // workspace bytes
};

template <int D, typename T, bool kNarrow, Mode M, bool kPuts>
static bsa_status launch_mode(const CacheAttn& a, const Plan& p, int grid, cudaStream_t st) {
    using S = Shape<D, T, kNarrow>;
    auto kern = cache_attn_mma_kernel<D, T, kNarrow, M, kPuts>;
    if (!once_per_device([&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) == cudaSuccess;
        }))
        return check_launch("cache_attn_mma_kernel: shared memory");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = M == kSplit ? p.splits : M == kUnits ? p.unit : 1;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = attr.val.clusterDim.x > 1 ? 1 : 0;
    cudaLaunchKernelEx(&cfg, kern, a, p);
    bsa_status rc = check_launch("cache_attn_mma_kernel");
    if (rc != BSA_OK || M != kStream) return rc;
    // parts of a row: about the warps per row; blocks take fewer heads, and share out the parts, where they are many.
    // Measured, us of both kernels with 1, 4 and 16 blocks a row: 4.8 parts 163, 170, 213; 12.7 parts 41.2, 40.8, 64.7;
    // 304 parts 88, 42, 31.
    const int parts = p.warps / p.rows, fold = parts <= 8 ? 1 : parts <= 64 ? 4 : S::kRows;
    cfg.gridDim = dim3(p.rows, fold);
    cfg.blockDim = dim3(fold == S::kRows ? 1024 : 512);
    cfg.dynamicSmemBytes = 0;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, T, kNarrow>, a, p);
    return check_launch("cache_attn_join_kernel");
}

template <int D, typename T, bool kNarrow>
static bsa_status launch(const CacheAttn& a, const Sizes& z, cudaStream_t st) {
    Plan p = z.plan;
    p.warps = z.grid * kWarps;
    p.stall = test_stall_tile();
    p.work = z.mode == kRows ? sched_counter(st) : nullptr;
    // A split row's warp has five tiles at most.  Rows that are short by their sizes have a kernel of their own: what
    // the other one holds for long ones costs 279 us instead of 274 (2048 tokens of 16 blocks of 64).
    constexpr bool kPuts = Shape<D, T, kNarrow>::kTerms == 1;
    switch (z.mode) {
        case kSplit: return launch_mode<D, T, kNarrow, kSplit, false>(a, p, z.grid, st);
        case kStream: return launch_mode<D, T, kNarrow, kStream, kPuts>(a, p, z.grid, st);
        case kUnits:
            if constexpr (Shape<D, T, kNarrow>::kBlocks == 2) return launch_mode<D, T, kNarrow, kUnits, kPuts>(a, p, z.grid, st);
            break;  // never asked for
        default: break;
    }
    if (kPuts && p.aside) return launch_mode<D, T, kNarrow, kRows, kPuts>(a, p, z.grid, st);
    return launch_mode<D, T, kNarrow, kRows, false>(a, p, z.grid, st);
}

// One translation unit each (they compile side by side).
bsa_status launch_64_f32(const CacheAttn& a, const Sizes& z, bool narrow, cudaStream_t st);
bsa_status launch_64_bf16(const CacheAttn& a, const Sizes& z, bool narrow, cudaStream_t st);
bsa_status launch_128_f32(const CacheAttn& a, const Sizes& z, bool narrow, cudaStream_t st);
bsa_status launch_128_bf16(const CacheAttn& a, const Sizes& z, bool narrow, cudaStream_t st);

}  // namespace cmma
}  // namespace bsa
