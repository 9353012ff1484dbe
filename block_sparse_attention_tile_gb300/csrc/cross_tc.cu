// a18 cross attention on the tensor cores: bf16, head dims up to 128 that are multiples of 8, float32 accumulation
// in TMEM.
//
// "VSA 实现详解：三维分块、均值路由与块稀疏 Attention" §6.3, §6.5 for the online softmax in the log2 domain.
//
// A persistent grid, one CTA per SM, 16 warps.  An item is 256 query rows (two tiles of 128: tokens x up to 64 of
// the heads that share a KV head) against a part of one sequence's keys; both tiles read the same K and V tiles, so
// that a key is brought from L2 once for 256 rows.  TMEM: S of the two tiles [0, 256), O behind it.
//   warp 3      scheduler: the next item's sequence, rows and key tiles into one of two headers
//   warps 0, 2  producers: Q and the K ring, the V ring, by 4-D TMA boxes straight from the strided tensors (channels
//               past D and rows past the tensor are filled with zeros).  V rows behind the sequence's last key are
//               set to zero in shared memory: a weight of 0 times a NaN there would be NaN.
//   warp 1      MMA issuer: per key tile j and row tile w, P_w V_j and then S_w of tile j + 1, so that one tile's
//               softmax runs while the tensor cores work for the other.
//   warps 4-7, 8-11  softmax of row tile 0 and 1, one row a thread: running maximum (O is rescaled only when it grows
//               by more than 2^8) and sum, the weights back to TMEM as bf16.
//   warps 12-15 output: O times 1 / sum to global memory while the softmax is at the next item.
// The products bound it where the keys are many and D = 128 (38912 tokens x 2 heads x 16384 keys: 1600 TFLOP/s, 82% of the
// measured matrix rate).  At D = 64 (1108 to 1131) neither they nor the exponentials do, the tensor pipe and the special function
// unit being busy 47% of the time each: it is a key tile's chain of S, softmax, P and P V.  Where the keys are few (115200
// tokens x 512 keys: 571 us, 371 of it products) the items' starts, outputs and changes of queries are the rest.
// Every wait is bounded (2 s, and 20 us for each key tile that an item may have, some ten times what one takes: the waits for
// an item's end last as long as the item): on expiry the CTA raises BSA_ERR_TIMEOUT, drains its copies and products, frees TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "cross.cuh"
#include "tc_ptx.cuh"

namespace bsa {
namespace cross {

constexpr int kBM = 128, kBN = 128;      // rows of a tile, keys of a tile
constexpr int kRows = 2 * kBM;           // rows of an item
constexpr int kThreads = 512;
constexpr int kMaxStages = 6;            // K and V tiles in flight, at most
constexpr uint64_t kWaitNs = 2000000000ull, kWaitTileNs = 20000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// The tensor cores cut off what they add to O: by up to 2^-23 of it at each of a key tile's eight products, which does not
// average out over values of one sign (unsplit 2^20 keys came out 5e-3 short).  Every so many key tiles the sums are
// therefore put aside, and those are added up rounded: 1.3e-4 at most for up to 2^20 keys.  Only calls whose states
// could be that long get the code for it, which makes the softmax's loop longer (D = 64, 6 x 4001 queries over up to 1024
// states: 82 us with it, 78.5 without).
constexpr int kAside = 128;
static_assert((kAside & (kAside - 1)) == 0, "kAside is a mask");
constexpr int kRegsLow = 64, kRegsHigh = 176, kRegsOut = 96, kRegsLaunch = 128;  // setmaxnreg (x 128 / 256 / 128 threads)
static_assert(128 * kRegsLow + 256 * kRegsHigh + 128 * kRegsOut <= kThreads * kRegsLaunch, "register split exceeds the launch");
constexpr uint32_t kHalf = kBN * 64 * 2;  // 128 rows x 64 channels

constexpr int kHeaders = 2;  // items known at once (with 4 a CTA holds more of a short batch's items than its share)
constexpr int BAR_QFULL = 0, BAR_QFREE = 2, BAR_FULL = 4, BAR_EMPTY = BAR_FULL + kMaxStages, BAR_SF = BAR_EMPTY + kMaxStages,
              BAR_PF = BAR_SF + 2, BAR_OF = BAR_PF + 2, BAR_OFREE = BAR_OF + 2, BAR_TFULL = BAR_OFREE + 2,
              BAR_TFREE = BAR_TFULL + kHeaders, BAR_XF = BAR_TFREE + kHeaders, BAR_RAW = BAR_XF + 2,
              BAR_DRAIN = BAR_RAW + 1, NBAR = BAR_DRAIN + 1;
constexpr int kTabUsers = 3 + 8 + 4;

template <int HD> struct Smem {
    static constexpr int kK = HD == 128 ? 2 : 3, kV = kK;              // stages of the K and V rings
    static constexpr uint32_t kTile = kBN * HD * 2;
    static constexpr uint32_t kRing = 2 * kTile;                       // Q first
    static constexpr uint32_t kOut = kRing + (kK + kV) * kTile;        // a row tile of the output, for whole-line stores
    static constexpr uint32_t kHdr = kOut + kTile;                     // Item[kHeaders]
    static constexpr uint32_t kInv = kHdr + kHeaders * 48;             // float[2][128]: 1 / sum of a row
    static constexpr uint32_t kBar = kInv + 4 * kRows;
    static constexpr uint32_t kMisc = kBar + 8 * NBAR;
    static constexpr uint32_t kBytes = kMisc + 32 + 1024;
};
static_assert(Smem<128>::kBytes <= 227 * 1024, "shared memory budget");

struct Params {
    Cross a;            // G: the heads side by side in a row tile
    int groups, per_kv; // groups of G query heads; of them per KV head
    int qbm, kbm, vbm, khm, vhm;  // multipliers of the TMA coordinates (0: broadcast dimension)
    float scale_log2;
    int items;
    unsigned* sched;
    uint64_t wait_ns;   // of a bounded wait
    int stall;          // tests only: this K tile of each CTA is not loaded, or -1
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& prm) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer() - t0 > prm.wait_ns) {
            *abort_flag = 1;
            raise_status(prm.a.status, BSA_ERR_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& prm) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, prm));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// 32 columns of this thread's TMEM lane, and the largest of them as floats.
__device__ __forceinline__ void ld32_max(uint32_t taddr, uint32_t* r, float& top) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
        : "r"(taddr)
        : "memory");
}

// Columns from `first` on of this thread's row of S become -inf, in TMEM: rare, and a few instructions of the softmax's
// straight code where a select for each of a row's 128 registers would be as long as the rest of it.
__device__ __forceinline__ void hide_columns(uint32_t tS, int first) {
    uint32_t none[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) none[e] = 0xff800000u;
#pragma unroll 1
    for (; first & 15; ++first) asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tS + first), "r"(none[0]) : "memory");
#pragma unroll 1
    for (; first < kBN; first += 16) ptx::tmem_st16(tS + first, none);
    ptx::tmem_wait_st();
}

// A shared-memory matrix descriptor (128-byte swizzle, stride 1024) from its address in units of 16 bytes.
__device__ __forceinline__ uint64_t desc(uint32_t addr16, uint32_t lbo_bytes) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | (lbo_bytes >> 4) << 16), "r"((1024u >> 4) | 1u << 14 | 2u << 29));
    return d;
}

__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// An item as the header holds it.
struct Item {
    int b, group, row, rows;     // row: the item's first of the sequence; rows <= 256 of it
    int key, keys, t0, t1;       // the sequence's keys; key tiles [t0, t1) of them
    int part, q0, shift, pad;    // q0: the sequence's first query; shift: log2 G
};

// Where row `at` of an item lies: batch, token, query head, and its row in the part's results.
struct RowAt {
    long long batch, tok, part;
    int hq;
};
__device__ __forceinline__ RowAt row_at(const Cross& a, const Item& x, int at) {
    const int r = x.row + at, t = r >> x.shift;  // G is a power of two
    RowAt p;
    p.hq = x.group * a.G + (r & (a.G - 1));
    p.batch = a.query_start ? 0 : x.b;
    p.tok = x.q0 + t;
    p.part = a.parts > 1 ? ((long long)x.part * (a.query_start ? a.N : (long long)a.B * a.N) + p.batch * a.N + p.tok) * a.HQ + p.hq : 0;
    return p;
}

template <int HD, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
cross_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const Params prm) {
    using L = Smem<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - raw);
    uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    auto bar = [&](int i) { return base + L::kBar + 8u * (uint32_t)i; };
    float* inv = reinterpret_cast<float*>(sm + L::kInv);
    auto hdr = [&](int b) { return reinterpret_cast<Item*>(sm + L::kHdr) + b; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(BAR_QFULL + i), 1);
            ptx::mbar_init(bar(BAR_QFREE + i), 1);
            ptx::mbar_init(bar(BAR_SF + i), 1);
            ptx::mbar_init(bar(BAR_PF + i), kBM);
            ptx::mbar_init(bar(BAR_OF + i), 1);
            ptx::mbar_init(bar(BAR_OFREE + i), kBM);
            ptx::mbar_init(bar(BAR_XF + i), kBM);
        }
        for (int i = 0; i < kHeaders; ++i) {
            ptx::mbar_init(bar(BAR_TFULL + i), 1);
            ptx::mbar_init(bar(BAR_TFREE + i), kTabUsers);
        }
        for (int i = 0; i < L::kK + L::kV; ++i) {
            ptx::mbar_init(bar(BAR_FULL + i), 1);
            ptx::mbar_init(bar(BAR_EMPTY + i), 1);
        }
        ptx::mbar_init(bar(BAR_RAW), 1);
        ptx::mbar_init(bar(BAR_DRAIN), 1);
        ptx::fence_mbar_init();
        misc[1] = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + L::kMisc, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc[0];

    // Every role walks the same items: item it uses header it % kHeaders.  Row tile w takes part in an item (is "live") when
    // the item has key tiles and more than 128 w rows; barriers of a row tile count its live items.
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
      if (warp == 3) {
        // Ragged batches of up to 32 sequences: a lane a sequence, the ones with the most keys first, so that the long
        // items do not begin last (16 prompts of 1 to 511 tokens over 64 to 4096 states: 189 us, and 229 in their own order; in a
        // graph 210 and 239).
        const bool sorted = prm.a.B <= 32 && (prm.a.query_start || prm.a.key_start || prm.a.key_lens);
        int sq0 = 0, sn = 0, sk0 = 0, sm_ = 0, sb = 0, stiles = 0, sends = 0;  // of the lane's sequence; sends: items up to its last
        if (sorted) {
            int q0 = 0, n = 0, k0 = 0, m = -1, rank = 0;
            if (lane < prm.a.B) {
                queries_of(prm.a, lane, q0, n);
                keys_of(prm.a, lane, k0, m);
            }
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                const int o = __shfl_sync(0xffffffffu, m, j);
                rank += o > m || (o == m && j < lane);
            }
#pragma unroll 1
            for (int j = 0; j < 32; ++j)
                if (__shfl_sync(0xffffffffu, rank, j) == lane) sb = j;
            sq0 = __shfl_sync(0xffffffffu, q0, sb), sn = __shfl_sync(0xffffffffu, n, sb);
            sk0 = __shfl_sync(0xffffffffu, k0, sb), sm_ = __shfl_sync(0xffffffffu, m, sb);
            stiles = (int)(((long long)sn * prm.a.G + kRows - 1) / kRows);
            sends = stiles * prm.groups * prm.a.parts;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sends, o);
                if (lane >= o) sends += x;
            }
        }
        int next = blockIdx.x;
        for (int it = 0;; ++it) {
            // the ticket is drawn only when the header is free: one drawn earlier would hold one more item of a ragged batch
            // back from CTAs that are done
            if (it >= kHeaders && !warp_wait(bar(BAR_TFREE + it % kHeaders), (uint32_t)(it / kHeaders - 1) & 1u, abort_flag, prm)) break;
            Item x{};
            x.b = -1;
            while (true) {
                int t;
                if (prm.sched && next != (int)blockIdx.x) {  // the first item needs no ticket
                    unsigned tk = 0;
                    if (lane == 0) tk = atomicAdd(prm.sched, 1u);
                    t = (int)(gridDim.x + __shfl_sync(0xffffffffu, tk, 0));
                } else {
                    t = next;
                    next += gridDim.x;
                }
                if (t < 0 || t >= prm.items) break;
                int row0, q0, n;
                if (sorted) {
                    const unsigned hit = __ballot_sync(0xffffffffu, sends > t);
                    if (!hit) break;  // behind the last sequence's items
                    const int l = __ffs(hit) - 1, tiles = __shfl_sync(0xffffffffu, stiles, l);
                    const int in = t - __shfl_sync(0xffffffffu, sends, l) + tiles * prm.groups * prm.a.parts;
                    x.part = in % prm.a.parts;
                    x.group = in / prm.a.parts / tiles;
                    row0 = (in / prm.a.parts - x.group * tiles) * kRows;
                    x.b = __shfl_sync(0xffffffffu, sb, l);
                    q0 = __shfl_sync(0xffffffffu, sq0, l), n = __shfl_sync(0xffffffffu, sn, l);
                    x.key = __shfl_sync(0xffffffffu, sk0, l), x.keys = __shfl_sync(0xffffffffu, sm_, l);
                } else {
                    const int u = t / prm.a.parts;
                    x.part = t - u * prm.a.parts;
                    x.group = u / prm.a.tiles;
                    tile_of<kRows>(prm.a, u % prm.a.tiles, x.b, row0);
                    if (x.b < 0) continue;  // behind the last sequence's tiles
                    queries_of(prm.a, x.b, q0, n);
                    keys_of(prm.a, x.b, x.key, x.keys);
                }
                x.q0 = q0;
                x.shift = __ffs(prm.a.G) - 1;
                x.row = row0;
                x.rows = min((long long)kRows, (long long)n * prm.a.G - row0);
                const int nt = (x.keys + kBN - 1) / kBN;
                x.t0 = (int)((long long)nt * x.part / prm.a.parts);
                x.t1 = (int)((long long)nt * (x.part + 1) / prm.a.parts);
                break;
            }
            if (lane == 0) {
                *hdr(it % kHeaders) = x;
                ptx::mbar_arrive(bar(BAR_TFULL + it % kHeaders));
            }
            if (x.b < 0) break;
        }
      } else if (warp == 0) {
        // ------------------------------------------------------------ Q and K
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        int cnt = 0, ql[2] = {0, 0};
        bool ok = true;
        for (int it = 0; ok; ++it) {
            if (!warp_wait(bar(BAR_TFULL + it % kHeaders), (uint32_t)(it / kHeaders) & 1u, abort_flag, prm)) break;
            const Item x = *hdr(it % kHeaders);
            if (x.b < 0) break;
            const int q0 = x.q0 + x.row / prm.a.G, h = x.group / prm.per_kv * prm.khm;
            // in the order in which they are needed and their buffers become free: K_0, Q_0, K_1, Q_1, K_2 ...
            for (int j = x.t0; j < x.t1 && ok; ++j) {
                const int st = cnt % L::kK;
                ok = warp_wait(bar(BAR_EMPTY + st), ((uint32_t)(cnt / L::kK) & 1u) ^ 1u, abort_flag, prm);
                if (!ok) break;
                if (lane == 0 && cnt != prm.stall) {
                    ptx::mbar_arrive_expect_tx(bar(BAR_FULL + st), L::kTile);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c)
                        tma_load_4d(base + L::kRing + st * L::kTile + c * kHalf, &tm_k, 64 * c, h, x.key + j * kBN,
                                    x.b * prm.kbm, bar(BAR_FULL + st));
                }
                ++cnt;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (x.rows <= w * kBM || (j != x.t0 + w && !(w == 1 && x.t1 - x.t0 == 1))) continue;
                    if (ql[w] > 0) ok = ok && warp_wait(bar(BAR_QFREE + w), (uint32_t)(ql[w] - 1) & 1u, abort_flag, prm);
                    if (!ok) break;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar(BAR_QFULL + w), L::kTile);
#pragma unroll
                        for (int c = 0; c < HD / 64; ++c)
                            tma_load_4d(base + w * L::kTile + c * kHalf, &tm_q, 64 * c, x.group * prm.a.G,
                                        q0 + w * (kBM / prm.a.G), x.b * prm.qbm, bar(BAR_QFULL + w));
                    }
                    ++ql[w];
                }
            }
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
        }
        if (*abort_flag) {  // wait (bounded) for this warp's copies in flight
            const uint64_t t0 = ptx::globaltimer();
            auto drain = [&](int b, uint32_t ph) {
                while (!ptx::mbar_try_wait(bar(b), ph) && ptx::globaltimer() - t0 < prm.wait_ns) {}
            };
            for (int c = max(0, cnt - L::kK); c < cnt; ++c) drain(BAR_FULL + c % L::kK, (uint32_t)(c / L::kK) & 1u);
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if (ql[w]) drain(BAR_QFULL + w, (uint32_t)(ql[w] - 1) & 1u);
        }
      } else if (warp == 2) {
        // ------------------------------------------------------------ V
        ptx::prefetch_tmap(&tm_v);
        int cnt = 0, patched = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            if (!warp_wait(bar(BAR_TFULL + it % kHeaders), (uint32_t)(it / kHeaders) & 1u, abort_flag, prm)) break;
            const Item x = *hdr(it % kHeaders);
            if (x.b < 0) break;
            const int h = x.group / prm.per_kv * prm.vhm;
            for (int j = x.t0; j < x.t1; ++j) {
                const int st = L::kK + cnt % L::kV, nv = x.keys - j * kBN;
                ok = warp_wait(bar(BAR_EMPTY + st), ((uint32_t)(cnt / L::kV) & 1u) ^ 1u, abort_flag, prm);
                if (!ok) break;
                const uint32_t dst = base + L::kRing + st * L::kTile, full = bar(nv < kBN ? BAR_RAW : BAR_FULL + st);
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c)
                        tma_load_4d(dst + c * kHalf, &tm_v, 64 * c, h, x.key + j * kBN, x.b * prm.vbm, full);
                }
                ++cnt;
                if (nv < kBN) {
                    ok = warp_wait(full, (uint32_t)patched & 1u, abort_flag, prm);
                    ++patched;
                    if (!ok) break;
                    for (int c = 0; c < HD / 64; ++c)
                        for (int i = nv * 8 + lane; i < kBN * 8; i += 32)
                            *reinterpret_cast<uint4*>(sm + (dst - base) + c * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(BAR_FULL + st));
                }
            }
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
        }
        if (*abort_flag) {
            const uint64_t t0 = ptx::globaltimer();
            for (int c = max(0, cnt - L::kV); c < cnt; ++c)
                while (!ptx::mbar_try_wait(bar(BAR_FULL + L::kK + c % L::kV), (uint32_t)(c / L::kV) & 1u) &&
                       ptx::globaltimer() - t0 < prm.wait_ns) {
                }
            if (patched)
                while (!ptx::mbar_try_wait(bar(BAR_RAW), (uint32_t)(patched - 1) & 1u) && ptx::globaltimer() - t0 < prm.wait_ns) {}
        }
      } else if (elect()) {
        // ------------------------------------------------------------ MMA issuer
        // One elected lane, which the compiler knows to be alone: a product then takes some 60 cycles to issue, of the
        // 64 that it runs (95 from `if (lane == 0)`; and with the whole warp in the loop every wait costs 100 more).
        // What it walks is kept short, because most of it is fetched anew for each item: sending the next item's first S
        // ahead of row tile 1's last product, and its queries to L2 ahead of that, cost more (611 us) than they gave (590).
        constexpr uint32_t idS = ptx::idesc_bf16(kBM, kBN, false), idO = ptx::idesc_bf16(kBM, HD, true);
        const uint32_t tm = tmem;
        int kc = 0, vc = 0;                // K and V tiles consumed
        int live0 = 0, live1 = 0, up0 = 0, up1 = 0;  // live items and P tiles consumed of the two row tiles
        bool ok = true;
        auto wait = [&](int b, uint32_t ph) { return wait_bar(bar(b), ph & 1u, abort_flag, prm); };
        const uint32_t lo = (base >> 4) & 0x3FFF;  // descriptors differ in their address alone, in units of 16 bytes
        auto issue_s = [&](int w, int st) {  // S of row tile w
            const uint32_t dq = lo + (uint32_t)w * (L::kTile >> 4), dk = lo + (L::kRing >> 4) + (uint32_t)st * (L::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                ptx::mma_ss(tm + (uint32_t)w * 128, desc(dq + off, 16), desc(dk + off, 16), idS, kk > 0);
            }
            ptx::mma_commit(bar(BAR_SF + w));
        };
        auto issue_pv = [&](int w, int st, bool add) {
            const uint32_t dv = lo + (L::kRing >> 4) + (uint32_t)st * (L::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
                ptx::mma_ts(tm + 256 + (uint32_t)w * HD, tm + (uint32_t)w * 128 + kk * 8, desc(dv + (kk * 2048 >> 4), kHalf),
                            idO, (add || kk > 0) ? 1u : 0u);
        };
        for (int it = 0; ok; ++it) {
            if (!wait(BAR_TFULL + it % kHeaders, (uint32_t)(it / kHeaders))) break;
            const Item* x = hdr(it % kHeaders);
            if (x->b < 0) break;
            const int n = x->t1 - x->t0, nw = x->rows > kBM ? 2 : 1;
            // step -1: S of the first key tile; step j: P V of tile j, then S of tile j + 1
#pragma unroll 1
            for (int j = -1; j < n && n > 0; ++j) {
                const int vst = L::kK + vc % L::kV, kst = kc % L::kK;
                const bool more = j + 1 < n;
#pragma unroll 1
                for (int w = 0; w < nw; ++w) {
                    if (j < 0) ok = wait(BAR_QFULL + w, (uint32_t)(w ? live1 : live0));
                    if (w == 0) ok = ok && (j < 0 || wait(BAR_FULL + vst, (uint32_t)(vc / L::kV))) &&
                                     (!more || wait(BAR_FULL + kst, (uint32_t)(kc / L::kK)));
                    if (j == 0 && (w ? live1 : live0) > 0) ok = ok && wait(BAR_OFREE + w, (uint32_t)((w ? live1 : live0) - 1));
                    if (j >= 0) ok = ok && wait(BAR_PF + w, (uint32_t)(w ? up1++ : up0++));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (j >= 0) {
                        issue_pv(w, vst, kLong ? (j & (kAside - 1)) != 0 : j > 0);
                        if (w == nw - 1) ptx::mma_commit(bar(BAR_EMPTY + vst));
                        if (!more) ptx::mma_commit(bar(BAR_OF + w));
                    }
                    if (more) {
                        issue_s(w, kst);
                        if (w == nw - 1) ptx::mma_commit(bar(BAR_EMPTY + kst));
                        if (j + 2 == n) ptx::mma_commit(bar(BAR_QFREE + w));
                    }
                }
                if (!ok) break;
                vc += j >= 0;
                kc += more;
            }
            if (!ok) break;
            live0 += n > 0;
            live1 += n > 0 && nw == 2;
            ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
        }
        // nothing that this warp issued may still run when TMEM is freed
        {
            ptx::mma_commit(bar(BAR_DRAIN));
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar(BAR_DRAIN), 0) && ptx::globaltimer() - t0 < prm.wait_ns) {}
        }
      }
    } else if (warp < 12) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
      // -------------------------------------------------------------- softmax and output
      const int w = (warp - 4) >> 2, row = threadIdx.x & 127;
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t tO = tmem + lane_off + 256 + HD * w, tS = tmem + lane_off + (uint32_t)w * 128;
      const Cross& a = prm.a;
      int su = 0, live = 0;  // S tiles, live items
      uint32_t r[16];
      float x[kBN];
      [[maybe_unused]] float aside[kLong ? HD : 1];  // in local memory
      for (int it = 0;; ++it) {
        if (!warp_wait(bar(BAR_TFULL + it % kHeaders), (uint32_t)(it / kHeaders) & 1u, abort_flag, prm)) break;
        const Item* hd = hdr(it % kHeaders);
        if (hd->b < 0) break;
        if (hd->rows <= w * kBM) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
            continue;
        }
        const int n = hd->t1 - hd->t0;
        int left = hd->keys - hd->t0 * kBN;  // keys from the current tile on
        float m_ref = -CUDART_INF_F, l = 0.f;
        [[maybe_unused]] float m_aside = -CUDART_INF_F, l_aside = 0.f;
        bool ok = true;
        [[maybe_unused]] const auto from_aside = [&] { return m_aside == -CUDART_INF_F ? 0.f : ptx::ex2(m_aside - m_ref); };
        for (int j = 0; j < n; ++j, left -= kBN) {
            const int nv = left;
            ok = warp_wait(bar(BAR_SF + w), (uint32_t)su & 1u, abort_flag, prm);
            if (!ok) break;
            ++su;
            ptx::tc_fence_after();
            if (nv < kBN) hide_columns(tS, nv);
            // maxima of raw Q.K come with the load: scale once (scale > 0 keeps the order)
            float mx;
            {
                uint32_t* xr = reinterpret_cast<uint32_t*>(x);
                float top[4];
                ld32_max(tS + 0, xr + 0, top[0]);
                ld32_max(tS + 32, xr + 32, top[1]);
                ld32_max(tS + 64, xr + 64, top[2]);
                ld32_max(tS + 96, xr + 96, top[3]);
                ptx::tmem_wait_ld();
                mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            }
            mx *= prm.scale_log2;
            const float m_new = fmaxf(m_ref, mx);
            const bool need = m_new > m_ref + kRescaleThreshold;
            if (__any_sync(0xffffffffu, need)) {
                const float alpha = need ? ptx::ex2(m_ref - m_new) : 1.f;
                if (need) m_ref = m_new;
                l *= alpha;
                if (j > 0) {
                    // S_j was issued after the last product added to O: O is complete here
#pragma unroll 1
                    for (int c = 0; c < HD / 16; ++c) {
                        ptx::tmem_ld16(tO + c * 16, r);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                        ptx::tmem_st16(tO + c * 16, r);
                    }
                    ptx::tmem_wait_st();
                }
            }
            if (kLong && j > 0 && (j & (kAside - 1)) == 0) {  // the next product begins O anew
                const float f = from_aside();
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                    ptx::tmem_ld16(tO + c * 16, r);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) aside[c * 16 + e] = __uint_as_float(r[e]) + (j == kAside ? 0.f : aside[c * 16 + e] * f);
                }
                l_aside = fmaf(l_aside, f, l);
                l = 0.f;
                m_aside = m_ref;
            }
            const bool some = m_ref != -CUDART_INF_F;
            const float sc = some ? prm.scale_log2 : 1.f, ref = some ? m_ref : 0.f;
            const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-ref, -ref);
            float2 acc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] = make_float2(0.f, 0.f);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
#pragma unroll
                for (int c = h * 32; c < h * 32 + 32; c += 2) {
                    const float2 z = ptx::ffma2(make_float2(x[c], x[c + 1]), sc2, nm2);
                    x[c] = ptx::ex2(z.x);
                    x[c + 1] = ptx::ex2(z.y);
                    acc[(c >> 1) & 3] = ptx::fadd2(acc[(c >> 1) & 3], make_float2(x[c], x[c + 1]));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = ptx::pack_bf16x2(x[h * 32 + 2 * e], x[h * 32 + 2 * e + 1]);
                ptx::tmem_st16(tS + h * 16, r);
            }
            l += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) + ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(BAR_PF + w));
        }
        if (!ok) break;
        if (n > 0) {
            if (kLong && n > kAside) {
                if (!warp_wait(bar(BAR_OF + w), (uint32_t)live & 1u, abort_flag, prm)) break;
                ptx::tc_fence_after();
                const float f = from_aside();
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                    ptx::tmem_ld16(tO + c * 16, r);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(fmaf(aside[c * 16 + e], f, __uint_as_float(r[e])));
                    ptx::tmem_st16(tO + c * 16, r);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                l = fmaf(l_aside, f, l);
            }
            // the output is another warpgroup's: it gets 1 / sum, once it has read the last item's
            if (live > 0 && !warp_wait(bar(BAR_OFREE + w), (uint32_t)(live - 1) & 1u, abort_flag, prm)) break;
            ++live;
            inv[w * kBM + row] = l == 0.f ? 0.f : 1.f / l;
            ptx::mbar_arrive(bar(BAR_XF + w));
        }
        const int at = w * kBM + row;
        if ((a.parts > 1 || a.lse) && at < hd->rows) {
            const RowAt p = row_at(a, *hd, at);
            const float lse = l == 0.f ? -CUDART_INF_F : (m_ref + log2f(l)) * kLn2;
            if (a.parts > 1) a.part_lse[p.part] = lse;
            else a.lse[p.batch * a.lb + p.tok * a.lt + p.hq * a.lh] = lse;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
      // -------------------------------------------------------------- output
      const int row = threadIdx.x & 127;
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      const Cross& a = prm.a;
      constexpr int kChunks = HD / 8;  // of 16 bytes, in a row
      uint4* stage = reinterpret_cast<uint4*>(sm + L::kOut);
      const auto pack = [](const uint32_t* v) { return ptx::pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
      int live[2] = {0, 0};
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!warp_wait(bar(BAR_TFULL + it % kHeaders), (uint32_t)(it / kHeaders) & 1u, abort_flag, prm)) break;
        const Item& hd = *hdr(it % kHeaders);
        if (hd.b < 0) break;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (!ok || hd.rows <= w * kBM) break;
            const int at = w * kBM + row;
            const bool some = hd.t1 > hd.t0;
            float scale = 0.f;
            if (some) {
                ok = warp_wait(bar(BAR_XF + w), (uint32_t)live[w] & 1u, abort_flag, prm) &&
                     warp_wait(bar(BAR_OF + w), (uint32_t)live[w] & 1u, abort_flag, prm);
                if (!ok) break;
                ++live[w];
                ptx::tc_fence_after();
                scale = inv[at];
            }
            const uint32_t tO = tmem + lane_off + 256 + HD * w;
            float* po = a.parts > 1 && at < hd.rows ? a.part_out + row_at(a, hd, at).part * a.D : nullptr;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t r[32];
                if (some) {
                    ptx::tmem_ld32(tO + c * 32, r);
                    ptx::tmem_wait_ld();
                    if (c == HD / 32 - 1) {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(bar(BAR_OFREE + w));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * scale);
                if (a.parts > 1) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (po && 32 * c + 8 * h < a.D) ptx::st_global_v8(po + 32 * c + 8 * h, r + 8 * h);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        stage[row * kChunks + ((4 * c + h) ^ (row & 7))] =
                            make_uint4(pack(r + 8 * h), pack(r + 8 * h + 2), pack(r + 8 * h + 4), pack(r + 8 * h + 6));
                }
            }
            if (a.parts > 1) continue;
            // a warp's own 32 rows, a whole row to adjacent lanes
            __syncwarp();
            const int ch = lane % kChunks, x0 = (warp & 3) * 32 + lane / kChunks, r0 = hd.row + w * kBM + x0;
            const int live_rows = 8 * ch < a.D ? hd.rows - w * kBM : 0, shift = hd.shift, low = a.G - 1;
            __nv_bfloat16* o = (__nv_bfloat16*)a.out + (a.query_start ? 0 : hd.b) * a.ob + hd.q0 * a.ot + (long long)hd.group * a.G * a.oh + 8 * ch;
#pragma unroll 8
            for (int i = 0; i < kChunks; ++i) {
                const int d = i * (32 / kChunks), x = x0 + d;
                if (x < live_rows)
                    *reinterpret_cast<uint4*>(o + ((r0 + d) >> shift) * a.ot + ((r0 + d) & low) * a.oh) = stage[x * kChunks + (ch ^ (x & 7))];
            }
            __syncwarp();
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_TFREE + it % kHeaders));
      }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && prm.sched) {
        __threadfence();
        if (atomicAdd(prm.sched + 1, 1u) == gridDim.x - 1) {
            atomicExch(prm.sched, 0u);
            atomicExch(prm.sched + 1, 0u);
        }
    }
}

// ---------------------------------------------------------------- host side

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// 4-D map (channel, head, token, batch) over a strided tensor, box {64, heads, tokens, 1}.  A dimension of one entry or
// of stride 0 (a broadcast) becomes one entry at coordinate 0, which the caller's multiplier says.
static bool make_map(CUtensorMap* m, const void* ptr, int D, int heads, long long tokens, int batch, long long sh,
                     long long st, long long sb, int box_heads, int box_tokens, int* head_mul, int* batch_mul) {
    auto fn = encode_fn();
    if (!fn || ((uintptr_t)ptr & 15)) return false;
    *head_mul = heads > 1 && sh != 0;
    *batch_mul = batch > 1 && sb != 0;
    if (tokens > 1 && st == 0) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(*head_mul ? heads : 1), (cuuint64_t)tokens,
                                (cuuint64_t)(*batch_mul ? batch : 1)};
    const long long s[3] = {*head_mul ? 2 * sh : 16, tokens > 1 ? 2 * st : 16, *batch_mul ? 2 * sb : 16};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        if (s[i] <= 0 || s[i] % 16 || s[i] >= (1LL << 40)) return false;
        strides[i] = (cuuint64_t)s[i];
    }
    const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool kLong>
static bsa_status launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Params& prm,
                         cudaStream_t st, bool* handled) {
    static int fits = 0;  // 0 unknown, 1 fits, -1 does not: setmaxnreg.inc would wait for registers
    if (!fits) {
        cudaFuncAttributes a;
        fits = (cudaFuncGetAttributes(&a, cross_tc_kernel<HD, kLong>) == cudaSuccess &&
                a.numRegs * kThreads >= 128 * kRegsLow + 256 * kRegsHigh + 128 * kRegsOut) ? 1 : -1;
    }
    if (fits < 0) return BSA_OK;
    *handled = true;
    cudaError_t e = cudaFuncSetAttribute(cross_tc_kernel<HD, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Smem<HD>::kBytes);
    if (e != cudaSuccess) return fail(BSA_ERR_CUDA, "cross attention attribute: %s", cudaGetErrorString(e));
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return fail(BSA_ERR_CUDA, "cross attention: device query failed");
    cross_tc_kernel<HD, kLong><<<std::min(prm.items, sms), kThreads, Smem<HD>::kBytes, st>>>(mq, mk, mv, prm);
    return check_launch("cross_tc_kernel");
}

}  // namespace cross

// The heads of a KV head that lie side by side in a row tile: the largest power of two that divides G, up to 64.
int cross_tc_heads(int G) {
    int g = G & -G;
    return g > 64 ? 64 : g;
}

// Whether the sizes suit the tensor-core kernel (strides and addresses are looked at at the launch).
bool cross_tc_sizes(bsa_dtype dtype, int D) { return dtype == BSA_BF16 && D % 8 == 0; }

bsa_status cross_tc(const Cross& a, cudaStream_t st, bool* handled) {
    using namespace cross;
    *handled = false;
    Params prm{};
    prm.a = a;
    prm.a.G = cross_tc_heads(a.G);
    prm.per_kv = a.G / prm.a.G;
    prm.groups = a.HQ / prm.a.G;
    const bool pq = a.query_start != nullptr, pk = a.key_start != nullptr;
    const long long tiles = row_tiles(a.B, a.N, prm.a.G, pq, kRows), items = tiles * prm.groups * a.parts;
    if (items > INT_MAX / 2) return BSA_OK;
    if (((uintptr_t)a.out & 15) || ((2 * a.ot) & 15) || ((2 * a.oh) & 15) || ((2 * a.ob) & 15)) return BSA_OK;
    prm.a.tiles = (int)tiles;
    prm.items = (int)items;
    CUtensorMap mq, mk, mv;
    int qhm;
    if (a.M == 0) return BSA_OK;  // no state at all: nothing to map
    if (!make_map(&mq, a.q, a.D, a.HQ, a.N, pq ? 1 : a.B, a.qh, a.qt, a.qb, prm.a.G, kBM / prm.a.G, &qhm, &prm.qbm) ||
        !make_map(&mk, a.k, a.D, a.H, a.M, pk ? 1 : a.B, a.kh, a.kt, a.kb, 1, kBN, &prm.khm, &prm.kbm) ||
        !make_map(&mv, a.v, a.D, a.H, a.M, pk ? 1 : a.B, a.vh, a.vt, a.vb, 1, kBN, &prm.vhm, &prm.vbm))
        return BSA_OK;
    if (a.HQ > 1 && !qhm) return BSA_OK;      // queries shared by the heads
    // a scale of 0 would turn a masked -inf into NaN: the smallest normal scale gives the same weights
    prm.scale_log2 = std::max(a.scale * kLog2e, 1.2e-38f);
    prm.sched = sched_counter(st);
    prm.stall = test_stall_tile();
    const int item_tiles = ((a.M + kBN - 1) / kBN + a.parts - 1) / a.parts;  // at most
    prm.wait_ns = prm.stall >= 0 ? 1000000ull : kWaitNs + kWaitTileNs * (uint64_t)item_tiles;
    const bool longs = item_tiles > kAside;
    if (a.D <= 64) return longs ? launch<64, true>(mq, mk, mv, prm, st, handled) : launch<64, false>(mq, mk, mv, prm, st, handled);
    return longs ? launch<128, true>(mq, mk, mv, prm, st, handled) : launch<128, false>(mq, mk, mv, prm, st, handled);
}

}  // namespace bsa
