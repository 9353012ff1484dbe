// Host side of attention over the 4-bit paged cache on the tensor cores (a14): how the work is cut.
#include "cache_attn_mma.cuh"

namespace bsa {
namespace cmma {
namespace {

constexpr int kSms = 152;
// From so many rows a warp on, lists' rows are taken whole, without a look at all of them first: full lists then gain
// up to a fifth, and only long ragged ones lose as much.  Measured, us, 4 requests' chunks, 16 heads on each of 4, rows against
// units, at 2.0, 3.9 and 6.1 rows a warp: 16 blocks of 64, all lists full, 81, 159, 256 against 90, 187, 313; 1 to 16
// blocks a row 78, 145, 195 against 69, 122, 182; 1 to 16 blocks of 128 144, 272, 364 against 104, 192, 292 (full 153,
// 301, 487 against 161, 317, 497).
constexpr int kRowsPerWarp = 6;

// How the work is cut, from the sizes that the host knows.
Sizes cut(int T, int HQ, int H, int D, bool f32, bool lists, long long max_keys) {
    Sizes z = {};
    Plan& p = z.plan;
    const int G = HQ / H;
    const bool narrow = G <= 8;
    const int grid = kSms * (!narrow ? Shape<128, float, false>::kBlocks : f32 ? Shape<128, float, true>::kBlocks
                                                                               : Shape<128, __nv_bfloat16, true>::kBlocks);
    p.head_tiles = (G + 15) / 16;
    const long long rows = (long long)T * H * p.head_tiles;
    p.rows = (int)std::min<long long>(rows, 0x7fffffff);
    p.G = G;
    p.inv_H = (0x100000000ull + H - 1) / H;
    p.tile_strips = kTile;
    p.tile_log2 = 2;
    const long long strips = (max_keys + kStrip - 1) / kStrip, tiles = (strips + kTile - 1) / kTile;
    // A row to a cluster, in one launch, while that leaves a warp five tiles at most and the CTAs fit at once.
    // Measured, us, split against stream: 64 rows of 8, 16, 32, 64 tiles 10.4, 11.1, 13.2, 18.1 against 13.8, 14.8,
    // 16.4, 21.6; 4 rows of 256 tiles (8 to a warp) 20.8 against 16.3.
    int s = 1;
    while (s < 8 && rows * s * 2 <= grid && strips > kWarps * s) s *= 2;
    if (rows * s <= grid && tiles <= 5 * kWarps * s) {
        z.mode = kSplit;
        p.splits = s;
        while (p.tile_strips > 1 && strips <= (long long)s * kWarps * (p.tile_strips / 2)) p.tile_strips /= 2, --p.tile_log2;
        z.grid = (int)(rows * s);
        return z;
    }
    const long long groups = lists ? (long long)T * H : T;
    const bool rows_balance = lists && rows >= (long long)kRowsPerWarp * grid * kWarps;
    z.mode = groups <= kScanGroups && rows * (tiles + 1) <= 0x7fffffffLL && !rows_balance ? kStream : kRows;
    z.grid = grid;
    if (z.mode == kStream) {
        // Whole rows to units where that leaves none with much more than its share: lists' rows are about as long as
        // one another.  A unit is the two CTAs that an SM holds: larger clusters do not tile the GPU (76 clusters of
        // four ran in two rounds: 143 us for 256 tokens of 2048 selected keys, against 99 with the join), and neither
        // do the three of bf16's up to 8 heads.  Measured, us, units against stream.  16 heads, lists of 16 blocks of
        // 128, the units' largest share 0, 4, 9, 14, 19, 27 and 43% over the mean: 51, 82, 128, 43, 61, 43, 42 against
        // 55, 90, 138, 45, 62, 43, 39; float32 of 8 heads, 1 to 9% over: 97, 87, 138 against 109, 94, 145; every key of
        // 12000 rows of 64 to 1024 keys (79 a unit): 388 against 436, float32 of 8 heads 357 against 399.  bf16 of 8
        // heads with clusters of three: 91, 139 and 318 against 72, 111 and 288.
        const long long most = (rows + kSms - 1) / kSms;
        if (grid == 2 * kSms && most * kSms * 100 <= rows * 108 && (lists || most >= 64)) z.mode = kUnits, p.unit = 2;
        const size_t slots = (size_t)grid * kWarps * 2 * (narrow ? 8 : 16);
        z.part = slots * D * sizeof(float);
        z.ml = slots * sizeof(float2);
        z.begun = z.mode == kUnits ? 0 : (size_t)rows * sizeof(int2);
    }
    if (!f32 && tiles > kAside) z.aside = (size_t)grid * kWarps * (narrow ? 8 : 16) * D * sizeof(float);
    return z;
}

}  // namespace
}  // namespace cmma

using namespace cmma;

size_t mma_cache_attention_workspace(int T, int HQ, int H, int D, long long max_keys) {
    size_t most = 0;  // of both types, with and without lists: a workspace is asked for by sizes alone
    for (int k = 0; k < 4; ++k) {
        const Sizes z = cut(T, HQ, H, D, k & 1, k >> 1, max_keys);
        most = std::max(most, z.aside + z.part + z.ml + z.begun);
    }
    return most;
}

int mma_cache_attention_way(int T, int HQ, int H, int D, bool f32, bool lists, long long max_keys) {
    return 1 + (int)cut(T, HQ, H, D, f32, lists, max_keys).mode;
}

bsa_status mma_cache_attention(const CacheAttn& a, bsa_dtype dtype, long long max_keys, void* workspace,
                               cudaStream_t st) {
    if ((long long)a.T * a.H * ((a.HQ / a.H + 15) / 16) > 0x7fffffffLL)
        return fail(BSA_ERR_UNSUPPORTED, "cache attention: too many (token, head) rows");
    Sizes z = cut(a.T, a.HQ, a.H, a.D, dtype == BSA_F32, a.blocks != nullptr, max_keys);
    char* ws = static_cast<char*>(workspace);
    z.plan.aside = z.aside ? reinterpret_cast<float*>(ws) : nullptr;  // first: it needs the workspace's alignment
    z.plan.part = reinterpret_cast<float*>(ws + z.aside);
    z.plan.ml = reinterpret_cast<float2*>(ws + z.aside + z.part);
    z.plan.begun = reinterpret_cast<int2*>(ws + z.aside + z.part + z.ml);
    const bool narrow = a.HQ / a.H <= 8;
    if (dtype == BSA_F32) return a.D == 128 ? launch_128_f32(a, z, narrow, st) : launch_64_f32(a, z, narrow, st);
    return a.D == 128 ? launch_128_bf16(a, z, narrow, st) : launch_64_bf16(a, z, narrow, st);
}

}  // namespace bsa
