// What the kernels of attention over the 4-bit paged cache share: their arguments and
// the walk from a token's row to its keys.
#pragma once

#include "cache.cuh"

namespace bsa {

struct CacheAttn {
    const void* q;
    int T, HQ, H, D;
    long long q_stride;
    const uint8_t* cache;
    int n_pages, sh;  // page_size = 1 << sh
    const int32_t* table;
    int R, max_pages;
    const int32_t *req, *pos;
    const float *k_scale, *v_scale;
    const int32_t *blocks, *counts;  // null: every key up to the token's position
    int S, block_strips;
    float scale_log2;
    void* out;
    float* lse;
    int* status;
};

// Row (t, h): its request (-1: a padding token, its output is left as it is), its
// position and its strips, counted in the order of its list.
struct Row {
    int req, pos, strips;
    const int32_t* blocks;
};

// From the loaded request, position and (with lists) count; r.blocks is left null.
__device__ __forceinline__ Row row_from(const CacheAttn& a, int req, int pos, int count, bool report) {
    Row r{req, pos, 0, nullptr};
    if (r.req >= a.R) {
        if (report) raise_status(a.status, BSA_ERR_INDEX);
        r.req = -1;
    }
    if (r.req < 0) return r;
    if (r.pos >= a.max_pages << a.sh) {  // no such key: an empty row
        if (report) raise_status(a.status, BSA_ERR_INDEX);
        r.pos = -1;
    }
    if (r.pos < 0) return r;
    if (!a.blocks) {
        r.strips = (r.pos >> 4) + 1;
        return r;
    }
    if (count > a.S) {
        if (report) raise_status(a.status, BSA_ERR_INDEX);
        count = a.S;
    }
    r.strips = max(count, 0) * a.block_strips;
    return r;
}
__device__ __forceinline__ Row row_of(const CacheAttn& a, int t, int h, bool report) {
    const long long at = (long long)t * a.H + h;
    Row r = row_from(a, a.req[t], a.pos[t], a.blocks ? a.counts[at] : 0, report);
    if (a.blocks) r.blocks = a.blocks + at * a.S;
    return r;
}

// First key of the row's n-th strip, or -1 when the row sees none of its keys.
__device__ __forceinline__ int first_key(const CacheAttn& a, const Row& r, int n, bool report) {
    if (!r.blocks) return n * kStrip;
    const int slot = n / a.block_strips, blk = r.blocks[slot];
    const long long first = ((long long)blk * a.block_strips + (n - slot * a.block_strips)) * kStrip;
    if (blk < 0 || (long long)blk * a.block_strips * kStrip >= (long long)a.max_pages << a.sh) {
        if (report) raise_status(a.status, BSA_ERR_INDEX);
        return -1;
    }
    return first <= r.pos ? (int)first : -1;
}

// Index of the strip in the cache, or -1 (and a latched error) when its page is none of the cache's.
__device__ __forceinline__ int strip_index(const CacheAttn& a, const Row& r, int h, int first, bool report) {
    const int page = a.table[(long long)r.req * a.max_pages + (first >> a.sh)];
    if ((unsigned)page >= (unsigned)a.n_pages) {
        if (report) raise_status(a.status, BSA_ERR_INDEX);
        return -1;
    }
    return ((page * a.H + h) << (a.sh - 4)) + ((first & ((1 << a.sh) - 1)) >> 4);
}

// The tensor-core kernels (D = 64 or 128).
size_t mma_cache_attention_workspace(int T, int HQ, int H, int D, long long max_keys);
int mma_cache_attention_way(int T, int HQ, int H, int D, bool f32, bool lists, long long max_keys);
bsa_status mma_cache_attention(const CacheAttn& a, bsa_dtype dtype, long long max_keys, void* workspace,
                               cudaStream_t st);

}  // namespace bsa
