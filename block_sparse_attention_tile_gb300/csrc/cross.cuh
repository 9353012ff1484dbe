// a18 cross attention: queries over an encoder's states of another length.
//
// Sequence b has the queries [q0, q0 + n) and the states [k0, k0 + m): padded (q0 = k0 = 0 at batch coordinate b,
// n = N, m = key_lens[b]) or packed (starts given, batch coordinate 0).  The rows of a sequence and KV head are the
// tokens' G = HQ / H heads side by side, row r = token r / G, head r % G: one read of the keys serves the group.
// The work is cut into (row tile, KV head, part of the keys) items; with more than one part each writes its own
// normalised output and log-sum-exp and a second kernel joins them.
#pragma once

#include "common.cuh"

namespace bsa {

struct Cross {
    const void *q, *k, *v;
    void* out;
    float* lse;
    long long qb, qt, qh, kb, kt, kh, vb, vt, vh, ob, ot, oh, lb, lt, lh;  // strides: batch, token, head
    const int32_t *query_start, *key_start, *key_lens;
    int B, N, M, HQ, H, D, G;
    float scale;
    int parts;
    float* part_out;  // [parts][rows][HQ][D], rows = B * N or N when packed
    float* part_lse;  // [parts][rows][HQ]
    int tiles;        // row tiles of all sequences (an upper bound when packed)
    int* status;
};

// A bad start or length (not ascending, outside the arrays) empties its sequence and latches BSA_ERR_INDEX.
__device__ __forceinline__ void queries_of(const Cross& a, int b, int& q0, int& n) {
    if (!a.query_start) {
        q0 = 0;
        n = a.N;
        return;
    }
    q0 = a.query_start[b];
    const int q1 = a.query_start[b + 1];
    n = q1 - q0;
    if (q0 < 0 || q1 > a.N || q1 < q0) {
        raise_status(a.status, BSA_ERR_INDEX);
        q0 = n = 0;
    }
}
__device__ __forceinline__ void keys_of(const Cross& a, int b, int& k0, int& m) {
    k0 = 0;
    m = a.M;
    if (a.key_start) {
        k0 = a.key_start[b];
        const int k1 = a.key_start[b + 1];
        m = k1 - k0;
        if (k0 < 0 || k1 > a.M || k1 < k0) {
            raise_status(a.status, BSA_ERR_INDEX);
            k0 = m = 0;
        }
    } else if (a.key_lens) {
        m = a.key_lens[b];
        if (m < 0 || m > a.M) {
            raise_status(a.status, BSA_ERR_INDEX);
            m = m < 0 ? 0 : a.M;
        }
    }
}

// The sequence and the first row of row tile `tile` (kRows rows each), by the whole warp; b = -1 behind the last.
template <int kRows>
__device__ __forceinline__ void tile_of(const Cross& a, int tile, int& b, int& row) {
    if (!a.query_start) {
        const int per = (int)(((long long)a.N * a.G + kRows - 1) / kRows);
        b = tile / per;
        row = (tile - b * per) * kRows;
        if (b >= a.B) b = -1;
        return;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int base = 0; base < a.B; base += 32) {
        int q0, n = 0;
        if (base + lane < a.B) queries_of(a, base + lane, q0, n);
        int sum = (int)(((long long)n * a.G + kRows - 1) / kRows);
        const int own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > tile);
        if (hit) {
            const int at = __ffs(hit) - 1;
            b = base + at;
            row = (tile - before - __shfl_sync(0xffffffffu, sum - own, at)) * kRows;
            return;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    b = -1;
    row = 0;
}

// Row tiles of kRows rows over all sequences: exact when padded, at most this many when packed.
inline long long row_tiles(int B, int N, int G, bool packed, int kRows) {
    const long long rows = (long long)N * G;
    return packed ? rows / kRows + B : B * ((rows + kRows - 1) / kRows);
}

int cross_tc_heads(int G);
bool cross_tc_sizes(bsa_dtype dtype, int D);
bsa_status cross_tc(const Cross& a, cudaStream_t st, bool* handled);
bsa_status cross_f32(const Cross& a, cudaStream_t st);
size_t cross_runs_bytes(int runs, int D);
bsa_status cross_rows(const Cross& a, int runs, cudaStream_t st, bool* handled);

}  // namespace bsa
