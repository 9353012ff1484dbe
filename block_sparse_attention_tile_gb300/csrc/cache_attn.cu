// Attention over the 4-bit paged cache (a14): arguments, and the CUDA-core kernel.
#include "cache_attn.cuh"

namespace bsa {

// One CTA per (token, KV head, tile of 16 query heads), one strip of 16 keys at a
// time: its K and V are unpacked to float32 in shared memory, the scores, the running
// maximum and sum and the output stay in float32.  For any D that the layout allows, and
// the form that the tensor-core kernel is checked against.
constexpr int kHeadTile = 16;

template <typename T>
__global__ void __launch_bounds__(128) cache_attn_simt_kernel(CacheAttn a) {
    __shared__ float Q[kHeadTile][128], K[kStrip][129], V[kStrip][128], Pm[kHeadTile][kStrip];
    __shared__ float m[kHeadTile], l[kHeadTile], corr[kHeadTile];
    const int tid = threadIdx.x, D = a.D, G = a.HQ / a.H, tiles = (G + kHeadTile - 1) / kHeadTile;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % a.H, t = blockIdx.x / tiles / a.H;
    const int heads = min(kHeadTile, G - tile * kHeadTile), hq0 = h * G + tile * kHeadTile;
    const Row row = row_of(a, t, h, tid == 0);
    if (row.req < 0) return;
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (long long)hq0 * D;
    for (int i = tid; i < heads * D; i += 128) Q[i / D][i % D] = to_f32(q[i]);
    if (tid < kHeadTile) m[tid] = -INFINITY, l[tid] = 0.f;
    float o[kHeadTile];
#pragma unroll
    for (int i = 0; i < kHeadTile; ++i) o[i] = 0.f;
    const float ks = (a.k_scale ? a.k_scale[h] : 1.f) * a.scale_log2, vs = a.v_scale ? a.v_scale[h] : 1.f;
    for (int n = 0; n < row.strips; ++n) {
        const int first = first_key(a, row, n, tid == 0);
        if (first < 0) continue;
        const int index = strip_index(a, row, h, first, tid == 0);
        if (index < 0) continue;
        const uint8_t* strip = a.cache + (long long)index * strip_bytes(D);
        const int seen = min(kStrip, row.pos - first + 1);
        __syncthreads();
        for (int i = tid; i < kStrip * D; i += 128) {
            const int j = i / D, c = i % D;
            const uint32_t kb = strip[j * (D / 2) + c / 2], vb = strip[8 * D + (c / 16 * 16 + j) * 8 + c % 16 / 2];
            const uint32_t kc = c & 1 ? kb >> 4 : kb & 15, vc = c & 1 ? vb >> 4 : vb & 15;
            K[j][c] = f16x2_to_f32(e2m1x2_to_f16x2(kc)).x *
                      f16x2_to_f32(e4m3x2_to_f16x2(strip[16 * D + j * (D / 16) + c / 16])).x;
            // keys that the token does not see may hold anything: their values are not looked at
            V[j][c] = j < seen ? f16x2_to_f32(e2m1x2_to_f16x2(vc)).x *
                                     f16x2_to_f32(e4m3x2_to_f16x2(strip[17 * D + c / 16 * 16 + j])).x
                               : 0.f;
        }
        __syncthreads();
        for (int i = tid; i < heads * kStrip; i += 128) {
            const int r = i / kStrip, j = i % kStrip;
            float s = 0.f;
            for (int c = 0; c < D; ++c) s = fmaf(Q[r][c], K[j][c], s);
            Pm[r][j] = j < seen ? s * ks : -INFINITY;
        }
        __syncthreads();
        if (tid < heads) {
            float top = m[tid];
            for (int j = 0; j < seen; ++j) top = fmaxf(top, Pm[tid][j]);
            const float base = top == -INFINITY ? 0.f : top;
            corr[tid] = exp2f(m[tid] - base);
            float sum = 0.f;  // of the strip first, so that a long row's sums take a sixteenth of the roundings
            for (int j = 0; j < kStrip; ++j) {
                const float p = exp2f(Pm[tid][j] - base);
                Pm[tid][j] = p;
                sum += p;
            }
            m[tid] = top;
            l[tid] = fmaf(l[tid], corr[tid], sum);
        }
        __syncthreads();
        if (tid < D)
            for (int r = 0; r < heads; ++r) {
                float x = 0.f;
                for (int j = 0; j < kStrip; ++j) x = fmaf(Pm[r][j], V[j][tid], x);
                o[r] = fmaf(o[r], corr[r], x);
            }
    }
    __syncthreads();
    T* out = static_cast<T*>(a.out) + ((long long)t * a.HQ + hq0) * D;
    if (tid < D)
        for (int r = 0; r < heads; ++r) out[(long long)r * D + tid] = from_f32<T>(l[r] > 0.f || l[r] != l[r] ? o[r] / l[r] * vs : 0.f);
    if (a.lse && tid < heads)
        a.lse[(long long)t * a.HQ + hq0 + tid] = l[tid] == 0.f ? -INFINITY : (m[tid] + log2f(l[tid])) * kLn2;
}

static bsa_status simt_cache_attention(const CacheAttn& a, bsa_dtype dtype, cudaStream_t st) {
    const long long grid = (long long)a.T * a.H * ((a.HQ / a.H + kHeadTile - 1) / kHeadTile);
    if (grid > 0x7fffffffLL) return fail(BSA_ERR_UNSUPPORTED, "cache attention: too many (token, head) rows");
    if (dtype == BSA_F32) cache_attn_simt_kernel<float><<<(unsigned)grid, 128, 0, st>>>(a);
    else cache_attn_simt_kernel<__nv_bfloat16><<<(unsigned)grid, 128, 0, st>>>(a);
    return check_launch("cache_attn_simt_kernel");
}

static bool on_tensor_cores(int D) { return D == 64 || D == 128; }

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsa_cache_attention_workspace(int T, int HQ, int H, int D, int max_keys) {
    if (T < 1 || H < 1 || HQ < 1 || HQ % H || max_keys < 1 || !on_tensor_cores(D)) return 0;
    return mma_cache_attention_workspace(T, HQ, H, D, max_keys);
}

int bsa_cache_attention_way(int T, int HQ, int H, int D, bsa_dtype dtype, int lists, int max_keys) {
    if (T < 1 || H < 1 || HQ < 1 || HQ % H || max_keys < 1 || D < 16 || D > 128 || D % 16) return -1;
    return on_tensor_cores(D) ? mma_cache_attention_way(T, HQ, H, D, dtype == BSA_F32, lists != 0, max_keys) : 0;
}

bsa_status bsa_fwd_cache_tokens(const void* q, bsa_dtype dtype, int T, int HQ, int H, int D, int64_t q_stride,
                                const void* cache, int n_pages, int page_size, const int32_t* block_table, int R,
                                int max_pages, const int32_t* token_req, const int32_t* token_pos,
                                const float* k_scale, const float* v_scale, const int32_t* block_indices,
                                const int32_t* block_counts, int S, int block_size, float scale, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream) {
    BSA_REQUIRE(cache && block_table && (T == 0 || (q && token_req && token_pos && out)), "cache attention: null pointer");
    BSA_REQUIRE(dtype == BSA_F32 || dtype == BSA_BF16, "cache attention: dtype");
    BSA_REQUIRE(T >= 0 && H > 0 && HQ > 0 && HQ % H == 0 && n_pages > 0 && R > 0 && max_pages > 0,
                "cache attention: sizes out of range (T=%d HQ=%d H=%d n_pages=%d R=%d max_pages=%d)", T, HQ, H, n_pages,
                R, max_pages);
    BSA_REQUIRE(page_size_ok(page_size), "cache attention: page_size must be a power of two in 16..1024, got %d",
                page_size);
    BSA_REQUIRE(D >= 16 && D <= 128 && D % 16 == 0, "cache attention: D must be a multiple of 16 up to 128, got %d", D);
    BSA_REQUIRE((long long)max_pages * page_size <= 0x7fffffffLL, "cache attention: max_pages * page_size must be below 2^31");
    BSA_REQUIRE(T <= 1 || q_stride >= (int64_t)HQ * D, "cache attention: a token's stride is below HQ * D");
    BSA_REQUIRE((((uintptr_t)cache | (uintptr_t)out) & 15) == 0, "cache attention: cache and out must be 16-byte aligned");
    BSA_REQUIRE(T == 0 || (block_indices == nullptr) == (block_counts == nullptr),
                "cache attention: block_indices and block_counts come together");
    BSA_REQUIRE(!block_indices || (S > 0 && block_size > 0 && (long long)S * block_size <= 0x7fffffffLL),
                "cache attention: block lists need S and block_size");
    if (block_indices && block_size % kStrip)
        return fail(BSA_ERR_UNSUPPORTED, "cache attention: block_size must be a multiple of 16, got %d", block_size);
    BSA_REQUIRE(((long long)n_pages * H << (log2i(page_size) - 4)) <= 0x7fffffffLL, "cache attention: too many strips");
    const long long max_keys = block_indices ? (long long)S * block_size : (long long)max_pages * page_size;
    const size_t need = bsa_cache_attention_workspace(T, HQ, H, D, (int)max_keys);
    BSA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && ((uintptr_t)workspace & 31) == 0),
                "cache attention: a 32-byte aligned workspace of %zu bytes is needed", need);
    if (T == 0) return BSA_OK;
    CacheAttn a;
    a.q = q, a.T = T, a.HQ = HQ, a.H = H, a.D = D, a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache), a.n_pages = n_pages, a.sh = log2i(page_size);
    a.table = block_table, a.R = R, a.max_pages = max_pages, a.req = token_req, a.pos = token_pos;
    a.k_scale = k_scale, a.v_scale = v_scale, a.blocks = block_indices, a.counts = block_counts;
    a.S = block_indices ? S : 0, a.block_strips = block_indices ? block_size / kStrip : 0;
    a.scale_log2 = scale * kLog2e, a.out = out, a.lse = lse, a.status = status_word();
    if (on_tensor_cores(D) && !force_simt()) return mma_cache_attention(a, dtype, max_keys, workspace, as_stream(stream));
    return simt_cache_attention(a, dtype, as_stream(stream));
}

}  // extern "C"
