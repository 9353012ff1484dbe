// a15 rotary table, a16 rotation of q and k.
//
// "The token path": queries and keys reach the attention after the projections, a norm over each head and
// the rotation by their positions; these two kernels are that step, from the projection's layout to the one
// that the attention reads.
#include <algorithm>

#include "rotary.cuh"
#include "tc_ptx.cuh"

namespace bsa {

// ---------------------------------------------------------------- a15 table
//
// A frequency is held as turns a position in units of 2^-64, so the angle's fraction of a turn is the low 64
// bits of an integer product, of which the upper 32 are kept: exact to 2^-32 turns for any position, where a
// float32 product would have lost the angle of position 2^24 altogether.  The upper 32 bits are cut into quadrant
// and remainder, and only the remainder, an eighth of a turn at most, becomes a float.  Its sine and cosine are the
// first five and six terms of their series: what is left out is below 2e-9 of the one and 1.2e-10 of the other.
// A thread keeps the frequencies of four neighbouring pairs (of one, where P is no multiple of 4) and walks the
// tokens, whose positions it reads one token ahead.  At 115200 tokens x 64 pairs, 59 MB of writes, it takes 13.6 us
// (16.3 with other outputs each time) of the 8.9 that the copy rate allows: the arithmetic, not the writes, fills the issue
// slots (63 to 73%).
__device__ __forceinline__ void cos_sin(uint32_t high, uint32_t low, int32_t pos, float factor, float& c, float& s) {
    // 2^-32 turns: the product's upper half, of an unsigned and a signed factor
    const uint32_t t = high * (uint32_t)pos + __umulhi(low, (uint32_t)pos) - (pos < 0 ? low : 0u);
    const uint32_t quad = (t + (1u << 29)) >> 30;
    const float x = (float)(int32_t)(t - (quad << 30)) * 0x1p-31f;  // half turns, |x| <= 1/4
    constexpr double kPi = 3.14159265358979323846, kPi2 = kPi * kPi;
    const float y = x * x;
    float sn = fmaf(y, (float)(kPi * kPi2 * kPi2 * kPi2 * kPi2 / 362880), (float)(-kPi * kPi2 * kPi2 * kPi2 / 5040));
    sn = fmaf(sn, y, (float)(kPi * kPi2 * kPi2 / 120));
    sn = fmaf(sn, y, (float)(-kPi * kPi2 / 6));
    sn = fmaf(sn * y, x, x * (float)kPi);
    float cs = fmaf(y, (float)(-kPi2 * kPi2 * kPi2 * kPi2 * kPi2 / 3628800), (float)(kPi2 * kPi2 * kPi2 * kPi2 / 40320));
    cs = fmaf(cs, y, (float)(-kPi2 * kPi2 * kPi2 / 720));
    cs = fmaf(cs, y, (float)(kPi2 * kPi2 / 24));
    cs = fmaf(cs, y, (float)(-kPi2 / 2));
    cs = fmaf(cs, y, 1.f);
    const float a = quad & 1 ? sn : cs, b = quad & 1 ? cs : sn;
    // minus signs: of the cosine in quadrants 1 and 2, of the sine in 2 and 3
    c = __uint_as_float(__float_as_uint(a * factor) ^ (quad + 1) >> 1 << 31);
    s = __uint_as_float(__float_as_uint(b * factor) ^ quad >> 1 << 31);
}

template <int V>
__global__ void __launch_bounds__(256) rotary_table_kernel(const int32_t* __restrict__ positions, int axes,
                                                           const int64_t* __restrict__ turns,
                                                           const int32_t* __restrict__ axis, int P, float factor,
                                                           float* __restrict__ cos_out, float* __restrict__ sin_out,
                                                           int T, int* status) {
    const int per = P / V, tokens = 256 / per;  // threads a token, tokens a block
    const int p = (int)(threadIdx.x % per) * V;
    uint32_t high[V], low[V];
    int ax[V];
    bool one = true;  // all pairs go by the same axis
#pragma unroll
    for (int j = 0; j < V; ++j) {
        high[j] = (uint32_t)((uint64_t)turns[p + j] >> 32);
        low[j] = (uint32_t)turns[p + j];
        ax[j] = axis ? axis[p + j] : 0;
        if ((unsigned)ax[j] >= (unsigned)axes) {
            raise_status(status, BSA_ERR_INDEX);
            ax[j] = 0;
        }
        one = one && ax[j] == ax[0];
    }
    if ((int)threadIdx.x >= tokens * per) return;
    const long long stride = (long long)gridDim.x * tokens;
    int32_t next[V];  // the next token's positions, read while this one's angles are taken
    auto read = [&](long long t) {
        if (t >= T) return;
        const int32_t* at = positions + t * axes;
        next[0] = at[ax[0]];
#pragma unroll
        for (int j = 1; j < V; ++j) next[j] = one ? next[0] : at[ax[j]];
    };
    const long long first = (long long)blockIdx.x * tokens + threadIdx.x / per;
    read(first);
    for (long long t = first; t < T; t += stride) {
        float c[V], s[V];
        int32_t pos[V];
#pragma unroll
        for (int j = 0; j < V; ++j) pos[j] = next[j];
        read(t + stride);
#pragma unroll
        for (int j = 0; j < V; ++j) cos_sin(high[j], low[j], pos[j], factor, c[j], s[j]);
        const long long to = t * P + p;
        if constexpr (V == 4) {
            *reinterpret_cast<float4*>(cos_out + to) = make_float4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<float4*>(sin_out + to) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            cos_out[to] = c[0];
            sin_out[to] = s[0];
        }
    }
}

// ---------------------------------------------------------------- a16 rotate
//
// A row of D channels is cut into units of 8: two runs of 4 channels that a lane reads at once and whose pairs lie
// inside the unit.  Half layout: pair i is (i, i + P), unit u < P / 4 holds channels 4u .. and P + 4u ..; the rest of
// the row, 8 at a time, is copied.  Interleaved layout: pair i is (2i, 2i + 1), unit u holds channels 8u .. 8u + 7.
// In both, unit u turns by the table's entries 4u .. 4u + 3.

// Four channels as they lie in memory (8- or 16-byte aligned), and as floats.
template <typename T> struct Run4;
template <> struct Run4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void floats(float* x) const {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <> struct Run4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void floats(float* x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
// Lanes that share a row of D channels: a power of two, 8 channels each.
__host__ __device__ constexpr int row_lanes(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Rows of `heads` heads to rotate, x into y (which may be x).
struct RowSet {
    const void* x;
    void* y;
    const float* weight;
    long long xb, xt, xh, yb, yt, yh;  // strides in elements: batch, token, head
    int heads;
};

// One token's heads [h0, h1) by a warp, 32 / kLanes rows a step; the lane's table entries stay in registers over them.
// The rows of kBatch steps are read before the first of them is written (y may be x: the compiler cannot move a read
// over a write).  What bounds it is the read and the write of every row once, so it is made for many bytes on their
// way at 64 registers: units of 8 channels, weights from L1.  (115200 tokens of 24 + 24 heads of 128 channels with a
// norm: units of 16 channels took 561 to 1000 us, by registers or spills; rows copied ahead into shared memory with
// 8 warps an SM 982; this one 489, 87% of the copy rate.)
template <typename T, int kLanes, bool kNorm, bool kInterleaved>
__device__ __forceinline__ void rotate_heads(const float* weight, const T* x, T* y, long long xh, long long yh, int h0,
                                             int h1, int D, int P, const float* c, const float* s, float eps) {
    constexpr int kRows = 32 / kLanes, kBatch = sizeof(T) == 2 ? 3 : 2;
    const int lane = threadIdx.x & 31, u = lane % kLanes, own = lane / kLanes;
    const bool live = 8 * u < D, turn = 4 * u < P;
    const int c0 = kInterleaved ? 8 * u : turn ? 4 * u : 2 * P + 8 * (u - P / 4), c1 = !kInterleaved && turn ? P + 4 * u : c0 + 4;
    x += (h0 + own) * xh + c0;
    y += (h0 + own) * yh + c0;
    const int d = c1 - c0;
    for (int h = h0; h < h1; h += kRows * kBatch) {
        Run4<T> a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (live && h + i * kRows + own < h1) {
                a[i].load(x);
                b[i].load(x + d);
            }
            x += kRows * xh;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (h + i * kRows >= h1) break;  // whole warps: shuffles below
            const bool on = live && h + i * kRows + own < h1;
            float z[8];
            a[i].floats(z);
            b[i].floats(z + 4);
            if (kNorm) {
                float ss = 0.f;
                if (on) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(z[e], z[e], ss);
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float n = rsqrtf(__fdividef(ss, (float)D) + eps);
                if (on) {
                    const float4 w0 = *reinterpret_cast<const float4*>(weight + c0), w1 = *reinterpret_cast<const float4*>(weight + c1);
                    z[0] *= n * w0.x, z[1] *= n * w0.y, z[2] *= n * w0.z, z[3] *= n * w0.w;
                    z[4] *= n * w1.x, z[5] *= n * w1.y, z[6] *= n * w1.z, z[7] *= n * w1.w;
                }
            }
            if (on) {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kInterleaved) rotate_pair(z[2 * e], z[2 * e + 1], c[e], s[e]);
                        else rotate_pair(z[e], z[4 + e], c[e], s[e]);
                    }
                }
                store4(y, z);
                store4(y + d, z + 4);
            }
            y += kRows * yh;
        }
    }
}

struct Rotate {
    RowSet set[2];
    const float* cos;
    const float* sin;
    long long table_batch;
    int T, D, P, splits;
    long long items;  // B * T * splits
    float eps;
    bool interleaved, transpose;
};

// Blocks y = 0 take q, y = 1 k: apart, a warp has fewer registers to hold.
template <typename T, int kLanes, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(256, 4) rotate_kernel(const Rotate a) {
    const int u = (threadIdx.x & 31) % kLanes;
    const RowSet& r = a.set[blockIdx.y];
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < a.items; i += (long long)gridDim.x * 8) {
        const long long tok = a.splits > 1 ? i / a.splits : i, b = tok < a.T ? 0 : tok / a.T, t = tok - b * a.T;
        const int part = (int)(i - tok * a.splits);
        float c[4], s[4];
        if (4 * u < a.P) {
            const long long at = b * a.table_batch + t * a.P + 4 * u;
            const float4 x = *reinterpret_cast<const float4*>(a.cos + at), y = *reinterpret_cast<const float4*>(a.sin + at);
            const float f = a.transpose ? -1.f : 1.f;
            c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
            s[0] = f * y.x, s[1] = f * y.y, s[2] = f * y.z, s[3] = f * y.w;
        }
        const int h0 = (int)((long long)r.heads * part / a.splits), h1 = (int)((long long)r.heads * (part + 1) / a.splits);
        const T* x = (const T*)r.x + b * r.xb + t * r.xt;
        T* y = (T*)r.y + b * r.yb + t * r.yt;
        if (kNorm && r.weight) rotate_heads<T, kLanes, true, kInterleaved>(r.weight, x, y, r.xh, r.yh, h0, h1, a.D, a.P, c, s, a.eps);
        else rotate_heads<T, kLanes, false, kInterleaved>(nullptr, x, y, r.xh, r.yh, h0, h1, a.D, a.P, c, s, 0.f);
    }
}

template <typename T, int kLanes>
static void start_rotate(const Rotate& a, dim3 grid, cudaStream_t st) {
    const bool norm = a.set[0].weight || a.set[1].weight;
    if (norm && a.interleaved) rotate_kernel<T, kLanes, true, true><<<grid, 256, 0, st>>>(a);
    else if (norm) rotate_kernel<T, kLanes, true, false><<<grid, 256, 0, st>>>(a);
    else if (a.interleaved) rotate_kernel<T, kLanes, false, true><<<grid, 256, 0, st>>>(a);
    else rotate_kernel<T, kLanes, false, false><<<grid, 256, 0, st>>>(a);
}

// Any D up to 256, any number of pairs, any strides: a channel a lane at a time (kJ of them), a token's heads by a warp,
// whose table entries, weights and partners' places stay in registers over them.  The rows of two heads are read before
// the first of them is written (y may be x).  Its instructions bound it (issue slots 66%, L2 14%): 115200 tokens of
// 24 + 24 heads of 128 bf16 channels, 63 pairs, with a norm take 1325 us, interleaved 1535 (a warp a row 3470 and 4145,
// four heads at a time 1900 and 1970, at 64 registers 1545 and 1874), where the wide kernel takes 489 for 64 pairs;
// float32, D = 64, 66% of the copy rate.  64 tokens of 64 + 4 heads take 5.2, and 4.4 with a warp a row: the host's call
// is three times that.
template <typename T, int kJ>
__global__ void __launch_bounds__(256) rotate_any_kernel(const Rotate a) {
    constexpr int kBatch = 2;
    const int lane = threadIdx.x & 31;
    const RowSet& r = a.set[blockIdx.y];
    int other[kJ];
    bool first[kJ];
    float w[kJ], wo[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int ch = lane + 32 * j;
        first[j] = a.interleaved ? !(ch & 1) : ch < a.P;
        other[j] = ch >= 2 * a.P ? ch : a.interleaved ? ch ^ 1 : first[j] ? ch + a.P : ch - a.P;
        w[j] = r.weight && ch < a.D ? r.weight[ch] : 1.f;
        wo[j] = r.weight && ch < a.D ? r.weight[other[j]] : 1.f;
    }
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < a.items; i += (long long)gridDim.x * 8) {
        const long long tok = a.splits > 1 ? i / a.splits : i, b = tok < a.T ? 0 : tok / a.T, t = tok - b * a.T;
        const int part = (int)(i - tok * a.splits);
        const long long at = b * a.table_batch + t * a.P;
        float c[kJ], s[kJ];  // s: with the sign of the sum, -fl(x s) being fl(x (-s))
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int ch = lane + 32 * j;
            if (ch >= 2 * a.P) continue;
            const int p = a.interleaved ? ch >> 1 : first[j] ? ch : ch - a.P;
            c[j] = a.cos[at + p];
            s[j] = first[j] != a.transpose ? -a.sin[at + p] : a.sin[at + p];
        }
        const int h0 = (int)((long long)r.heads * part / a.splits), h1 = (int)((long long)r.heads * (part + 1) / a.splits);
        const T* x = (const T*)r.x + b * r.xb + t * r.xt;
        T* y = (T*)r.y + b * r.yb + t * r.yt;
        for (int h = h0; h < h1; h += kBatch) {
            float v[kBatch][kJ], o[kBatch][kJ];
#pragma unroll
            for (int n = 0; n < kBatch; ++n)
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    v[n][j] = o[n][j] = 0.f;
                    if (h + n < h1 && lane + 32 * j < a.D) {
                        v[n][j] = to_f32(x[(h + n) * r.xh + lane + 32 * j]);
                        o[n][j] = to_f32(x[(h + n) * r.xh + other[j]]);
                    }
                }
            __syncwarp();
#pragma unroll
            for (int n = 0; n < kBatch; ++n) {
                if (h + n >= h1) break;
                if (r.weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) ss = fmaf(v[n][j], v[n][j], ss);
                    const float norm = rsqrtf(warp_sum(ss) / a.D + a.eps);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) v[n][j] *= norm * w[j], o[n][j] *= norm * wo[j];
                }
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int ch = lane + 32 * j;
                    if (ch >= a.D) break;
                    const float z = ch < 2 * a.P ? __fadd_rn(__fmul_rn(v[n][j], c[j]), __fmul_rn(o[n][j], s[j])) : v[n][j];
                    y[(h + n) * r.yh + ch] = from_f32<T>(z);
                }
            }
        }
    }
}

template <typename T>
static bsa_status launch_rotate(Rotate& a, long long tokens, bool wide, cudaStream_t st) {
    const auto blocks = [](long long warps) { return (unsigned)std::min<long long>((warps + 7) / 8, 152 * 64); };
    const int most = std::max(a.set[0].heads, a.set[1].heads), lanes = row_lanes(a.D);
    const int steps = wide ? (most * lanes + 31) / 32 : (most + 1) / 2;  // of a token
    // a share of the heads to a warp where there are few tokens
    a.splits = (int)std::max<long long>(1, std::min<long long>(steps, 152 * 32 / std::max<long long>(tokens, 1)));
    a.items = tokens * a.splits;
    const dim3 grid(blocks(a.items), a.set[1].heads ? 2 : 1);
    if (!wide) {
        if (a.D <= 64) rotate_any_kernel<T, 2><<<grid, 256, 0, st>>>(a);
        else if (a.D <= 128) rotate_any_kernel<T, 4><<<grid, 256, 0, st>>>(a);
        else rotate_any_kernel<T, 8><<<grid, 256, 0, st>>>(a);
        return check_launch("rotate_any_kernel");
    }
    if (lanes == 4) start_rotate<T, 4>(a, grid, st);
    else if (lanes == 8) start_rotate<T, 8>(a, grid, st);
    else if (lanes == 16) start_rotate<T, 16>(a, grid, st);
    else start_rotate<T, 32>(a, grid, st);
    return check_launch("rotate_kernel");
}

}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsa_rotary_table(const int32_t* positions, int T, int axes, const int64_t* turns, const int32_t* axis,
                            int P, float factor, float* cos_out, float* sin_out, void* stream) {
    BSA_REQUIRE(T >= 0 && axes >= 1 && axes <= 8 && P >= 1 && P <= 128,
                "rotary table: sizes out of range (T=%d axes=%d P=%d)", T, axes, P);
    BSA_REQUIRE(turns && (T == 0 || (positions && cos_out && sin_out)), "rotary table: null pointer");
    BSA_REQUIRE(axes == 1 || axis, "rotary table: several axes need an axis for each frequency");
    if (T == 0) return BSA_OK;
    const bool wide = P % 4 == 0 && (((uintptr_t)cos_out | (uintptr_t)sin_out) & 15) == 0;
    const int tokens = 256 / (wide ? P / 4 : P);
    const unsigned grid = (unsigned)std::min<long long>(((long long)T + tokens - 1) / tokens, 152 * 5);
    cudaStream_t st = as_stream(stream);
    if (wide)
        rotary_table_kernel<4><<<grid, 256, 0, st>>>(positions, axes, turns, axis, P, factor, cos_out, sin_out, T,
                                                     status_word());
    else
        rotary_table_kernel<1><<<grid, 256, 0, st>>>(positions, axes, turns, axis, P, factor, cos_out, sin_out, T,
                                                     status_word());
    return check_launch("rotary_table_kernel");
}

bsa_status bsa_rotate(bsa_dtype dtype, int B, int T, int D, int P, int interleaved, int transpose,
                      const float* cos_table, const float* sin_table, int64_t table_batch_stride, const void* q, int HQ,
                      const float* q_weight, void* q_out, const void* k, int H, const float* k_weight, void* k_out,
                      const int64_t* strides, float eps, void* stream) {
    BSA_REQUIRE(dtype == BSA_F32 || dtype == BSA_BF16, "rotate: dtype");
    BSA_REQUIRE(B >= 0 && T >= 0 && D >= 2 && D <= 256 && P >= 1 && 2 * P <= D && HQ >= 1 && HQ <= (1 << 20) && H >= 0 &&
                    H <= (1 << 20),
                "rotate: sizes out of range (B=%d T=%d D=%d P=%d HQ=%d H=%d)", B, T, D, P, HQ, H);
    BSA_REQUIRE(strides, "rotate: null strides");
    if (B == 0 || T == 0) return BSA_OK;
    BSA_REQUIRE(cos_table && sin_table && q && q_out && (H == 0 || (k && k_out)), "rotate: null pointer");
    BSA_REQUIRE(table_batch_stride >= 0, "rotate: the table's batch stride must not be negative");
    BSA_REQUIRE(!transpose || (!q_weight && !k_weight), "rotate: the transposed rotation takes no norm");
    BSA_REQUIRE(!(q_weight || k_weight) || (eps >= 0.f && eps <= 1.f), "rotate: eps must lie in [0, 1]");
    Rotate a{};
    const void* in[2] = {q, k};
    void* out[2] = {q_out, k_out};
    const float* weight[2] = {q_weight, k_weight};
    const int heads[2] = {HQ, H};
    const int size = dtype == BSA_F32 ? 4 : 2;
    const uintptr_t run = 4 * size - 1;  // runs of four channels
    bool wide = D % 8 == 0 && P % 4 == 0 && (((uintptr_t)cos_table | (uintptr_t)sin_table) & 15) == 0 &&
                table_batch_stride % 4 == 0;
    for (int n = 0; n < 2; ++n) {
        const int64_t* s = strides + 6 * n;
        a.set[n] = RowSet{in[n], out[n], weight[n], s[0], s[1], s[2], s[3], s[4], s[5], heads[n]};
        if (!heads[n]) continue;
        BSA_REQUIRE(in[n] != out[n] || ((B == 1 || s[0] == s[3]) && (T == 1 || s[1] == s[4]) && (heads[n] == 1 || s[2] == s[5])),
                    "rotate: an output over its input needs the same strides, others must not overlap");
        BSA_REQUIRE(H == 0 || (out[n] != in[1 - n] && out[0] != out[1]), "rotate: outputs must not overlap the other tensor");
        uintptr_t any = (uintptr_t)in[n] | (uintptr_t)out[n];
        for (int j = 0; j < 6; ++j) any |= (uintptr_t)(s[j] * size);
        wide = wide && (any & run) == 0 && ((uintptr_t)weight[n] & 15) == 0;
    }
    a.cos = cos_table;
    a.sin = sin_table;
    a.table_batch = table_batch_stride;
    a.T = T;
    a.D = D;
    a.P = P;
    a.eps = eps;
    a.interleaved = interleaved != 0;
    a.transpose = transpose != 0;
    cudaStream_t st = as_stream(stream);
    const long long tokens = (long long)B * T;
    return dtype == BSA_F32 ? launch_rotate<float>(a, tokens, wide, st)
                            : launch_rotate<__nv_bfloat16>(a, tokens, wide, st);
}

}  // extern "C"
