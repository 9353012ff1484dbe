// The paged cache's tables (a12) and the write of new rows into it (a13).
#include <algorithm>

#include "cache.cuh"
#include "tc_ptx.cuh"

namespace bsa {

// ---------------------------------------------------------------- a12 tables
//
// Exclusive sums over the requests of (new tokens, pages taken, pages given back)
// place everything: token i of request r goes to row start[r] + i, its k-th new
// page is page take[r] + k of the call, and so on.  The pool is a stack of free
// pages: the call's given-back pages are pushed, last request's last page first, and its
// new pages popped one by one.  Both are only index arithmetic on the "virtual
// stack" pool[0 .. count) + given-back pages, so every new page is known without
// waiting for any write of the call, and no two threads touch the same word.
//
// Nothing here computes; a small call is bound by the launch and the scan's
// latency (64 requests of one token: 4.8 us on the device), a large one by its two
// launches and the dependent lookups of each page (1024 mixed requests, 786432 token
// rows, 12.8 MB: 12 us, of which the bytes are 2).

struct Tables {
    const int32_t* old_lens;
    int32_t* new_lens;
    int R, P, max_pages, n_pages, max_tokens;
    int32_t *table, *pool;
    const int32_t* count;
    int32_t *count_out, *start, *req, *pos;
    int64_t* slots;
    int* status;
    bool wide;  // the token arrays are 16-byte aligned
};

// What the second half of the work needs of the scan: in shared memory when one
// CTA does everything, in the workspace when a grid follows.
struct Sums {
    int32_t *start, *take, *give;  // R + 1 each
    const int32_t *old_lens, *new_lens;
    int ok, count, taken, given, total;
};

constexpr int kScanThreads = 1024;
// Up to here one CTA does all: 4 tokens a thread cost less than a second launch.  The pages given back count nothing
// here, since the host does not know them: many long requests that end at once take longer in one CTA (64 of 512 pages
// 23 us, in a grid 6; 1024 of 128 pages 115 against 15).
constexpr int kOneCtaTokens = 4096;
constexpr int kOneCtaRequests = 1024;
inline bool one_cta(int R, int max_tokens) { return R <= kOneCtaRequests && max_tokens <= kOneCtaTokens; }

__device__ __forceinline__ int pages_of(int len, int sh) { return (int)(((unsigned)len + (1u << sh) - 1) >> sh); }

// The largest r in [0, R) with sums[r] <= i (sums ascending, sums[R] > i).
__device__ __forceinline__ int owner(const int32_t* sums, int R, int i) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Page at a position of the virtual stack.
__device__ __forceinline__ int stack_page(const Tables& a, const Sums& s, int sh, int at) {
    if (at < s.count) return a.pool[at];
    const int i = s.given - 1 - (at - s.count);
    const int r = owner(s.give, a.R, i);
    return a.table[(long long)r * a.max_pages + pages_of(s.new_lens[r], sh) + i - s.give[r]];
}

// Token rows, kPer consecutive ones a thread: one where each is likely to be another request's (a decode step), four
// where they mostly share request and page and the 16 bytes written for each count.
template <int kPer>
__device__ void place_tokens(const Tables& a, const Sums& s, int sh, unsigned tid, unsigned stride) {
    const unsigned live = s.ok ? s.total : 0, most = a.max_tokens;
    for (unsigned i0 = tid * kPer; i0 < most; i0 += stride * kPer) {
        int req[kPer], pos[kPer];
        int64_t slot[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) req[k] = pos[k] = -1, slot[k] = -1;
        if (i0 < live) {
            int r = owner(s.start, a.R, i0), end = s.start[r + 1], old = s.old_lens[r], held = -1, page = 0;
            int p = old + (int)i0 - s.start[r];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (i0 + k >= live) break;
                if ((int)i0 + k >= end) {  // the next request with new tokens
                    while (s.start[r + 1] <= (int)i0 + k) ++r;
                    end = s.start[r + 1], p = old = s.old_lens[r], held = -1;
                }
                const int j = p >> sh;
                if (j != held) {
                    const int before = pages_of(old, sh);
                    page = j < before ? a.table[(long long)r * a.max_pages + j]
                                      : stack_page(a, s, sh, s.count + s.given - 1 - (s.take[r] + j - before));
                    held = j;
                }
                req[k] = r, pos[k] = p;
                if ((unsigned)page < (unsigned)a.n_pages) slot[k] = ((int64_t)page << sh) + (p & (a.P - 1));
                else raise_status(a.status, BSA_ERR_INDEX);
                ++p;
            }
        }
        if (kPer == 4 && a.wide && i0 + 4 <= most) {
            *reinterpret_cast<int4*>(a.req + i0) = make_int4(req[0], req[1 % kPer], req[2 % kPer], req[3 % kPer]);
            *reinterpret_cast<int4*>(a.pos + i0) = make_int4(pos[0], pos[1 % kPer], pos[2 % kPer], pos[3 % kPer]);
            reinterpret_cast<longlong2*>(a.slots + i0)[0] = make_longlong2(slot[0], slot[1 % kPer]);
            reinterpret_cast<longlong2*>(a.slots + i0)[1] = make_longlong2(slot[2 % kPer], slot[3 % kPer]);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (i0 + k < most) a.req[i0 + k] = req[k], a.pos[i0 + k] = pos[k], a.slots[i0 + k] = slot[k];
        }
    }
}

// New table entries and pages pushed.
__device__ void place_pages(const Tables& a, const Sums& s, int sh, unsigned tid, unsigned stride) {
    if (!s.ok) return;
    for (unsigned i = tid; i < (unsigned)s.taken; i += stride) {
        const int r = owner(s.take, a.R, i);
        a.table[(long long)r * a.max_pages + pages_of(s.old_lens[r], sh) + i - s.take[r]] =
            stack_page(a, s, sh, s.count + s.given - 1 - i);
    }
    const int pushed = s.given - s.taken;
    for (int i = (int)tid; i < pushed; i += (int)stride) {  // pushed <= n_pages
        const int page = stack_page(a, s, sh, s.count + i);
        if ((unsigned)page >= (unsigned)a.n_pages) raise_status(a.status, BSA_ERR_INDEX);
        a.pool[s.count + i] = page;
    }
}

// One CTA: the three exclusive sums, the checks, the new count; with kAll the rest too.
template <bool kAll>
__global__ void __launch_bounds__(kScanThreads) cache_scan_kernel(Tables a, int sh, int32_t* ws) {
    extern __shared__ int32_t dyn[];
    __shared__ long long part[3][32];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!kAll) asm volatile("griddepcontrol.launch_dependents;");
    Sums s;
    s.start = kAll ? dyn : a.start;
    s.take = kAll ? dyn + (a.R + 1) : ws ? ws + 8 : nullptr;  // without a workspace nobody asks for these sums
    s.give = s.take ? s.take + (a.R + 1) : nullptr;
    s.old_lens = a.old_lens, s.new_lens = a.new_lens;
    if (tid == 0) bad = 0;
    s.count = a.count[0];
    __syncthreads();
    // token sums in 64 bits: R requests of up to 2^31 tokens; page sums fit 32 (R * max_pages < 2^31)
    long long run[3] = {0, 0, 0};
    const long long longest = (long long)a.max_pages << sh;
    for (int base = 0; base < a.R; base += kScanThreads) {
        const int r = base + tid;
        long long x[3] = {0, 0, 0};
        if (r < a.R) {
            const int o = a.old_lens[r], n = a.new_lens[r];
            if (o < 0 || n < 0 || o > longest || n > longest) {
                bad = 1;
            } else {
                const int before = pages_of(o, sh), after = pages_of(n, sh);
                x[0] = max(0, n - o);
                x[1] = max(0, after - before);
                x[2] = max(0, before - after);
            }
        }
        long long inc[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            inc[k] = x[k];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc[k], d);
                if (lane >= d) inc[k] += y;
            }
            if (lane == 31) part[k][warp] = inc[k];
        }
        __syncthreads();
        if (warp < 3) {
            long long y = part[warp][lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long z = __shfl_up_sync(0xffffffffu, y, d);
                if (lane >= d) y += z;
            }
            part[warp][lane] = y;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long before = run[k] + (warp ? part[k][warp - 1] : 0) + inc[k] - x[k];
            if (r < a.R && (k == 0 || s.take)) (k == 0 ? s.start : k == 1 ? s.take : s.give)[r] = (int32_t)min(before, 0x7fffffffLL);
            run[k] += part[k][31];
        }
        __syncthreads();
    }
    s.taken = (int)run[1];
    s.given = (int)run[2];
    s.total = (int)min(run[0], 0x7fffffffLL);
    int code = BSA_OK;
    if (bad || s.count < 0 || s.count > a.n_pages || (long long)s.count + s.given - s.taken > a.n_pages)
        code = BSA_ERR_INDEX;
    else if ((long long)s.count + s.given < s.taken || run[0] > a.max_tokens)
        code = BSA_ERR_CAPACITY;
    s.ok = code == BSA_OK;
    if (tid == 0) {
        s.start[a.R] = s.total;
        if (s.take) s.take[a.R] = s.taken, s.give[a.R] = s.given;
        a.count_out[0] = s.ok ? s.count + s.given - s.taken : s.count;
        if (!s.ok) raise_status(a.status, code);
        if (!kAll && ws) {
            ws[0] = s.ok;
            ws[1] = s.count;
            ws[2] = s.taken;
            ws[3] = s.given;
            ws[4] = s.total;
        }
    }
    __syncthreads();
    if (!s.ok)
        for (int r = tid; r < a.R; r += kScanThreads) a.new_lens[r] = a.old_lens[r];
    if (kAll) {
        for (int r = tid; r <= a.R; r += kScanThreads) a.start[r] = s.ok ? s.start[r] : 0;
        place_tokens<1>(a, s, sh, tid, kScanThreads);
        place_pages(a, s, sh, tid, kScanThreads);
    } else if (!s.ok) {
        for (int r = tid; r <= a.R; r += kScanThreads) a.start[r] = 0;
    }
}

// The rest of a large step: blocks of tokens, then blocks of pages.  kShared: every block sums the lengths again, into
// shared memory, where the ten or so dependent steps of a search cost a tenth of what they cost in L2 (and which needs
// no workspace).  It can, because the scan has set new_lens back where the call cannot be carried out: then nothing
// grows or shrinks, and every token row is -1.
constexpr int kSharedRequests = 2400;  // 5 * (R + 1) ints in 48 KB
constexpr int kPageBlocks = 32;

template <bool kShared>
__global__ void __launch_bounds__(256) cache_place_kernel(Tables a, int sh, const int32_t* ws) {
    extern __shared__ int32_t dyn[];
    __shared__ int part[3][8];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the scan still runs
    Sums s;
    if (kShared) {
        const int n = a.R + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        s.start = dyn, s.take = dyn + n, s.give = dyn + 2 * n, s.old_lens = dyn + 3 * n, s.new_lens = dyn + 4 * n;
        const int left = a.count_out[0], per = (a.R + 255) / 256, r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
        int sum[3] = {0, 0, 0}, before[3], all[3] = {0, 0, 0};
        for (int r = tid; r < a.R; r += 256) {
            dyn[3 * n + r] = a.old_lens[r];
            dyn[4 * n + r] = a.new_lens[r];
        }
        __syncthreads();
        auto add = [&](int r) {
            const int o = s.old_lens[r], w = s.new_lens[r], b = pages_of(o, sh), e = pages_of(w, sh);
            sum[0] += max(0, w - o), sum[1] += max(0, e - b), sum[2] += max(0, b - e);
        };
        for (int r = r0; r < r1; ++r) add(r);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            int inc = sum[k];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += y;
            }
            if (lane == 31) part[k][warp] = inc;
            before[k] = inc - sum[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w < warp) before[k] += part[k][w];
                all[k] += part[k][w];
            }
            sum[k] = before[k];
        }
        for (int r = r0; r < r1; ++r) {
            s.start[r] = sum[0], s.take[r] = sum[1], s.give[r] = sum[2];
            add(r);
        }
        if (tid == 0) s.start[a.R] = all[0], s.take[a.R] = all[1], s.give[a.R] = all[2];
        s.ok = 1, s.total = all[0], s.taken = all[1], s.given = all[2];
        s.count = left - s.given + s.taken;  // before the call
        __syncthreads();
    } else {
        s.start = a.start;
        s.take = const_cast<int32_t*>(ws) + 8;
        s.give = s.take + (a.R + 1);
        s.old_lens = a.old_lens, s.new_lens = a.new_lens;
        s.ok = ws[0];
        s.count = ws[1];
        s.taken = ws[2];
        s.given = ws[3];
        s.total = ws[4];
    }
    const int blocks = gridDim.x - kPageBlocks, b = blockIdx.x;
    if (b < blocks) place_tokens<4>(a, s, sh, b * 256 + threadIdx.x, blocks * 256);
    else place_pages(a, s, sh, (b - blocks) * 256 + threadIdx.x, kPageBlocks * 256);
}

// ---------------------------------------------------------------- a13 append
//
// A thread rounds one group of 16 channels of one token and head, for K and for V:
//   y = x * (1 / head scale),  s = E4M3(max |y| / 6),  code = E2M1(y / s).
// Both quotients are rounded once, to float32 (max / 6 by the division instruction's routine, y / s
// by Markstein's three steps from the rounded reciprocal of s): a quotient that is not a border of the short format is
// never moved onto one by that, because a float32 next to a product of border and scale leaves a quotient more than
// half a step away, so the codes are those of the exact quotient.  The largest |y| is the product of the largest |x|
// (products round monotonically), found on the inputs' bits: bf16 in pairs, and a group that
// holds a NaN or an infinity shows there.  It is stored with the scale NaN, so that it reads back as NaN and not as
// a finite number.
//
// Per element: 2 bytes read and 9/16 written (and 2 for the values), and about 20 instructions with the
// values: at 16.8M elements a tensor (32768 tokens, 153 MB) 28 us, 80% of the copy bandwidth, with the issue
// slots 63% busy.  Without the values 19.4 us for 86 MB (66%), where the instructions bind; float32 30 us without (76%)
// and 46 with them (93%).

// Sixteen elements as they lie in memory.
template <typename T> struct Group { uint32_t w[4 * sizeof(T)]; };

template <typename T, bool kVec>
__device__ __forceinline__ Group<T> load16(const T* p) {
    Group<T> x;
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
            x.w[4 * i] = a.x, x.w[4 * i + 1] = a.y, x.w[4 * i + 2] = a.z, x.w[4 * i + 3] = a.w;
        }
    } else if constexpr (sizeof(T) == 2) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.w[i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x.w[i] = __float_as_uint(to_f32(p[i]));
    }
    return x;
}
template <typename T>
__device__ __forceinline__ float element(const Group<T>& x, int i) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? x.w[i / 2] & 0xffff0000u : x.w[i / 2] << 16);
    else return __uint_as_float(x.w[i]);
}
template <typename T, bool kVec>
__device__ __forceinline__ void store16(T* p, const float* x) {
    if constexpr (kVec) {
        uint32_t w[4 * sizeof(T)];
#pragma unroll
        for (int i = 0; i < (int)(4 * sizeof(T)); ++i) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                w[i] = __float_as_uint(x[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) ptx::st_global_v8(p + i * 32 / sizeof(T), w + 8 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = from_f32<T>(x[i]);
    }
}

// Codes (8 bytes) and scale byte of a group; with kValues x becomes the group's stored values.
template <typename T, bool kValues>
__device__ __forceinline__ uint2 quantise16(const Group<T>& g, float head_scale, uint32_t* scale, float* x) {
    const float inv = __fdiv_rn(1.f, head_scale);
    uint32_t most = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) most = __vmaxu2(most, g.w[i] & 0x7fff7fffu);
        most = max(most << 16, most & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) most = max(most, g.w[i] & 0x7fffffffu);
    }
    const float top = __uint_as_float(most) * inv;
    const bool finite = most < 0x7f800000u && top <= 3.402823466e38f;
    const uint32_t sb = finite ? f32_to_e4m3(__fdiv_rn(top, kE2M1Max)) : 0x7fu;
    const uint32_t s16 = e4m3x2_to_f16x2(sb | sb << 8);  // (s, s)
    const float s = f16x2_to_f32(s16).x, r = s > 0.f ? __frcp_rn(s) : 0.f;  // a scale of zero stores zeros
    // Two at a time; adding -0 leaves a product as it is.  From -y, with -r: of y = -0 the remainder q0 s + (-y) is +0
    // and -r of it -0, so the quotient keeps its sign (y - q0 s would be +0, and +0 r + -0 is +0).
    const float2 inv2 = make_float2(-inv, -inv), r2 = make_float2(-r, -r), s2 = make_float2(s, s), none = make_float2(-0.f, -0.f);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 ny = ptx::ffma2(make_float2(element<T>(g, 2 * i), element<T>(g, 2 * i + 1)), inv2, none);
        const float2 q0 = ptx::ffma2(ny, r2, none), q = ptx::ffma2(ptx::ffma2(q0, s2, ny), r2, q0);
        const uint32_t two = f32x2_to_e2m1x2(q.x, q.y);
        w[i >> 2] |= two << (8 * (i & 3));
        if constexpr (kValues) {
            const uint32_t c = e2m1x2_to_f16x2(two);
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&c), *reinterpret_cast<const __half2*>(&s16));
            const float2 f = __half22float2(v);  // code * s is exact in float16
            const float2 z = ptx::ffma2(f, make_float2(head_scale, head_scale), none);
            x[2 * i] = z.x;
            x[2 * i + 1] = z.y;
        }
    }
    *scale = sb;
    return make_uint2(w[0], w[1]);
}

template <typename T, bool kVec, bool kValues>
__global__ void __launch_bounds__(256) cache_append_kernel(
    const T* __restrict__ k, const T* __restrict__ v, long long k_stride, long long v_stride, unsigned items, int H,
    int D, const int64_t* __restrict__ slots, uint8_t* __restrict__ cache, long long n_slots, int sh,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale, T* __restrict__ k_val, T* __restrict__ v_val,
    int* status) {
    const unsigned ng = D / 16;
    for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < items; i += gridDim.x * blockDim.x) {
        const unsigned row = i / ng, t = row / (unsigned)H;
        const int g = (int)(i - row * ng), h = (int)(row - t * H);
        const long long slot = slots[t];
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1) raise_status(status, BSA_ERR_INDEX);
            continue;
        }
        const Group<T> kx = load16<T, kVec>(k + t * k_stride + h * D + g * 16);
        const Group<T> vx = load16<T, kVec>(v + t * v_stride + h * D + g * 16);
        const float ks = k_scale ? k_scale[h] : 1.f, vs = v_scale ? v_scale[h] : 1.f;
        const long long page = slot >> sh, at = (long long)i * 16;
        const int in = (int)(slot & ((1 << sh) - 1)), j = in & 15;
        uint8_t* strip = cache + (((page * H + h) << (sh - 4)) + (in >> 4)) * strip_bytes(D);
        float x[16];
        uint32_t byte;
        *reinterpret_cast<uint2*>(strip + j * (D / 2) + g * 8) = quantise16<T, kValues>(kx, ks, &byte, x);
        strip[16 * D + j * ng + g] = (uint8_t)byte;
        if (kValues) store16<T, kVec>(k_val + at, x);
        *reinterpret_cast<uint2*>(strip + 8 * D + (g * 16 + j) * 8) = quantise16<T, kValues>(vx, vs, &byte, x);
        strip[17 * D + g * 16 + j] = (uint8_t)byte;
        if (kValues) store16<T, kVec>(v_val + at, x);
    }
}

template <typename T>
static bsa_status launch_append(const void* k, const void* v, long long ks, long long vs, int T_, int H, int D,
                                const int64_t* slots, uint8_t* cache, long long n_slots, int sh, const float* k_scale,
                                const float* v_scale, void* k_val, void* v_val, cudaStream_t st) {
    const long long items = (long long)T_ * H * (D / 16);
    if (items > (1LL << 31)) return fail(BSA_ERR_UNSUPPORTED, "cache append: too many rows (T=%d H=%d D=%d)", T_, H, D);
    const unsigned grid = (unsigned)std::min<long long>((items + 255) / 256, 1 << 20);  // i stays below 2^32
    const uintptr_t in = (uintptr_t)k | (uintptr_t)v | (uintptr_t)(ks * (long long)sizeof(T)) |
                         (uintptr_t)(vs * (long long)sizeof(T)), out = (uintptr_t)k_val | (uintptr_t)v_val;
    const bool vec = (in & 15) == 0 && (out & 31) == 0;
#define BSA_APPEND(V, W)                                                                                        \
    cache_append_kernel<T, V, W><<<grid, 256, 0, st>>>((const T*)k, (const T*)v, ks, vs, items, H, D, slots, cache, \
                                                       n_slots, sh, k_scale, v_scale, (T*)k_val, (T*)v_val,     \
                                                       status_word())
    if (vec) {
        if (k_val) BSA_APPEND(true, true); else BSA_APPEND(true, false);
    } else {
        if (k_val) BSA_APPEND(false, true); else BSA_APPEND(false, false);
    }
#undef BSA_APPEND
    return check_launch("cache_append_kernel");
}

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsa_cache_bytes(int n_pages, int H, int page_size, int D) {
    if (n_pages < 1 || H < 1 || !page_size_ok(page_size) || D < 16 || D > 128 || D % 16) return 0;
    return (size_t)n_pages * H * (page_size / kStrip) * strip_bytes(D);
}

size_t bsa_cache_tables_workspace(int R) {
    return R <= kSharedRequests ? 0 : (8 + 2 * ((size_t)R + 1)) * sizeof(int32_t);
}

bsa_status bsa_cache_tables(const int32_t* old_lens, int32_t* new_lens, int R, int page_size,
                            int32_t* block_table, int max_pages, int32_t* pool, int n_pages,
                            const int32_t* pool_count, int32_t* pool_count_out, int32_t* query_start,
                            int32_t* token_req, int32_t* token_pos, int64_t* slots, int max_tokens, void* workspace,
                            size_t workspace_bytes, void* stream) {
    BSA_REQUIRE(old_lens && new_lens && block_table && pool && pool_count && pool_count_out && query_start,
                "cache tables: null pointer");
    BSA_REQUIRE(max_tokens == 0 || (token_req && token_pos && slots), "cache tables: null token arrays");
    BSA_REQUIRE(R > 0 && R <= (1 << 20) && max_pages > 0 && n_pages > 0 && max_tokens >= 0 && max_tokens <= (1 << 30),
                "cache tables: sizes out of range (R=%d max_pages=%d n_pages=%d max_tokens=%d)", R, max_pages, n_pages,
                max_tokens);
    BSA_REQUIRE(page_size_ok(page_size), "cache tables: page_size must be a power of two in 16..1024, got %d", page_size);
    BSA_REQUIRE((long long)R * max_pages <= 0x7fffffffLL && (long long)max_pages * page_size <= 0x7fffffffLL,
                "cache tables: R * max_pages and max_pages * page_size must be below 2^31");
    const size_t need = bsa_cache_tables_workspace(R);
    BSA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && ((uintptr_t)workspace & 3) == 0),
                "cache tables: a workspace of %zu bytes is needed", need);
    cudaStream_t st = as_stream(stream);
    const int sh = log2i(page_size);
    Tables a{old_lens, new_lens, R, page_size, max_pages, n_pages, max_tokens, block_table, pool, pool_count,
             pool_count_out, query_start, token_req, token_pos, slots, status_word(),
             (((uintptr_t)token_req | (uintptr_t)token_pos | (uintptr_t)slots) & 15) == 0};
    int32_t* ws = need ? static_cast<int32_t*>(workspace) : nullptr;
    if (one_cta(R, max_tokens)) {
        cache_scan_kernel<true><<<1, kScanThreads, 3 * (R + 1) * sizeof(int32_t), st>>>(a, sh, ws);
        return check_launch("cache_scan_kernel");
    }
    cache_scan_kernel<false><<<1, kScanThreads, 0, st>>>(a, sh, ws);
    bsa_status rc = check_launch("cache_scan_kernel");
    if (rc != BSA_OK) return rc;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = std::min(max_tokens / 1024 + 1, 152 * 4 - kPageBlocks) + kPageBlocks;
    cfg.blockDim = 256;
    cfg.dynamicSmemBytes = R <= kSharedRequests ? 5 * (R + 1) * sizeof(int32_t) : 0;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, R <= kSharedRequests ? cache_place_kernel<true> : cache_place_kernel<false>, a, sh, (const int32_t*)ws);
    return check_launch("cache_place_kernel");
}

bsa_status bsa_cache_append(const void* k, const void* v, bsa_dtype dtype, int T, int H, int D, int64_t k_stride,
                            int64_t v_stride, const int64_t* slots, void* cache, int n_pages, int page_size,
                            const float* k_scale, const float* v_scale, void* k_val, void* v_val, void* stream) {
    BSA_REQUIRE(cache && (T == 0 || (k && v && slots)), "cache append: null pointer");
    BSA_REQUIRE(T == 0 || (k_val == nullptr) == (v_val == nullptr), "cache append: k_val and v_val come together");
    BSA_REQUIRE(dtype == BSA_F32 || dtype == BSA_BF16, "cache append: dtype");
    BSA_REQUIRE(T >= 0 && H > 0 && n_pages > 0, "cache append: sizes out of range (T=%d H=%d n_pages=%d)", T, H, n_pages);
    BSA_REQUIRE(page_size_ok(page_size), "cache append: page_size must be a power of two in 16..1024, got %d", page_size);
    BSA_REQUIRE(D >= 16 && D <= 128 && D % 16 == 0, "cache append: D must be a multiple of 16 up to 128, got %d", D);
    BSA_REQUIRE(H <= (1 << 20) && (T <= 1 || (k_stride >= (int64_t)H * D && v_stride >= (int64_t)H * D)),
                "cache append: a token's stride is below H * D");
    BSA_REQUIRE(((uintptr_t)cache & 15) == 0, "cache append: the cache must be 16-byte aligned");
    if (T == 0) return BSA_OK;
    const long long n_slots = (long long)n_pages * page_size;
    const int sh = log2i(page_size);
    cudaStream_t st = as_stream(stream);
    return dtype == BSA_F32
               ? launch_append<float>(k, v, k_stride, v_stride, T, H, D, slots, (uint8_t*)cache, n_slots, sh, k_scale,
                                      v_scale, k_val, v_val, st)
               : launch_append<__nv_bfloat16>(k, v, k_stride, v_stride, T, H, D, slots, (uint8_t*)cache, n_slots, sh,
                                              k_scale, v_scale, k_val, v_val, st);
}

}  // extern "C"
