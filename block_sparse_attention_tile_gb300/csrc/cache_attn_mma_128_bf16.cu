// Attention over the 4-bit paged cache on the tensor cores (a14): D = 128, bfloat16.
#include "cache_attn_mma.cuh"

namespace bsa {
namespace cmma {

bsa_status launch_128_bf16(const CacheAttn& a, const Sizes& z, bool narrow, cudaStream_t st) {
    return narrow ? launch<128, __nv_bfloat16, true>(a, z, st) : launch<128, __nv_bfloat16, false>(a, z, st);
}

}  // namespace cmma
}  // namespace bsa
