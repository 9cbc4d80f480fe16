// Attention over the paged key/value cache, bf16: instantiations of
// its kernels and of the packed forward kernel over a prefix.
#include "fa_packed_fwd.cuh"
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_fwd_bf16(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                                cudaStream_t stream) {
    return p.c.d == 64 ? paged::launch<64, false>(q, k, v, p, stream) : paged::launch<128, false>(q, k, v, p, stream);
}

cudaError_t launch_prefix_fwd_bf16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                   const PrefixFwdParams& p, cudaStream_t stream) {
    return d == 64 ? packed::launch_prefix<64, false>(q, k, v, p, stream)
                   : packed::launch_prefix<128, false>(q, k, v, p, stream);
}

}  // namespace fa
