// Attention over packed sequences, bf16: instantiations of the forward and the
// backward kernel.
#include "fa_bwd_kernel.cuh"
#include "fa_packed_fwd.cuh"

namespace fa {

cudaError_t launch_packed_fwd_bf16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                   const PackedFwdParams& p, unsigned int grid, cudaStream_t stream) {
    if (d == 64)
        return p.seqs.causal ? packed::launch_variant<64, false, true>(q, k, v, p, grid, stream)
                             : packed::launch_variant<64, false, false>(q, k, v, p, grid, stream);
    return p.seqs.causal ? packed::launch_variant<128, false, true>(q, k, v, p, grid, stream)
                         : packed::launch_variant<128, false, false>(q, k, v, p, grid, stream);
}

cudaError_t launch_packed_bwd_bf16(int d, const PackedMaps& m, const PackedBwdParams& p, unsigned int grid,
                                 cudaStream_t stream) {
    if (d == 64)
        return p.seqs.causal ? launch_packed_bwd_variant<64, false, true>(m, p, grid, stream)
                             : launch_packed_bwd_variant<64, false, false>(m, p, grid, stream);
    return p.seqs.causal ? launch_packed_bwd_variant<128, false, true>(m, p, grid, stream)
                         : launch_packed_bwd_variant<128, false, false>(m, p, grid, stream);
}

}  // namespace fa
