// Variants of the prompt-weights kernel (fa_weights_kernel.cuh): head
// dimension 64 or 128, bf16 or fp16.
#include "fa_weights_kernel.cuh"

namespace fa {

cudaError_t launch_weights(int d, bool f16, const CUtensorMap& q, const CUtensorMap& k, const WeightsParams& p,
                           unsigned int grid, cudaStream_t stream) {
    if (d == 128)
        return f16 ? launch_weights_variant<128, true>(q, k, p, grid, stream)
                   : launch_weights_variant<128, false>(q, k, p, grid, stream);
    return f16 ? launch_weights_variant<64, true>(q, k, p, grid, stream)
               : launch_weights_variant<64, false>(q, k, p, grid, stream);
}

}  // namespace fa
