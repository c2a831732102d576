// linear_wgrad.cu -- dw (+)= dz^T x, the weight gradient of a linear layer, and db (+)= the
// column sums of dz.
#include "linear_kernel.cuh"

namespace fsdp {

cudaError_t launch_linear_wgrad(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3)
        return p.out_bf16 ? launch_product<kWgrad, uint16_t, 3, 0>(p, launch_pair_as<kWgrad, uint16_t, 3, 0>, st)
                          : launch_product<kWgrad, float, 3, 2>(p, launch_pair_as<kWgrad, float, 3, 2>, st);
    return p.out_bf16 ? launch_product<kWgrad, uint16_t, 1, 0>(p, launch_pair_as<kWgrad, uint16_t, 1, 0>, st)
                      : launch_product<kWgrad, float, 1, 8>(p, launch_pair_as<kWgrad, float, 1, 8>, st);
}

cudaError_t take_wait_error_wgrad(unsigned int* flag) { return take_local_wait_error(flag); }

}  // namespace fsdp
