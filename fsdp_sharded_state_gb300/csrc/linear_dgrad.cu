// linear_dgrad.cu -- dx = residual + act'(z) drop(dz w): the input gradient of a linear
// layer, through the dropout and the activation of the layer before it.
#include "linear_launch.cuh"

namespace fsdp {

cudaError_t launch_linear_dgrad(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3) return launch_product<kDgrad, float, 3, 2>(p, launch_pair_as<kDgrad, float, 3, 2>, st);
    return launch_product<kDgrad, uint16_t, 1, 0>(p, launch_pair_dgrad, st);
}

cudaError_t take_wait_error_dgrad(unsigned int* flag) { return take_product_wait_error(flag); }

}  // namespace fsdp
