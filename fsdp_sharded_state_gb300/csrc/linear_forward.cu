// linear_forward.cu -- y = residual + drop(act(x w^T + bias)): the forward product of a
// linear layer and its epilogue.
#include "linear_launch.cuh"

namespace fsdp {

cudaError_t launch_linear_forward(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3) return launch_product<kForward, float, 3, 2>(p, launch_pair_as<kForward, float, 3, 2>, st);
    return launch_product<kForward, uint16_t, 1, 0>(p, launch_pair_forward, st);
}

cudaError_t take_wait_error_forward(unsigned int* flag) { return take_product_wait_error(flag); }

}  // namespace fsdp
