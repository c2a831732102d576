// linear_forward.cu -- y = residual + drop(act(x w^T + bias)): the forward product of a
// linear layer and its epilogue.
#include "linear_kernel.cuh"

namespace fsdp {

cudaError_t launch_linear_forward(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3) return launch_cfg<LinCfg<kForward, float, 1, 128, 3, 4, false>>(p, 1, st);
    return launch_cfg<LinCfg<kForward, uint16_t, 1, 128, 1, 0, false>>(p, 1, st);
}

cudaError_t take_wait_error_forward(unsigned int* flag) { return take_local_wait_error(flag); }

}  // namespace fsdp
