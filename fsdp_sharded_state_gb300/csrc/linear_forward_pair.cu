// linear_forward_pair.cu -- the CTA-pair kernels of forward with bf16 results, one per
// activation, with and without dropout, and one for rows of any alignment.
#include "linear_launch.cuh"

namespace fsdp {

cudaError_t launch_pair_forward(const LinProblem& p, int bn, cudaStream_t st) {
    if (p.epi.vec != 2) return launch_pair_as<kForward, uint16_t, 1, 0, -1, true>(p, bn, st);
    switch (p.epi.act + (p.epi.drop.on ? 4 : 0)) {
        case 0: return launch_pair_as<kForward, uint16_t, 1, 0, 0>(p, bn, st);
        case 1: return launch_pair_as<kForward, uint16_t, 1, 0, 1>(p, bn, st);
        case 2: return launch_pair_as<kForward, uint16_t, 1, 0, 2>(p, bn, st);
        case 3: return launch_pair_as<kForward, uint16_t, 1, 0, 3>(p, bn, st);
        case 4: return launch_pair_as<kForward, uint16_t, 1, 0, 4>(p, bn, st);
        case 5: return launch_pair_as<kForward, uint16_t, 1, 0, 5>(p, bn, st);
        case 6: return launch_pair_as<kForward, uint16_t, 1, 0, 6>(p, bn, st);
        case 7: return launch_pair_as<kForward, uint16_t, 1, 0, 7>(p, bn, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t take_wait_error_forward_pair(unsigned int* flag) { return take_product_wait_error(flag); }

}  // namespace fsdp
