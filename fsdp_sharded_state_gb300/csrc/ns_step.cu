// ns_step.cu -- instances of the Newton-Schulz product kernel: step.
#include "ns_kernel.cuh"

namespace fsdp {

cudaError_t launch_ns_step(const NsProduct& p, cudaStream_t st) { return ns_product<kNsStep>(p, st); }
float cost_ns_step(const NsProduct& p) { return ns_cost<kNsStep>(p); }
cudaError_t take_wait_error_ns_step(unsigned int* flag) { return take_ns_wait_error(flag); }

}  // namespace fsdp
