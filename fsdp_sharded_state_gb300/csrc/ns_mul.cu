// ns_mul.cu -- instances of the Newton-Schulz product kernel: mul.
#include "ns_kernel.cuh"

namespace fsdp {

cudaError_t launch_ns_mul(const NsProduct& p, cudaStream_t st) { return ns_product<kNsMul>(p, st); }
float cost_ns_mul(const NsProduct& p) { return ns_cost<kNsMul>(p); }
cudaError_t take_wait_error_ns_mul(unsigned int* flag) { return take_ns_wait_error(flag); }

}  // namespace fsdp
