// ns_poly.cu -- instances of the Newton-Schulz product kernel: poly.
#include "ns_kernel.cuh"

namespace fsdp {

cudaError_t launch_ns_poly(const NsProduct& p, cudaStream_t st) { return ns_product<kNsPoly>(p, st); }
cudaError_t take_wait_error_ns_poly(unsigned int* flag) { return take_ns_wait_error(flag); }

}  // namespace fsdp
