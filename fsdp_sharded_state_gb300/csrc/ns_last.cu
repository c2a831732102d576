// ns_last.cu -- instances of the Newton-Schulz product kernel: last.
#include "ns_kernel.cuh"

namespace fsdp {

cudaError_t launch_ns_last(const NsProduct& p, cudaStream_t st) { return ns_product<kNsLast>(p, st); }
cudaError_t take_wait_error_ns_last(unsigned int* flag) { return take_ns_wait_error(flag); }

}  // namespace fsdp
