// ns_gram.cu -- instances of the Newton-Schulz product kernel: gram.
#include "ns_kernel.cuh"

namespace fsdp {

cudaError_t launch_ns_gram(const NsProduct& p, cudaStream_t st) { return ns_product<kNsGram>(p, st); }
float cost_ns_gram(const NsProduct& p) { return ns_cost<kNsGram>(p); }
cudaError_t take_wait_error_ns_gram(unsigned int* flag) { return take_ns_wait_error(flag); }

}  // namespace fsdp
