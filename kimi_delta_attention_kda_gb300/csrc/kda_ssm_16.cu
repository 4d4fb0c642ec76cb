// kda_ssm_16.cu -- the scan of prompts with rows of up to 16 states.
#include "kda_ssm_scan.cuh"

namespace kda {

cudaError_t ssm_prefill_16(const SsmArgs& a, cudaStream_t stream, int* launches) { return prefill<1>(a, stream, launches); }

}  // namespace kda
