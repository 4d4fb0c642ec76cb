// kda_ssm_32.cu -- the scan of prompts with rows of up to 32 states.
#include "kda_ssm_scan.cuh"

namespace kda {

cudaError_t ssm_prefill_32(const SsmArgs& a, cudaStream_t stream, int* launches) { return prefill<2>(a, stream, launches); }

}  // namespace kda
