// kda_ssm_64.cu -- the scan of prompts with rows of up to 64 states.
#include "kda_ssm_scan.cuh"

namespace kda {

cudaError_t ssm_prefill_64(const SsmArgs& a, cudaStream_t stream, int* launches) { return prefill<4>(a, stream, launches); }

}  // namespace kda
