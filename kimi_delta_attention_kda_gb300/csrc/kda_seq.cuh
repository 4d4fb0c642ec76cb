// kda_seq.cuh -- where a CTA of the convolution and of the scan stands in a
// packed batch: the offsets' check and the sequence of a token (sm_103a).
#pragma once

#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {

// Waits for the end of the kernel before this one in the stream: every kernel
// launched by launch_after does so ahead of its first access to global memory.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be placed where this one leaves room.
__device__ __forceinline__ void let_next_kernel_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// a / b for a >= 0 and b > 0: 64-bit division costs a hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// The number of sequences that end at or before token `key`, for non-decreasing offsets.
__device__ __forceinline__ int64_t ended_by(const int64_t* cu, int64_t n_seqs, int64_t key) {
    int64_t lo = 0, hi = n_seqs;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (cu[mid + 1] <= key)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Whether the offsets keep their contract, with the whole CTA.  `valid` is the
// verdict of a kernel before this one, or null where there are few offsets: then
// every CTA looks at them all, and the first reports.
__device__ __forceinline__ bool offsets_hold(const int64_t* cu, int64_t n_seqs, int64_t tokens, const int32_t* valid, int* status) {
    if (valid) return *valid != 0;
    bool ok = threadIdx.x > 0 || (cu[0] == 0 && cu[n_seqs] == tokens);
    for (int64_t n = threadIdx.x; n < n_seqs; n += blockDim.x) ok = ok && cu[n] <= cu[n + 1];
    ok = __syncthreads_and(ok);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kDevBadSeqlens);
    return ok;
}

// A launch that is set up while what the stream has before it ends.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute after;
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &after;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kda
