// kda_wait.cuh -- waits on mbarriers beside those of kda_common.cuh (sm_103a):
// that of kernels with many roles, bounded in time, in a handful of instructions
// where it is used; and what a ring of copies is left with when a wait ran out.
#pragma once

#include "kda_common.cuh"

namespace kda {

// A try of a barrier that nobody completes suspends the warp until the
// hardware's own limit: 7,800 cycles, whatever the number of warps and a time
// hint given with it (measured on GB300; tests/test_gpu_wait_phase.py holds the
// wait's whole time to this).
constexpr long long kTryCycles = 8000;
constexpr uint32_t kWaitTries = static_cast<uint32_t>(kWaitBoundCycles / kTryCycles);
static_assert(kWaitTries > 0 && kWaitBoundCycles / kTryCycles < 1LL << 31, "tries of a wait");

static __device__ __noinline__ void timed_out(int* status) { atomicOr(status, kDevPipeTimeout); }

// Wait, with the whole warp, for a phase of an mbarrier, for kWaitBoundCycles
// (about 2 s) at most.  The bound is a number of tries: the roles of a kernel
// share an instruction cache and their registers are short, and reading the
// clock, even out of line behind 256 to 65,536 tries, made la_prefill 3 to 12%
// slower.  The vote makes the loop's branches the same for the whole warp.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* status) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
        "W%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n vote.sync.all.pred p, p, 0xffffffff;\n"
        " @p bra.uni D%=;\n add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra.uni W%=;\n"
        "D%=:\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "n"(kWaitTries) : "memory");
    if (ok) return true;
    timed_out(status);
    return false;
}

// Before a CTA leaves a ring of `stages` copies early, with one warp: waits for
// the `left` copies under way from stage s on (phase `parity` there, the other
// one behind the ring's end).  False if one does not come.
__device__ __forceinline__ bool drain_ring(uint64_t* full, int stages, int s, uint32_t parity, int left, int* status) {
    for (int i = 0; i < left; ++i) {
        if (!mbar_wait_warp(&full[s], parity, status)) return false;
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    return true;
}

}  // namespace kda
